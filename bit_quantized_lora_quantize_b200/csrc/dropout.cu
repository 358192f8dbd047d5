// Dropout from a counter-based generator: Y = keep * (X * gain) [+ residual].
//
// The mask is a function of (seed, counter) alone, so the backward pass draws
// it again and it is never stored: a training step moves the activations and
// nothing else.  One 128-bit Philox output serves eight elements with 16 bits
// each: about 100 instructions per group of eight with the rest of the work,
// two thirds of what the SMs can issue in the time HBM needs to move the group
// in bf16.  Elementwise and HBM-bound: each thread loads its groups first and
// draws while the loads are in flight; float32 arithmetic, one rounding per
// output.  Measured by replayed graphs: 8192 x 11008 in bf16 55.3 us = 6.5 TB/s,
// 0.99 of the measured copy bandwidth (single calls with the host between them
// 61.6).  Ragged rows take scalar accesses and are bound by their number: 119 us
// for 8192 x 11007; in fp16 7.0 us for 777 x 5003, against 4.1 of 777 x 5000.
//
// Dropped elements are selected away, not multiplied by zero: an infinity or
// a NaN there leaves no trace.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "abi_internal.h"
#include "kernels.h"
#include "ptx.cuh"
#include "rows_host.h"

namespace qlora {

namespace {

constexpr int kDropThreads = 256;

__device__ __forceinline__ float drop_value(float x, float r, bool keep, float gain) {
  return keep ? fmaf(x, gain, r) : r;
}

// Aligned rows: groups of eight are consecutive in memory and in the counter.
template <typename T, bool RES, int U>
__global__ void __launch_bounds__(kDropThreads)
    dropout_vec_kernel(const T* __restrict__ X, const T* __restrict__ R, T* __restrict__ Y, int64_t ngroups,
                       const DropArgs d) {
  griddep_launch_dependents();  // a GEMM that reads Y may set itself up meanwhile
  const int64_t g0 = static_cast<int64_t>(blockIdx.x) * (kDropThreads * U) + threadIdx.x;
  const uint64_t base = drop_base(d);
  Raw8<T> x[U], r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t g = g0 + u * kDropThreads;
    if (g < ngroups) {
      x[u] = load_group_stream(X + g * 8);
      if (RES) r[u] = load_group_stream(R + g * 8);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t g = g0 + u * kDropThreads;
    if (g >= ngroups) return;
    const KeepGroup keep = keep_group(d, base + g);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = drop_value(raw_f32(x[u], e), RES ? raw_f32(r[u], e) : 0.0f, keep(e), d.gain);
    store_group_stream(Y + g * 8, raw_from<T>(v));
  }
}

// Ragged rows: one warp per 256 columns of a row, scalar accesses.
template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads)
    dropout_ragged_kernel(const T* __restrict__ X, const T* __restrict__ R, T* __restrict__ Y, int cols,
                          int64_t chunks_per_row, int64_t nchunks, const DropArgs d) {
  const int lane = threadIdx.x & 31;
  const int64_t chunk = static_cast<int64_t>(blockIdx.x) * (kDropThreads / 32) + (threadIdx.x >> 5);
  if (chunk >= nchunks) return;
  // (a 64-bit division takes as many instructions as a draw)
  const int64_t row = nchunks >> 32 ? chunk / chunks_per_row
                                    : static_cast<uint32_t>(chunk) / static_cast<uint32_t>(chunks_per_row);
  const int c0 = static_cast<int>(chunk - row * chunks_per_row) * 256;
  const int64_t at = row * cols;
  const Raw8<T> x = load_cols<kRagged>(X + at, c0, cols, lane);
  Raw8<T> r;
  if (RES) r = load_cols<kRagged>(R + at, c0, cols, lane);
  const KeepBits keep = keep_cols<kRagged>(d, drop_base(d) + row * d.groups + c0 / 8, lane);
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = drop_value(raw_f32(x, e), RES ? raw_f32(r, e) : 0.0f, keep(e), d.gain);
  store_cols<kRagged>(Y + at, c0, cols, lane, raw_from<T>(v));
}

template <typename T, bool RES>
cudaError_t launch_typed(const T* X, const T* R, T* Y, int64_t rows, int64_t cols, const DropArgs& d,
                         cudaStream_t stream) {
  if (vector_rows(X, cols) && vector_rows(Y, cols) && (!RES || vector_rows(R, cols))) {
    const int64_t n = rows * (cols / 8);
    // Four groups in flight per thread once that still fills every SM (bf16,
    // 8192 x 11008: 55.6 us, 70.4 with one; 1024 x 8192: 6.8 against 8.0).
    if (n >= static_cast<int64_t>(device_sm_count()) * kDropThreads * 16) {
      const int64_t grid = (n + kDropThreads * 4 - 1) / (kDropThreads * 4);
      dropout_vec_kernel<T, RES, 4><<<static_cast<unsigned>(grid), kDropThreads, 0, stream>>>(X, R, Y, n, d);
    } else {
      const int64_t grid = (n + kDropThreads - 1) / kDropThreads;
      dropout_vec_kernel<T, RES, 1><<<static_cast<unsigned>(grid), kDropThreads, 0, stream>>>(X, R, Y, n, d);
    }
  } else {
    const int64_t per_row = (cols + 255) / 256, n = rows * per_row;
    const int64_t grid = (n + kDropThreads / 32 - 1) / (kDropThreads / 32);
    dropout_ragged_kernel<T, RES>
        <<<static_cast<unsigned>(grid), kDropThreads, 0, stream>>>(X, R, Y, static_cast<int>(cols), per_row, n, d);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_any(const void* X, const void* R, void* Y, int64_t rows, int64_t cols, const DropArgs& d,
                       cudaStream_t stream) {
  const T* x = static_cast<const T*>(X);
  const T* r = static_cast<const T*>(R);
  T* y = static_cast<T*>(Y);
  return r ? launch_typed<T, true>(x, r, y, rows, cols, d, stream)
           : launch_typed<T, false>(x, r, y, rows, cols, d, stream);
}

}  // namespace

cudaError_t launch_dropout(int32_t dtype, const void* X, const void* residual, void* Y, int64_t rows, int64_t cols,
                           const DropArgs& d, cudaStream_t stream) {
  if (dtype == QLORA_DTYPE_BF16) return launch_any<__nv_bfloat16>(X, residual, Y, rows, cols, d, stream);
  if (dtype == QLORA_DTYPE_FP16) return launch_any<__half>(X, residual, Y, rows, cols, d, stream);
  return launch_any<float>(X, residual, Y, rows, cols, d, stream);
}

}  // namespace qlora

using namespace qlora;

extern "C" {

qlora_status qlora_dropout_fwd(const void* X, const void* residual, void* Y, int64_t rows, int64_t cols,
                               int32_t dtype, double p, uint64_t seed, uint64_t offset, const uint64_t* offset_dev,
                               void* stream) {
  if (!X || !Y || !known_dtype(dtype)) return QLORA_ERR_INVALID_ARG;
  const qlora_status sh = check_rows(rows, cols);
  if (sh != QLORA_OK) return sh;
  DropArgs d;
  if (!(p >= 0.0 && p <= 1.0)) return QLORA_ERR_INVALID_ARG;
  const int es = dtype_bytes(dtype);
  if (!aligned_to(X, es) || !aligned_to(Y, es) || !aligned_to(residual, es) ||
      !make_drop_args(p, seed, offset, offset_dev, cols, &d))
    return QLORA_ERR_ALIGNMENT;
  const int64_t n = rows * cols * es;
  if (!disjoint({{Y, n}}, {{X, n}, {residual, n}})) return QLORA_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope prof(st, "dropout", 1);
  const cudaError_t e = launch_dropout(dtype, X, residual, Y, rows, cols, d, st);
  prof.done();
  return e == cudaSuccess ? QLORA_OK : cuda_fail(e);
}

qlora_status qlora_dropout_bwd(const void* dY, void* dX, int64_t rows, int64_t cols, int32_t dtype, double p,
                               uint64_t seed, uint64_t offset, const uint64_t* offset_dev, void* stream) {
  return qlora_dropout_fwd(dY, nullptr, dX, rows, cols, dtype, p, seed, offset, offset_dev, stream);
}

}  // extern "C"
