// Layer norm over the rows of a matrix, forward and backward, alone or fused
// with the residual dropout in front of it:
//
//   Z = residual + dropout(X)                       (fused form; else Z = X)
//   mean = sum(z) / n,  var = sum((z - mean)^2) / n,  rstd = 1 / sqrt(var + eps)
//   h = (z - mean) rstd,  Y = h weight + bias
//
//   g = dY weight,  dz = rstd (g - sum(g) / n - h sum(g h) / n) [+ dZ]
//   dweight = sum over rows of dY h,  dbias = sum over rows of dY
//   fused form: dresidual = dz, dX = dropout(dz) with the forward's draws
//
// All of it is HBM-bound: a row is read once into registers, the mean first
// and then the squared distances from it (no difference of large sums), both
// in float32.  The fused form takes the statistics of Z as rounded to its
// type, which is what the backward pass reads.
//
// Forward: `wpr` warps share a row, 256 columns per warp and step, so that a
// row of up to 32768 columns stays in registers; many rows per SM hide each
// other's reduction.  With few rows each gets as many warps as its columns
// allow instead (one step per warp).  Longer rows are read three times.
//
// Backward: one persistent block per SM walks over the rows.  A ring of
// stages in shared memory, filled by bulk copies, keeps whole rows of dY and Z
// in flight while earlier ones are reduced; each thread carries the sums of
// dweight and dbias for its columns in registers across all rows of the block.
// The blocks' partial sums are added by a second, small kernel in a fixed
// order, so results are the same from run to run.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "abi_internal.h"
#include "kernels.h"
#include "ptx.cuh"
#include "rows_host.h"

namespace qlora {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kFwdMaxGroups = 4;         // steps of 256 columns a warp holds in the forward
constexpr int kBwdGroups = 2;            // the same in the backward
constexpr int kBwdWarps = 16;
constexpr int kBwdCols = kBwdWarps * 256 * kBwdGroups;  // widest row of the ring kernel
constexpr int kBwdMaxBlocks = 160;       // partial sums in the workspace
constexpr int kRingBytes = 200 * 1024;
constexpr int kMaxStages = 8;
constexpr size_t kLnStatusBytes = 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Sum over the wpr warps of a row; `buf` holds one float per warp.  Every
// thread of the block calls it.
__device__ __forceinline__ float row_sum(float v, float* buf, int warp, int first, int wpr) {
  v = warp_sum(v);
  if (wpr == 1) return v;
  if ((threadIdx.x & 31) == 0) buf[warp] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < wpr; ++i) s += buf[first + i];
  return s;
}

template <bool VEC>
__device__ __forceinline__ bool col_in(int64_t c0, int lane, int e, int64_t cols) {
  return c0 + warp_col<VEC>(lane, e) < cols;
}

struct LnFwdArgs {
  const void* x;
  const void* residual;
  const void* w;
  const void* b;
  void* z;
  void* y;
  float* mean;
  float* rstd;
  int64_t rows, cols;
  float eps, inv_n;
  int wpr;
  DropArgs drop;
};

// Values of one lane's eight columns after the residual dropout, rounded to
// T and stored to Z.
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> add_dropped(const LnFwdArgs& a, int64_t row, int64_t c0, int lane, uint64_t base,
                                               const Raw8<T>& x) {
  const int64_t at = row * a.cols;
  const Raw8<T> r = load_cols<VEC>(static_cast<const T*>(a.residual) + at, c0, a.cols, lane);
  const uint32_t keep = keep_bits_cols<VEC>(a.drop, base + row * a.drop.groups + c0 / 8, lane);
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = ((keep >> e) & 1u) ? fmaf(raw_f32(x, e), a.drop.gain, raw_f32(r, e)) : raw_f32(r, e);
  store_cols<VEC>(static_cast<T*>(a.z) + at, c0, a.cols, lane, v);
  return raw_from<T>(v);
}

template <typename T, typename W, bool VEC>
__device__ __forceinline__ void normalise(const LnFwdArgs& a, int64_t row, int64_t c0, int lane, float mean, float rstd,
                                          const Raw8<T>& x) {
  Raw8<W> w, b;
  if (a.w) w = load_cols<VEC>(static_cast<const W*>(a.w), c0, a.cols, lane);
  if (a.b) b = load_cols<VEC>(static_cast<const W*>(a.b), c0, a.cols, lane);
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = fmaf((raw_f32(x, e) - mean) * rstd, a.w ? raw_f32(w, e) : 1.0f, a.b ? raw_f32(b, e) : 0.0f);
  store_cols<VEC>(static_cast<T*>(a.y) + row * a.cols, c0, a.cols, lane, v);
}

template <typename T, typename W, int G, bool VEC, bool FUSED>
__global__ void __launch_bounds__(1024) ln_fwd_kernel(const LnFwdArgs a) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % a.wpr, first = warp - part;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32 / a.wpr) + warp / a.wpr;
  const bool valid = row < a.rows;
  const T* xr = static_cast<const T*>(a.x) + row * a.cols;
  Raw8<T> x[G];
  float s = 0.0f;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t c0 = static_cast<int64_t>(part + g * a.wpr) * 256;
    if (valid && c0 < a.cols) x[g] = load_cols<VEC>(xr, c0, a.cols, lane);
  }
  const uint64_t base = FUSED ? drop_base(a.drop) : 0;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t c0 = static_cast<int64_t>(part + g * a.wpr) * 256;
    if (valid && c0 < a.cols) {
      if (FUSED) x[g] = add_dropped<T, VEC>(a, row, c0, lane, base, x[g]);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col_in<VEC>(c0, lane, e, a.cols)) s += raw_f32(x[g], e);
    }
  }
  const float mean = row_sum(s, red[0], warp, first, a.wpr) * a.inv_n;
  float q = 0.0f;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t c0 = static_cast<int64_t>(part + g * a.wpr) * 256;
    if (valid && c0 < a.cols) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = raw_f32(x[g], e) - mean;
        if (col_in<VEC>(c0, lane, e, a.cols)) q = fmaf(d, d, q);
      }
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum(q, red[1], warp, first, a.wpr) * a.inv_n + a.eps);
  if (!valid) return;
  if (part == 0 && lane == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t c0 = static_cast<int64_t>(part + g * a.wpr) * 256;
    if (c0 < a.cols) normalise<T, W, VEC>(a, row, c0, lane, mean, rstd, x[g]);
  }
}

// Rows too long for the registers of a block: three passes, the later ones
// mostly from L2.
template <typename T, typename W, bool FUSED>
__global__ void __launch_bounds__(1024) ln_fwd_long_kernel(const LnFwdArgs a) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const T* xr = static_cast<const T*>(a.x) + row * a.cols;
  const uint64_t base = FUSED ? drop_base(a.drop) : 0;
  float s = 0.0f;
  for (int64_t c0 = static_cast<int64_t>(warp) * 256; c0 < a.cols; c0 += 32 * 256) {
    Raw8<T> x = load_cols<false>(xr, c0, a.cols, lane);
    if (FUSED) x = add_dropped<T, false>(a, row, c0, lane, base, x);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col_in<false>(c0, lane, e, a.cols)) s += raw_f32(x, e);
  }
  const float mean = row_sum(s, red[0], warp, 0, 32) * a.inv_n;
  // Each thread reads back only what it stored itself.
  const T* zr = FUSED ? static_cast<const T*>(a.z) + row * a.cols : xr;
  float q = 0.0f;
  for (int64_t c0 = static_cast<int64_t>(warp) * 256; c0 < a.cols; c0 += 32 * 256) {
    const Raw8<T> x = load_cols<false>(zr, c0, a.cols, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = raw_f32(x, e) - mean;
      if (col_in<false>(c0, lane, e, a.cols)) q = fmaf(d, d, q);
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum(q, red[1], warp, 0, 32) * a.inv_n + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  for (int64_t c0 = static_cast<int64_t>(warp) * 256; c0 < a.cols; c0 += 32 * 256)
    normalise<T, W, false>(a, row, c0, lane, mean, rstd, load_cols<false>(zr, c0, a.cols, lane));
}

// ---------------------------------------------------------------- backward
struct LnBwdArgs {
  const void* dy;
  const void* z;
  const void* dz;    // fused form: gradient that reaches Z directly, or null
  const float* mean;
  const float* rstd;
  const void* w;
  void* dx;          // fused form: dropout(dz total); else dz itself
  void* dres;        // fused form: dz total
  float* part;       // [blocks][2][cols] sums of dweight and dbias, or null
  int64_t rows, cols;
  float inv_n;
  int wpr;
  int stages;
  uint32_t tensor_bytes;  // one tensor's rows in a stage
  int* status;
  uint64_t wait_ns;
  DropArgs drop;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ float grad_value(float dy, float h, float w, float s1, float s2, float rstd) {
  return rstd * (fmaf(dy, w, -s1) - h * s2);
}

template <typename T, bool VEC, bool FUSED>
__device__ __forceinline__ void store_grad(const LnBwdArgs& a, int64_t row, int64_t c0, int lane, uint64_t base,
                                           float (&v)[8]) {
  const int64_t at = row * a.cols;
  if (!FUSED) {
    store_cols<VEC>(static_cast<T*>(a.dx) + at, c0, a.cols, lane, v);
    return;
  }
  store_cols<VEC>(static_cast<T*>(a.dres) + at, c0, a.cols, lane, v);
  const uint32_t keep = keep_bits_cols<VEC>(a.drop, base + row * a.drop.groups + c0 / 8, lane);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = ((keep >> e) & 1u) ? v[e] * a.drop.gain : 0.0f;
  store_cols<VEC>(static_cast<T*>(a.dx) + at, c0, a.cols, lane, v);
}

// RING: aligned rows through the ring of bulk copies; otherwise ragged rows
// by scalar loads.
template <typename T, typename W, bool RING, bool FUSED>
__global__ void __launch_bounds__(kBwdWarps * 32, 1) ln_bwd_kernel(const LnBwdArgs a) {
  constexpr int G = kBwdGroups;
  constexpr bool VEC = RING;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[2][2][kBwdWarps];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  __shared__ volatile int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % a.wpr, first = warp - part, slot = warp / a.wpr;
  const int rpi = kBwdWarps / a.wpr;  // rows per step of the block
  const int64_t steps = (a.rows + rpi - 1) / rpi;
  const int64_t mine = (steps - blockIdx.x + gridDim.x - 1) / gridDim.x;
  const bool has_dz = FUSED && a.dz;
  const int tensors = has_dz ? 3 : 2;
  const uint32_t stage_bytes = a.tensor_bytes * tensors;
  int64_t issued = 0;  // by thread 0

  auto issue = [&](int64_t i) {
    ++issued;
    const int s = static_cast<int>(i % a.stages);
    const int64_t row = (blockIdx.x + i * gridDim.x) * rpi;
    const uint32_t bytes = static_cast<uint32_t>(min(static_cast<int64_t>(rpi), a.rows - row) * a.cols * sizeof(T));
    uint8_t* dst = ring + s * stage_bytes;
    const int64_t at = row * a.cols;
    mbar_arrive_expect_tx(&full[s], bytes * tensors);
    bulk_load(dst, static_cast<const T*>(a.dy) + at, bytes, &full[s]);
    bulk_load(dst + a.tensor_bytes, static_cast<const T*>(a.z) + at, bytes, &full[s]);
    if (has_dz) bulk_load(dst + 2 * a.tensor_bytes, static_cast<const T*>(a.dz) + at, bytes, &full[s]);
  };

  if (RING) {
    if (threadIdx.x == 0) {
      for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1);
      abort_flag = 0;
      fence_mbarrier_init();
      for (int64_t i = 0; i < min(mine, static_cast<int64_t>(a.stages)); ++i) issue(i);
    }
    __syncthreads();
  }
  const WaitCtx ctx{&abort_flag, a.status, 41, a.wait_ns};
  const uint64_t base = FUSED ? drop_base(a.drop) : 0;

  Raw8<W> w[G];
  float aw[G][8], ab[G][8];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t c0 = static_cast<int64_t>(part + g * a.wpr) * 256;
    if (a.w && c0 < a.cols) w[g] = load_cols<VEC>(static_cast<const W*>(a.w), c0, a.cols, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) aw[g][e] = ab[g][e] = 0.0f;
  }
  float mean_n = 0.0f, rstd_n = 0.0f;
  {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * rpi + slot;
    if (mine > 0 && row < a.rows) {
      mean_n = __ldg(a.mean + row);
      rstd_n = __ldg(a.rstd + row);
    }
  }

  for (int64_t i = 0; i < mine; ++i) {
    const int64_t row = (blockIdx.x + i * gridDim.x) * rpi + slot;
    const bool valid = row < a.rows;
    const float mean = mean_n, rstd = rstd_n;
    const int64_t row_n = row + static_cast<int64_t>(gridDim.x) * rpi;
    if (i + 1 < mine && row_n < a.rows) {
      mean_n = __ldg(a.mean + row_n);
      rstd_n = __ldg(a.rstd + row_n);
    }
    const int s = RING ? static_cast<int>(i % a.stages) : 0;
    if (RING) mbar_wait(&full[s], static_cast<uint32_t>((i / a.stages) & 1), ctx);
    const T* dyr = RING ? reinterpret_cast<const T*>(ring + s * stage_bytes) + slot * a.cols
                        : static_cast<const T*>(a.dy) + row * a.cols;
    const T* zr = RING ? reinterpret_cast<const T*>(ring + s * stage_bytes + a.tensor_bytes) + slot * a.cols
                       : static_cast<const T*>(a.z) + row * a.cols;
    const T* dzr = RING ? reinterpret_cast<const T*>(ring + s * stage_bytes + 2 * a.tensor_bytes) + slot * a.cols
                        : static_cast<const T*>(a.dz) + row * a.cols;
    Raw8<T> dy[G], z[G], dz[G];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t c0 = static_cast<int64_t>(part + g * a.wpr) * 256;
      if (valid && c0 < a.cols) {
        dy[g] = load_cols<VEC>(dyr, c0, a.cols, lane);
        z[g] = load_cols<VEC>(zr, c0, a.cols, lane);
        if (has_dz) dz[g] = load_cols<VEC>(dzr, c0, a.cols, lane);
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t c0 = static_cast<int64_t>(part + g * a.wpr) * 256;
      if (valid && c0 < a.cols) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // columns past the end hold dY = 0 and add nothing
          const float d = raw_f32(dy[g], e);
          const float h = col_in<VEC>(c0, lane, e, a.cols) ? (raw_f32(z[g], e) - mean) * rstd : 0.0f;
          const float gr = a.w ? d * raw_f32(w[g], e) : d;
          s1 += gr;
          s2 = fmaf(gr, h, s2);
          aw[g][e] = fmaf(d, h, aw[g][e]);
          ab[g][e] += d;
        }
      }
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    float(*rb)[kBwdWarps] = red[i & 1];
    if (lane == 0) {
      rb[0][warp] = s1;
      rb[1][warp] = s2;
    }
    __syncthreads();  // sums visible; the stage has been read by everyone
    if (RING && threadIdx.x == 0 && i + a.stages < mine && !abort_flag) issue(i + a.stages);
    s1 = s2 = 0.0f;
    for (int k = 0; k < a.wpr; ++k) {
      s1 += rb[0][first + k];
      s2 += rb[1][first + k];
    }
    s1 *= a.inv_n;
    s2 *= a.inv_n;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t c0 = static_cast<int64_t>(part + g * a.wpr) * 256;
      if (valid && c0 < a.cols) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float h = (raw_f32(z[g], e) - mean) * rstd;
          v[e] = grad_value(raw_f32(dy[g], e), h, a.w ? raw_f32(w[g], e) : 1.0f, s1, s2, rstd);
          if (has_dz) v[e] += raw_f32(dz[g], e);
        }
        store_grad<T, VEC, FUSED>(a, row, c0, lane, base, v);
      }
    }
  }

  if (RING && abort_flag) {
    // Copies still in flight must land before the block leaves.
    if (threadIdx.x == 0)
      for (int64_t i = max(int64_t(0), issued - a.stages); i < issued; ++i)
        mbar_drain(&full[i % a.stages], static_cast<uint32_t>((i / a.stages) & 1));
    __syncthreads();
  }
  if (!a.part) return;
  // Add the row slots' sums in shared memory, slot by slot in order.
  float* pw = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
  float* acc = reinterpret_cast<float*>(ring);
  __syncthreads();
  for (int k = 0; k < rpi; ++k) {
    if (slot == k) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int64_t c0 = static_cast<int64_t>(part + g * a.wpr) * 256;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int64_t c = c0 + warp_col<VEC>(lane, e);
          if (c < a.cols) {
            const float vw = k ? acc[c] + aw[g][e] : aw[g][e];
            const float vb = k ? acc[a.cols + c] + ab[g][e] : ab[g][e];
            if (k + 1 < rpi) {
              acc[c] = vw;
              acc[a.cols + c] = vb;
            } else {
              pw[c] = vw;
              pw[a.cols + c] = vb;
            }
          }
        }
      }
    }
    if (k + 1 < rpi) __syncthreads();
  }
}

// dweight / dbias = sum of the blocks' partial sums, in block order within
// each of eight interleaved chains.
__global__ void __launch_bounds__(256) ln_param_sum_kernel(const float* __restrict__ part, int blocks, int64_t cols,
                                                           float* dw, float* db) {
  __shared__ float red[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  float s = 0.0f;
  if (c < cols)
    for (int b = warp; b < blocks; b += 8) s += part[(static_cast<int64_t>(b) * 2 + blockIdx.y) * cols + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += red[k][lane];
    out[c] = s;
  }
}

// Rows too long for the ring kernel's registers: one block per row for the
// input gradient, reading the row twice.
template <typename T, typename W, bool FUSED>
__global__ void __launch_bounds__(1024) ln_bwd_long_kernel(const LnBwdArgs a) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x, at = row * a.cols;
  const T* dyr = static_cast<const T*>(a.dy) + at;
  const T* zr = static_cast<const T*>(a.z) + at;
  const W* wr = static_cast<const W*>(a.w);
  const float mean = __ldg(a.mean + row), rstd = __ldg(a.rstd + row);
  const uint64_t base = FUSED ? drop_base(a.drop) : 0;
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t c0 = static_cast<int64_t>(warp) * 256; c0 < a.cols; c0 += 32 * 256) {
    const Raw8<T> dy = load_cols<false>(dyr, c0, a.cols, lane);
    const Raw8<T> z = load_cols<false>(zr, c0, a.cols, lane);
    Raw8<W> w;
    if (wr) w = load_cols<false>(wr, c0, a.cols, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float h = col_in<false>(c0, lane, e, a.cols) ? (raw_f32(z, e) - mean) * rstd : 0.0f;
      const float gr = wr ? raw_f32(dy, e) * raw_f32(w, e) : raw_f32(dy, e);
      s1 += gr;
      s2 = fmaf(gr, h, s2);
    }
  }
  s1 = row_sum(s1, red[0], warp, 0, 32) * a.inv_n;
  s2 = row_sum(s2, red[1], warp, 0, 32) * a.inv_n;
  for (int64_t c0 = static_cast<int64_t>(warp) * 256; c0 < a.cols; c0 += 32 * 256) {
    const Raw8<T> dy = load_cols<false>(dyr, c0, a.cols, lane);
    const Raw8<T> z = load_cols<false>(zr, c0, a.cols, lane);
    Raw8<W> w;
    if (wr) w = load_cols<false>(wr, c0, a.cols, lane);
    Raw8<T> dz;
    if (FUSED && a.dz) dz = load_cols<false>(static_cast<const T*>(a.dz) + at, c0, a.cols, lane);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float h = (raw_f32(z, e) - mean) * rstd;
      v[e] = grad_value(raw_f32(dy, e), h, wr ? raw_f32(w, e) : 1.0f, s1, s2, rstd);
      if (FUSED && a.dz) v[e] += raw_f32(dz, e);
    }
    store_grad<T, false, FUSED>(a, row, c0, lane, base, v);
  }
}

// The parameter gradients of such rows: block (x, y) sums 256 columns over
// the rows y, y + gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(256) ln_param_long_kernel(const LnBwdArgs a) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float sw = 0.0f, sb = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float d = to_f32(static_cast<const T*>(a.dy)[row * a.cols + c]);
    const float h = (to_f32(static_cast<const T*>(a.z)[row * a.cols + c]) - __ldg(a.mean + row)) * __ldg(a.rstd + row);
    sw = fmaf(d, h, sw);
    sb += d;
  }
  float* pw = a.part + static_cast<int64_t>(blockIdx.y) * 2 * a.cols;
  pw[c] = sw;
  pw[a.cols + c] = sb;
}

// ---------------------------------------------------------------- launches
// Warps per row: the fewest whose `groups` steps of 256 columns cover it.
int warps_for(int64_t cols, int groups) {
  int w = 1;
  while (static_cast<int64_t>(w) * 256 * groups < cols) w *= 2;
  return w;
}

template <typename T, typename W, bool VEC, bool FUSED>
cudaError_t launch_fwd(LnFwdArgs a, cudaStream_t stream) {
  if (a.cols > 32 * 256 * kFwdMaxGroups) {
    ln_fwd_long_kernel<T, W, FUSED><<<static_cast<unsigned>(a.rows), 1024, 0, stream>>>(a);
    return cudaGetLastError();
  }
  // Few rows: one step per warp where 32 warps allow it, for latency.
  // Otherwise four steps, so that several rows share an SM.
  int groups = kFwdMaxGroups;
  if (a.rows <= 2 * device_sm_count())
    for (groups = 1; groups < kFwdMaxGroups && warps_for(a.cols, groups) > 32;) groups *= 2;
  a.wpr = warps_for(a.cols, groups);
  while (groups > 1 && static_cast<int64_t>(a.wpr) * 256 * (groups / 2) >= a.cols) groups /= 2;
  const int warps = std::max(a.wpr, 4);
  const int64_t rpb = warps / a.wpr;
  const unsigned grid = static_cast<unsigned>((a.rows + rpb - 1) / rpb);
  if (groups == 1) ln_fwd_kernel<T, W, 1, VEC, FUSED><<<grid, warps * 32, 0, stream>>>(a);
  else if (groups == 2) ln_fwd_kernel<T, W, 2, VEC, FUSED><<<grid, warps * 32, 0, stream>>>(a);
  else ln_fwd_kernel<T, W, 4, VEC, FUSED><<<grid, warps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, typename W>
cudaError_t launch_fwd_any(const LnFwdArgs& a, bool vec, bool fused, cudaStream_t stream) {
  if (fused) return vec ? launch_fwd<T, W, true, true>(a, stream) : launch_fwd<T, W, false, true>(a, stream);
  return vec ? launch_fwd<T, W, true, false>(a, stream) : launch_fwd<T, W, false, false>(a, stream);
}

cudaError_t launch_ln_fwd(const LnFwdArgs& a, int32_t dtype, int32_t wdtype, bool fused, cudaStream_t stream) {
  const bool vec = vector_rows(a.x, a.cols) && vector_rows(a.y, a.cols) && vector_rows(a.w, a.cols) &&
                   vector_rows(a.b, a.cols) && (!fused || (vector_rows(a.residual, a.cols) && vector_rows(a.z, a.cols)));
  if (dtype == QLORA_DTYPE_FP32) return launch_fwd_any<float, float>(a, vec, fused, stream);
  if (dtype == QLORA_DTYPE_BF16)
    return wdtype == dtype ? launch_fwd_any<__nv_bfloat16, __nv_bfloat16>(a, vec, fused, stream)
                           : launch_fwd_any<__nv_bfloat16, float>(a, vec, fused, stream);
  return wdtype == dtype ? launch_fwd_any<__half, __half>(a, vec, fused, stream)
                         : launch_fwd_any<__half, float>(a, vec, fused, stream);
}

// Stages of the ring for these rows (0: a stage does not fit).
int ring_stages(int64_t stage_bytes) {
  return static_cast<int>(std::min<int64_t>(kMaxStages, kRingBytes / stage_bytes));
}

template <typename T, typename W, bool RING, bool FUSED>
cudaError_t launch_bwd_rows(const LnBwdArgs& a, int grid, size_t smem, cudaStream_t stream) {
  auto kern = ln_bwd_kernel<T, W, RING, FUSED>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingBytes));
  if (e != cudaSuccess) return e;
  kern<<<grid, kBwdWarps * 32, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, typename W, bool FUSED>
cudaError_t launch_bwd(LnBwdArgs a, bool vec, float* dw, float* db, cudaStream_t stream) {
  int blocks;
  cudaError_t e;
  if (a.cols > kBwdCols) {
    ln_bwd_long_kernel<T, W, FUSED><<<static_cast<unsigned>(a.rows), 1024, 0, stream>>>(a);
    e = cudaGetLastError();
    blocks = static_cast<int>(std::min<int64_t>(a.rows, 64));
    if (e == cudaSuccess && a.part) {
      const dim3 grid(static_cast<unsigned>((a.cols + 255) / 256), static_cast<unsigned>(blocks));
      ln_param_long_kernel<T><<<grid, 256, 0, stream>>>(a);
      e = cudaGetLastError();
    }
  } else {
    a.wpr = warps_for(a.cols, kBwdGroups);
    const int rpi = kBwdWarps / a.wpr;
    const int64_t steps = (a.rows + rpi - 1) / rpi;
    blocks = static_cast<int>(std::min<int64_t>(steps, std::min(device_sm_count(), kBwdMaxBlocks)));
    a.tensor_bytes = static_cast<uint32_t>(rpi * a.cols * sizeof(T));
    const int64_t stage = static_cast<int64_t>(a.tensor_bytes) * (FUSED && a.dz ? 3 : 2);
    a.stages = ring_stages(stage);
    const size_t acc = rpi > 1 ? static_cast<size_t>(a.cols) * 8 : 0;  // sums of the row slots
    if (vec && a.stages > 0)
      e = launch_bwd_rows<T, W, true, FUSED>(a, blocks, std::max<size_t>(a.stages * stage, acc), stream);
    else
      e = launch_bwd_rows<T, W, false, FUSED>(a, blocks, std::max<size_t>(acc, 16), stream);
  }
  if (e != cudaSuccess || !a.part) return e;
  ln_param_sum_kernel<<<dim3(static_cast<unsigned>((a.cols + 31) / 32), 2), 256, 0, stream>>>(a.part, blocks, a.cols,
                                                                                             dw, db);
  return cudaGetLastError();
}

template <typename T, typename W>
cudaError_t launch_bwd_any(const LnBwdArgs& a, bool vec, bool fused, float* dw, float* db, cudaStream_t stream) {
  return fused ? launch_bwd<T, W, true>(a, vec, dw, db, stream) : launch_bwd<T, W, false>(a, vec, dw, db, stream);
}

cudaError_t launch_ln_bwd(const LnBwdArgs& a, int32_t dtype, int32_t wdtype, bool fused, float* dw, float* db,
                          cudaStream_t stream) {
  const bool vec = vector_rows(a.dy, a.cols) && vector_rows(a.z, a.cols) && vector_rows(a.w, a.cols) &&
                   vector_rows(a.dx, a.cols) && (!fused || (vector_rows(a.dz, a.cols) && vector_rows(a.dres, a.cols)));
  if (dtype == QLORA_DTYPE_FP32) return launch_bwd_any<float, float>(a, vec, fused, dw, db, stream);
  if (dtype == QLORA_DTYPE_BF16)
    return wdtype == dtype ? launch_bwd_any<__nv_bfloat16, __nv_bfloat16>(a, vec, fused, dw, db, stream)
                           : launch_bwd_any<__nv_bfloat16, float>(a, vec, fused, dw, db, stream);
  return wdtype == dtype ? launch_bwd_any<__half, __half>(a, vec, fused, dw, db, stream)
                         : launch_bwd_any<__half, float>(a, vec, fused, dw, db, stream);
}

qlora_status check_types(int32_t dtype, int32_t wdtype) {
  if (!known_dtype(dtype) || !known_dtype(wdtype)) return QLORA_ERR_INVALID_ARG;
  return wdtype == dtype || wdtype == QLORA_DTYPE_FP32 ? QLORA_OK : QLORA_ERR_UNSUPPORTED;
}

size_t ln_workspace_bytes(int64_t cols) { return kLnStatusBytes + static_cast<size_t>(kBwdMaxBlocks) * 2 * cols * 4; }

qlora_status fwd_call(LnFwdArgs& a, int64_t rows, int64_t cols, int32_t dtype, int32_t wdtype, float eps, bool fused,
                      const char* name, void* stream) {
  qlora_status s = check_types(dtype, wdtype);
  if (s == QLORA_OK) s = check_rows(rows, cols);
  if (s != QLORA_OK) return s;
  if (!std::isfinite(eps) || eps < 0.0f) return QLORA_ERR_INVALID_ARG;
  const int es = dtype_bytes(dtype), ws = dtype_bytes(wdtype);
  if (!aligned_to(a.x, es) || !aligned_to(a.y, es) || !aligned_to(a.residual, es) || !aligned_to(a.z, es) ||
      !aligned_to(a.w, ws) || !aligned_to(a.b, ws) || !aligned_to(a.mean, 4) || !aligned_to(a.rstd, 4))
    return QLORA_ERR_ALIGNMENT;
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  a.inv_n = static_cast<float>(1.0 / static_cast<double>(cols));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope prof(st, name, 1);
  const cudaError_t e = launch_ln_fwd(a, dtype, wdtype, fused, st);
  prof.done();
  return e == cudaSuccess ? QLORA_OK : cuda_fail(e);
}

qlora_status bwd_call(LnBwdArgs& a, int64_t rows, int64_t cols, int32_t dtype, int32_t wdtype, float* dweight,
                      float* dbias, bool fused, const char* name, void* workspace, size_t ws_bytes, void* stream) {
  qlora_status s = check_types(dtype, wdtype);
  if (s == QLORA_OK) s = check_rows(rows, cols);
  if (s != QLORA_OK) return s;
  const int es = dtype_bytes(dtype);
  if (!aligned_to(a.dy, es) || !aligned_to(a.z, es) || !aligned_to(a.dz, es) || !aligned_to(a.dx, es) ||
      !aligned_to(a.dres, es) || !aligned_to(a.w, dtype_bytes(wdtype)) || !aligned_to(a.mean, 4) ||
      !aligned_to(a.rstd, 4) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4))
    return QLORA_ERR_ALIGNMENT;
  if (!workspace || ws_bytes < ln_workspace_bytes(cols)) return QLORA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return QLORA_ERR_ALIGNMENT;
  a.rows = rows;
  a.cols = cols;
  a.inv_n = static_cast<float>(1.0 / static_cast<double>(cols));
  a.status = static_cast<int*>(workspace);
  a.wait_ns = wait_limit_ns();
  if (dweight || dbias) a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kLnStatusBytes);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope prof(st, name, a.part ? 2 : 1);
  const cudaError_t e = launch_ln_bwd(a, dtype, wdtype, fused, dweight, dbias, st);
  prof.done();
  return e == cudaSuccess ? QLORA_OK : cuda_fail(e);
}

}  // namespace

}  // namespace qlora

using namespace qlora;

extern "C" {

qlora_status qlora_layernorm_fwd(const void* X, const void* weight, const void* bias, void* Y, float* mean,
                                 float* rstd, int64_t rows, int64_t cols, int32_t dtype, int32_t wdtype, float eps,
                                 void* stream) {
  if (!X || !Y) return QLORA_ERR_INVALID_ARG;
  LnFwdArgs a{};
  a.x = X;
  a.w = weight;
  a.b = bias;
  a.y = Y;
  a.mean = mean;
  a.rstd = rstd;
  return fwd_call(a, rows, cols, dtype, wdtype, eps, false, "layernorm_fwd", stream);
}

qlora_status qlora_dropout_add_layernorm_fwd(const void* X, const void* residual, const void* weight,
                                             const void* bias, void* Z, void* Y, float* mean, float* rstd,
                                             int64_t rows, int64_t cols, int32_t dtype, int32_t wdtype, float eps,
                                             double p, uint64_t seed, uint64_t offset, const uint64_t* offset_dev,
                                             void* stream) {
  if (!X || !residual || !Z || !Y || !(p >= 0.0 && p <= 1.0)) return QLORA_ERR_INVALID_ARG;
  LnFwdArgs a{};
  if (!make_drop_args(p, seed, offset, offset_dev, cols, &a.drop)) return QLORA_ERR_ALIGNMENT;
  a.x = X;
  a.residual = residual;
  a.w = weight;
  a.b = bias;
  a.z = Z;
  a.y = Y;
  a.mean = mean;
  a.rstd = rstd;
  return fwd_call(a, rows, cols, dtype, wdtype, eps, true, "dropout_add_layernorm_fwd", stream);
}

size_t qlora_layernorm_workspace_bytes(int64_t rows, int64_t cols) {
  return check_rows(rows, cols) == QLORA_OK ? ln_workspace_bytes(cols) : 0;
}

qlora_status qlora_layernorm_bwd(const void* dY, const void* X, const float* mean, const float* rstd,
                                 const void* weight, void* dX, float* dweight, float* dbias, int64_t rows,
                                 int64_t cols, int32_t dtype, int32_t wdtype, void* workspace, size_t ws_bytes,
                                 void* stream) {
  if (!dY || !X || !mean || !rstd || !dX) return QLORA_ERR_INVALID_ARG;
  LnBwdArgs a{};
  a.dy = dY;
  a.z = X;
  a.mean = mean;
  a.rstd = rstd;
  a.w = weight;
  a.dx = dX;
  return bwd_call(a, rows, cols, dtype, wdtype, dweight, dbias, false, "layernorm_bwd", workspace, ws_bytes, stream);
}

qlora_status qlora_dropout_add_layernorm_bwd(const void* dY, const void* dZ, const void* Z, const float* mean,
                                             const float* rstd, const void* weight, void* dX, void* dresidual,
                                             float* dweight, float* dbias, int64_t rows, int64_t cols, int32_t dtype,
                                             int32_t wdtype, double p, uint64_t seed, uint64_t offset,
                                             const uint64_t* offset_dev, void* workspace, size_t ws_bytes,
                                             void* stream) {
  if (!dY || !Z || !mean || !rstd || !dX || !dresidual || !(p >= 0.0 && p <= 1.0)) return QLORA_ERR_INVALID_ARG;
  LnBwdArgs a{};
  if (!make_drop_args(p, seed, offset, offset_dev, cols, &a.drop)) return QLORA_ERR_ALIGNMENT;
  a.dy = dY;
  a.dz = dZ;
  a.z = Z;
  a.mean = mean;
  a.rstd = rstd;
  a.w = weight;
  a.dx = dX;
  a.dres = dresidual;
  return bwd_call(a, rows, cols, dtype, wdtype, dweight, dbias, true, "dropout_add_layernorm_bwd", workspace,
                  ws_bytes, stream);
}

}  // extern "C"
