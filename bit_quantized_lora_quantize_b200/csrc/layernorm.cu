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
// HBM sets the floor of all of it: a row is read once into registers, the mean
// first and then the squared distances from it (no difference of large sums),
// both in float32.  The fused form takes the statistics of Z as rounded to its
// type, which is what the backward pass reads.
//
// Forward: `wpr` warps share a row, 256 columns per warp and step, so that a
// row of up to 16384 columns stays in registers; many rows per SM hide each
// other's reduction.  With few rows each gets as many warps as its columns
// allow instead (one step per warp).  Longer rows are read three times.
//
// Backward: one persistent block per SM walks over the rows.  A ring of
// stages in shared memory, filled by bulk copies, keeps whole rows of dY and Z
// in flight; each thread carries the sums of dweight and dbias for its columns
// in registers across all rows of the block.  The blocks' partial sums are
// added by a second, small kernel in a fixed order, so results are the same
// from run to run.  Rows of over 8192 columns take one block each and a second
// pass for the parameters.
//
// Measured on 4096 x 8192, as a fraction of the copy bandwidth: forward 28.5 us
// (0.72) in bf16 and 49.3 (0.83) in float32, fused 47.4 (0.86) and 96.0 (0.85);
// backward 46.8 (0.66) and 68.3 (0.90), fused 70.9 (0.72) and 109 (0.94).  In
// float32 HBM is the bound.  In bf16 latency is: the forward's loads wait for the
// block's reductions before them, with nothing of the next row in flight; in the
// backward 17 warps per SM, at 96 registers, wait for shared memory (each stage
// is read and unpacked twice), for the ring and for one another, with issue
// slots 49 %, the ALU 32 % and DRAM 46 % busy.  Ragged rows take scalar accesses:
// 777 x 5003 in fp16 8.8 us forward and 15.8 backward, against 6.6 and 13.9 of
// 777 x 5000.  Long rows: backward 166 us for 4096 x 11008 and 203 for
// 4096 x 16384 in bf16, forward 141 for 4096 x 20480 (55 for 4096 x 16384, still
// in registers).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>
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
constexpr int kFwdWarps = 16;            // warps of a forward block (32 with one step each)
constexpr int kBwdGroups = 2;            // the same in the backward
constexpr int kBwdWarps = 16;            // that compute; one more feeds the ring
constexpr int kBwdThreads = (kBwdWarps + 1) * 32;
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

// Sum over the wpr warps of a row (a power of two); `buf` holds one float per
// warp.  Every thread of the block calls it.
__device__ __forceinline__ float row_sum(float v, float* buf, int warp, int first, int wpr) {
  v = warp_sum(v);
  if (wpr == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  v = buf[first + (lane & (wpr - 1))];
#pragma unroll
  for (int o = 1; o < 32; o *= 2)
    if (o < wpr) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

template <int VEC>
__device__ __forceinline__ bool col_in(int c0, int lane, int e, int cols) {
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
  int64_t rows;
  int cols;
  float eps, inv_n;
  int wpr;
};

// The draws' constants, only where there are draws.
struct NoDrop {};
template <bool FUSED>
using FwdDrop = std::conditional_t<FUSED, DropArgs, NoDrop>;

// Values of one lane's eight columns after the residual dropout, rounded to
// T and stored to Z.
template <typename T, int VEC>
__device__ __forceinline__ Raw8<T> add_dropped(const LnFwdArgs& a, const DropArgs& drop, int64_t row, int c0, int lane,
                                               uint64_t base, const Raw8<T>& x, const Raw8<T>& r) {
  const auto keep = keep_cols<VEC>(drop, base + row * drop.groups + c0 / 8, lane);
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = keep(e) ? fmaf(raw_f32(x, e), drop.gain, raw_f32(r, e)) : raw_f32(r, e);
  const Raw8<T> z = raw_from<T>(v);
  store_cols<VEC>(static_cast<T*>(a.z) + row * a.cols, c0, a.cols, lane, z);
  return z;
}

// Sum of a lane's eight values (zeros past the end), and of their squared
// distances from the mean.
__device__ __forceinline__ float group_sum(const F2 (&x)[4]) {
  return f2_sum(add2(add2(x[0], x[1]), add2(x[2], x[3])));
}
template <int VEC>
__device__ __forceinline__ float group_spread(const F2 (&x)[4], float mean, int c0, int lane, int cols) {
  const F2 m = f2_all(-mean);
  F2 q = 0;
  if (VEC == kWhole || c0 + 256 <= cols) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const F2 d = add2(x[p], m);
      q = fma2(d, d, q);
    }
    return f2_sum(q);
  }
  float s = 0.0f;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 d = f2_get(add2(x[p], m));
    if (col_in<VEC>(c0, lane, 2 * p, cols)) s = fmaf(d.x, d.x, s);
    if (col_in<VEC>(c0, lane, 2 * p + 1, cols)) s = fmaf(d.y, d.y, s);
  }
  return s;
}

template <typename T, typename W, int VEC>
__device__ __forceinline__ void normalise(const LnFwdArgs& a, int64_t row, int c0, int lane, float mean, float rstd,
                                          const F2 (&x)[4]) {
  const Raw8<W> w = a.w ? load_cols<VEC>(static_cast<const W*>(a.w), c0, a.cols, lane) : raw_ones<W>();
  const Raw8<W> b = a.b ? load_cols<VEC>(static_cast<const W*>(a.b), c0, a.cols, lane) : raw_zero<W>();
  const F2 m = f2_all(-mean), r = f2_all(rstd);
  F2 v[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const F2 h = mul2(add2(x[p], m), r);
    v[p] = fma2(h, raw_f2(w, p), raw_f2(b, p));
  }
  store_cols<VEC>(static_cast<T*>(a.y) + row * a.cols, c0, a.cols, lane, raw_from_pairs<T>(v));
}

template <typename T, typename W, int G, int VEC, bool FUSED>
__global__ void __launch_bounds__(kFwdWarps * 32 * (G == 1 ? 2 : 1))
    ln_fwd_kernel(const LnFwdArgs a, const FwdDrop<FUSED> drop) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp & (a.wpr - 1), first = warp - part, shift = __ffs(a.wpr) - 1;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> (5 + shift)) + (warp >> shift);
  const bool valid = row < a.rows;
  const T* xr = static_cast<const T*>(a.x) + row * a.cols;
  const T* rr = static_cast<const T*>(a.residual) + row * a.cols;
  Raw8<T> x[G], r[FUSED ? G : 1];
  float s = 0.0f;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c0 = (part + g * a.wpr) * 256;
    if (valid && c0 < a.cols) {
      x[g] = load_cols<VEC>(xr, c0, a.cols, lane);
      if constexpr (FUSED) r[g] = load_cols<VEC>(rr, c0, a.cols, lane);
    }
  }
  uint64_t base = 0;
  if constexpr (FUSED) base = drop_base(drop);
  F2 v[G][4];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c0 = (part + g * a.wpr) * 256;
    if (valid && c0 < a.cols) {
      if constexpr (FUSED) x[g] = add_dropped<T, VEC>(a, drop, row, c0, lane, base, x[g], r[g]);
      raw_pairs(x[g], v[g]);
      s += group_sum(v[g]);
    }
  }
  const float mean = row_sum(s, red[0], warp, first, a.wpr) * a.inv_n;
  float q = 0.0f;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c0 = (part + g * a.wpr) * 256;
    if (valid && c0 < a.cols) q += group_spread<VEC>(v[g], mean, c0, lane, a.cols);
  }
  const float rstd = 1.0f / sqrtf(row_sum(q, red[1], warp, first, a.wpr) * a.inv_n + a.eps);
  if (!valid) return;
  if (part == 0 && lane == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c0 = (part + g * a.wpr) * 256;
    if (c0 < a.cols) normalise<T, W, VEC>(a, row, c0, lane, mean, rstd, v[g]);
  }
}

// Rows too long for the registers of a block: three passes, the later ones
// mostly from L2.
template <typename T, typename W, int VEC, bool FUSED>
__global__ void __launch_bounds__(1024) ln_fwd_long_kernel(const LnFwdArgs a, const FwdDrop<FUSED> drop) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const T* xr = static_cast<const T*>(a.x) + row * a.cols;
  uint64_t base = 0;
  if constexpr (FUSED) base = drop_base(drop);
  float s = 0.0f;
  for (int c0 = warp * 256; c0 < a.cols; c0 += 32 * 256) {
    Raw8<T> x = load_cols<VEC>(xr, c0, a.cols, lane);
    if constexpr (FUSED)
      x = add_dropped<T, VEC>(a, drop, row, c0, lane, base, x,
                                load_cols<VEC>(static_cast<const T*>(a.residual) + row * a.cols, c0, a.cols, lane));
    F2 v[4];
    raw_pairs(x, v);
    s += group_sum(v);
  }
  const float mean = row_sum(s, red[0], warp, 0, 32) * a.inv_n;
  // Each thread reads back only what it stored itself.
  const T* zr = FUSED ? static_cast<const T*>(a.z) + row * a.cols : xr;
  float q = 0.0f;
  for (int c0 = warp * 256; c0 < a.cols; c0 += 32 * 256) {
    F2 v[4];
    raw_pairs(load_cols<VEC>(zr, c0, a.cols, lane), v);
    q += group_spread<VEC>(v, mean, c0, lane, a.cols);
  }
  const float rstd = 1.0f / sqrtf(row_sum(q, red[1], warp, 0, 32) * a.inv_n + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  for (int c0 = warp * 256; c0 < a.cols; c0 += 32 * 256) {
    F2 v[4];
    raw_pairs(load_cols<VEC>(zr, c0, a.cols, lane), v);
    normalise<T, W, VEC>(a, row, c0, lane, mean, rstd, v);
  }
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
  float* dw;         // where a single block leaves the sums
  float* db;
  int64_t rows;
  int cols;
  float inv_n;
  int wpr;
  int stages;
  uint32_t tensor_bytes;  // room for one tensor's rows in a stage
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

// dz = rstd (dy w - s1 - h s2) [+ the gradient past the norm], four pairs of it
// to memory, and dropout(dz) in the fused form.
template <typename T, int VEC, bool FUSED>
__device__ __forceinline__ void store_grad(const LnBwdArgs& a, int64_t row, int64_t at, int c0, int lane, uint64_t base,
                                           const F2 (&v)[4]) {
  if constexpr (!FUSED) {
    store_cols<VEC, false>(static_cast<T*>(a.dx) + at, c0, a.cols, lane, raw_from_pairs<T>(v));
  } else {
    store_cols<VEC, false>(static_cast<T*>(a.dres) + at, c0, a.cols, lane, raw_from_pairs<T>(v));
    const auto keep = keep_cols<VEC>(a.drop, base + row * a.drop.groups + c0 / 8, lane);
    float f[8];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float2 d = f2_get(mul2(v[p], f2_all(a.drop.gain)));
      f[2 * p] = keep(2 * p) ? d.x : 0.0f;
      f[2 * p + 1] = keep(2 * p + 1) ? d.y : 0.0f;
    }
    store_cols<VEC, false>(static_cast<T*>(a.dx) + at, c0, a.cols, lane, raw_from<T>(f));
  }
}

// A lane's eight float32 values to row[c0 ..]; `row` is aligned for vectors when
// VEC and the columns a multiple of eight.
template <int VEC>
__device__ __forceinline__ void store_pairs(float* row, int c0, int cols, int lane, const F2 (&v)[4]) {
  if (c0 >= cols) return;
  if (VEC && aligned_group(row)) {
    const int c = c0 + lane * 8;
    if (VEC == kWhole || c < cols) store_group(row + c, raw_from_pairs<float>(v));
    return;
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 d = f2_get(v[p]);
    const int c = c0 + warp_col<VEC>(lane, 2 * p), e = c0 + warp_col<VEC>(lane, 2 * p + 1);
    if (c < cols) row[c] = d.x;
    if (e < cols) row[e] = d.y;
  }
}

// Ring of bulk copies over one tensor's rows.  Rows need not be aligned: a
// copy covers the 16-byte blocks around a stage's rows, except that it stays
// inside the tensor; the few elements this leaves out at the tensor's two ends
// are stored by the issuing thread.
template <typename T>
struct RowRing {
  const T* base;
  int64_t total;  // elements
  __device__ __forceinline__ uint32_t shift(int64_t at) const {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(base + at) & 15u);
  }
  // Bytes that load() will copy for elements [at, at + n).
  __device__ __forceinline__ void span(int64_t at, int64_t n, uintptr_t& lo, uintptr_t& hi) const {
    const uintptr_t b = reinterpret_cast<uintptr_t>(base), e = reinterpret_cast<uintptr_t>(base + total);
    lo = reinterpret_cast<uintptr_t>(base + at) & ~uintptr_t(15);
    hi = (reinterpret_cast<uintptr_t>(base + at + n) + 15) & ~uintptr_t(15);
    if (lo < b) lo = (b + 15) & ~uintptr_t(15);
    if (hi > e) hi = e & ~uintptr_t(15);
    if (hi < lo) hi = lo;
  }
  // Element `at` lands at dst + shift(at).
  __device__ __forceinline__ void load(uint8_t* dst, int64_t at, int64_t n, uint64_t* bar) const {
    uintptr_t lo, hi;
    span(at, n, lo, hi);
    const uintptr_t from = reinterpret_cast<uintptr_t>(base + at) & ~uintptr_t(15);
    if (hi > lo)
      bulk_load(dst + (lo - from), reinterpret_cast<const void*>(lo), static_cast<uint32_t>(hi - lo), bar);
  }
  // The elements that load() leaves out, at most seven at each end of the tensor.
  // A later copy into the same stage, which the same thread starts, overwrites
  // them: the fence orders these stores before it.
  __device__ __forceinline__ void ends(uint8_t* dst, int64_t at, int64_t n) const {
    uintptr_t lo, hi;
    span(at, n, lo, hi);
    const uintptr_t b = reinterpret_cast<uintptr_t>(base + at), e = reinterpret_cast<uintptr_t>(base + at + n);
    T* to = reinterpret_cast<T*>(dst + shift(at));
    if (lo > b) {
      const int64_t head = min(n, static_cast<int64_t>((lo - b) / sizeof(T)));
      for (int64_t i = 0; i < head; ++i) to[i] = base[at + i];
    }
    if (hi < e) {
      const int64_t tail = min(n, static_cast<int64_t>((e - hi) / sizeof(T)));
      for (int64_t i = n - tail; i < n; ++i) to[i] = base[at + i];
    }
    if (lo > b || hi < e) fence_proxy_async_smem();
  }
};

// The rows' sums over the wpr warps that share them, from the block's per-warp
// values: pairs (sum g, sum g h) of R rows.
template <int R>
__device__ __forceinline__ void row_sums(const float (*red)[2 * R], int first, int wpr, F2 (&s)[R]) {
  if constexpr (R == 2) {
    s[0] = s[1] = 0;
#pragma unroll 4
    for (int k = 0; k < wpr; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(red[first + k]);
      s[0] = add2(s[0], f2(v.x, v.y));
      s[1] = add2(s[1], f2(v.z, v.w));
    }
  } else {
    s[0] = *reinterpret_cast<const F2*>(red[first]);
    if (wpr == 1) return;
    s[0] = 0;
#pragma unroll 8
    for (int k = 0; k < wpr; k += 2) {
      const float4 v = *reinterpret_cast<const float4*>(red[first + k]);
      s[0] = add2(s[0], add2(f2(v.x, v.y), f2(v.z, v.w)));
    }
  }
}

// A warp's sums of R rows (s[2 q]: sum g of row q, s[2 q + 1]: sum g h) over its
// lanes, to `out`.  Halves, then quarters of the warp go on with a share of the
// values each.
template <int R>
__device__ __forceinline__ void publish_sums(float (&s)[2 * R], float* out) {
  const int lane = threadIdx.x & 31;
  int own = 0;
#pragma unroll
  for (int n = 2 * R, o = 16; n > 1; n /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int k = 0; k < n / 2; ++k) {
      const float give = upper ? s[k] : s[k + n / 2];
      s[k] = (upper ? s[k + n / 2] : s[k]) + __shfl_xor_sync(kAll, give, o);
    }
    own = own * 2 + (upper ? 1 : 0);
  }
#pragma unroll
  for (int o = 16 / (2 * R); o > 0; o >>= 1) s[0] += __shfl_xor_sync(kAll, s[0], o);
  if ((lane & (32 / (2 * R) - 1)) == 0) out[own] = s[0];
}

// Each step of a block: the gradients of step i, whose sums the barrier at the
// end of the previous step made visible, then the sums over step i + 1.  So one
// barrier per step, with independent work on both sides of it.  A warp of
// its own feeds the ring: its address arithmetic would otherwise hold up the
// barrier of every step (2 us a step before, whatever the columns).
template <typename T, typename W, int VEC, bool FUSED, int R>
__global__ void __launch_bounds__(kBwdThreads, 1) ln_bwd_kernel(const LnBwdArgs a) {
  constexpr int G = kBwdGroups;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float red[2][kBwdWarps][2 * R];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ float2 row_stats[kMaxStages][kBwdWarps * R];  // mean and rstd of a stage's rows
  __shared__ volatile int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int log = __ffs(a.wpr) - 1, part = warp & (a.wpr - 1), first = warp - part, slot = (warp >> log) * R;
  const int rpi = (kBwdWarps >> log) * R;  // rows per step of the block
  const int64_t steps = (a.rows + rpi - 1) / rpi;
  const int mine = static_cast<int>((steps - blockIdx.x + gridDim.x - 1) / gridDim.x);
  const bool has_dz = FUSED && a.dz;
  const int tensors = has_dz ? 3 : 2;
  const uint32_t stage_bytes = a.tensor_bytes * tensors;
  const RowRing<T> ring_of[3] = {{static_cast<const T*>(a.dy), a.rows * a.cols},
                                 {static_cast<const T*>(a.z), a.rows * a.cols},
                                 {static_cast<const T*>(a.dz), a.rows * a.cols}};

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kBwdWarps);
    }
    abort_flag = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  if (warp == kBwdWarps) {
    const WaitCtx ctx{&abort_flag, a.status, 42, a.wait_ns};
    // Lane l looks after the statistics of a step's row l, one step ahead.
    float2 ahead;
    const auto look = [&](int i) {
      const int64_t row = (static_cast<int64_t>(i) * gridDim.x + blockIdx.x) * rpi + lane;
      const bool in = lane < rpi && row < a.rows;
      ahead.x = in ? __ldg(a.mean + row) : 0.0f;
      ahead.y = in ? __ldg(a.rstd + row) : 0.0f;
    };
    look(0);
    int issued = 0;
    for (; issued < mine; ++issued) {
      const int s = issued % a.stages;
      if (!__all_sync(kAll, mbar_wait(&empty[s], static_cast<uint32_t>((issued / a.stages) & 1) ^ 1, ctx))) break;
      const int64_t row = (static_cast<int64_t>(issued) * gridDim.x + blockIdx.x) * rpi, at = row * a.cols;
      const int64_t n = min(static_cast<int64_t>(rpi), a.rows - row) * a.cols;
      uint8_t* dst = ring + s * stage_bytes;
      if (lane < rpi) row_stats[s][lane] = ahead;
      __syncwarp();
      if (lane == 0) {
        // The arrival publishes the statistics and the ends to whoever waits
        // for the stage.
        uint32_t bytes = 0;
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          if (t < tensors) {
            if (!VEC) ring_of[t].ends(dst + t * a.tensor_bytes, at, n);
            uintptr_t lo, hi;
            ring_of[t].span(at, n, lo, hi);
            bytes += static_cast<uint32_t>(hi - lo);
          }
        }
        mbar_arrive_expect_tx(&full[s], bytes);
#pragma unroll
        for (int t = 0; t < 3; ++t)
          if (t < tensors) ring_of[t].load(dst + t * a.tensor_bytes, at, n, &full[s]);
      }
      look(issued + 1);
    }
    if (abort_flag && lane == 0)  // copies still in flight must land before the block leaves
      for (int i = max(0, issued - a.stages); i < issued; ++i)
        mbar_drain(&full[i % a.stages], static_cast<uint32_t>((i / a.stages) & 1));
    return;
  }
  const WaitCtx ctx{&abort_flag, a.status, 41, a.wait_ns};
  const uint64_t base = FUSED ? drop_base(a.drop) : 0;

  F2 w[G][4], aw[G][4], ab[G][4];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c0 = (part + g * a.wpr) * 256;
    const Raw8<W> raw =
        a.w && c0 < a.cols ? load_cols<VEC>(static_cast<const W*>(a.w), c0, a.cols, lane) : raw_ones<W>();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      w[g][p] = raw_f2(raw, p);
      aw[g][p] = ab[g][p] = 0;
    }
  }
  // The warp's rows (R neighbours) of this step and the next: the first one's
  // number and element, their statistics and place in the ring.
  const int64_t stride = static_cast<int64_t>(gridDim.x) * rpi, stride_at = stride * a.cols;
  struct Rows {
    int64_t row, at;
    uint32_t stage;
    float mean[R], rstd[R];
  };
  // Row q's columns of tensor t in the ring (a stage starts at its first row).
  const uint32_t row_bytes = static_cast<uint32_t>(a.cols * sizeof(T)), slot_bytes = slot * row_bytes;
  const auto row_in = [&](const Rows& r, int q, int t) {
    const uint32_t shift = VEC ? 0u : ring_of[t].shift(r.at - static_cast<int64_t>(slot) * a.cols);
    return r.stage + t * a.tensor_bytes + shift + slot_bytes + q * row_bytes;
  };
  // 32-bit offsets from the array's name, so that the accesses stay shared-memory ones.
  const auto load_in = [&](uint32_t row, int c0) {
    return load_cols<VEC, false>(reinterpret_cast<const T*>(ring + row), c0, a.cols, lane);
  };
  // A step of 256 columns: what one row adds to the sums ...
  const auto add_up = [&](const Rows& r, int q, int g, int c0, F2& s1, F2& s2) {
    const F2 nm = f2_all(-r.mean[q]), rs = f2_all(r.rstd[q]);
    // columns past the end hold dY = 0 and add nothing
    const Raw8<T> dy = load_in(row_in(r, q, 0), c0), z = load_in(row_in(r, q, 1), c0);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const F2 d = raw_f2(dy, p), h = mul2(add2(raw_f2(z, p), nm), rs), gr = mul2(d, w[g][p]);
      aw[g][p] = fma2(d, h, aw[g][p]);
      ab[g][p] = add2(ab[g][p], d);
      s1 = add2(s1, gr);
      s2 = fma2(gr, h, s2);
    }
  };
  // ... and a row's gradients, from its two sums:
  // rstd (dy w - s1 - h s2) = rstd dy w - rstd s1 - (z - mean) rstd^2 s2
  const auto gradients = [&](const Rows& r, int q, int g, int c0, F2 k1, F2 k2) {
    const F2 nm = f2_all(-r.mean[q]), rs = f2_all(r.rstd[q]);
    const Raw8<T> dy = load_in(row_in(r, q, 0), c0), z = load_in(row_in(r, q, 1), c0);
    F2 v[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = fma2(mul2(raw_f2(dy, p), w[g][p]), rs, fma2(add2(raw_f2(z, p), nm), k2, k1));
    if (has_dz) {
      const Raw8<T> dz = load_in(row_in(r, q, 2), c0);
#pragma unroll
      for (int p = 0; p < 4; ++p) v[p] = add2(v[p], raw_f2(dz, p));
    }
    store_grad<T, VEC, FUSED>(a, r.row + q, r.at + q * static_cast<int64_t>(a.cols), c0, lane, base, v);
  };
  // A step's rows into the sums; the warp's share of each row's two to `out`.
  const auto first_pass = [&](Rows& r, int s, float* out) {
    F2 t1[R], t2[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const float2 st = row_stats[s][slot + q];
      r.mean[q] = st.x;
      r.rstd[q] = st.y;
      t1[q] = t2[q] = 0;
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c0 = (part + g * a.wpr) * 256;
      if (c0 < a.cols) {
#pragma unroll
        for (int q = 0; q < R; ++q)
          if (r.row + q < a.rows) add_up(r, q, g, c0, t1[q], t2[q]);
      }
    }
    float sum[2 * R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      sum[2 * q] = f2_sum(t1[q]);
      sum[2 * q + 1] = f2_sum(t2[q]);
    }
    publish_sums<R>(sum, out);
  };

  Rows cur, next;
  next.row = static_cast<int64_t>(blockIdx.x) * rpi + slot;
  next.at = next.row * a.cols;
  next.stage = 0;
  int s = 0;             // stage of `next`
  uint32_t parity = 0;
  const auto advance = [&] {
    next.row += stride;
    next.at += stride_at;
    if (++s == a.stages) {
      s = 0;
      parity ^= 1;
    }
    next.stage = s * stage_bytes;
  };
  // The computing warps' own barrier.
  const auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kBwdWarps * 32) : "memory"); };
  mbar_wait(&full[0], 0, ctx);  // every block has a step
  first_pass(next, 0, red[0][warp]);
  cur = next;
  advance();
  sync();
  int s_cur = 0;
  for (int i = 0; i < mine; ++i) {
    F2 k1[R], k2[R];
    {
      F2 sum[R];
      row_sums<R>(red[i & 1], first, a.wpr, sum);
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const float2 v = f2_get(sum[q]);
        k1[q] = f2_all(-cur.rstd[q] * (v.x * a.inv_n));
        k2[q] = f2_all(-cur.rstd[q] * (cur.rstd[q] * (v.y * a.inv_n)));
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c0 = (part + g * a.wpr) * 256;
      if (c0 < a.cols) {
#pragma unroll
        for (int q = 0; q < R; ++q)
          if (cur.row + q < a.rows) gradients(cur, q, g, c0, k1[q], k2[q]);
      }
    }
    // The stage goes back as soon as the warps have read it, before they turn
    // to the next: the ring then holds one stage in use and all others in
    // flight (4096 x 8192 fused: float32, two stages, 146 -> 110 us; bf16 without
    // the dropout, three stages, 47.4 -> 46.5).
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s_cur]);
    if (++s_cur == a.stages) s_cur = 0;
    if (i + 1 < mine) {
      mbar_wait(&full[s], parity, ctx);
      first_pass(next, s, red[(i + 1) & 1][warp]);
    }
    cur = next;
    advance();
    sync();  // step i + 1's sums are visible
  }
  griddep_launch_dependents();

  if (!a.part && !a.dw && !a.db) return;
  float* pw = a.part ? a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.cols : a.dw;
  float* pb = a.part ? pw + a.cols : a.db;
  const int slots = rpi / R, mine_slot = slot / R;
  if (slots == 1) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c0 = (part + g * a.wpr) * 256;
      if (pw) store_pairs<VEC>(pw, c0, a.cols, lane, aw[g]);
      if (pb) store_pairs<VEC>(pb, c0, a.cols, lane, ab[g]);
    }
    return;
  }
  // The row slots' sums, added in slot order: [slot][dweight, dbias][column].
  float* acc = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c0 = (part + g * a.wpr) * 256;
    store_pairs<VEC>(acc + (mine_slot * 2) * a.cols, c0, a.cols, lane, aw[g]);
    store_pairs<VEC>(acc + (mine_slot * 2 + 1) * a.cols, c0, a.cols, lane, ab[g]);
  }
  sync();
  for (int c = threadIdx.x; c < 2 * a.cols; c += kBwdWarps * 32) {
    float sum = 0.0f;
    for (int k = 0; k < slots; ++k) sum += acc[k * 2 * a.cols + c];
    if (c < a.cols) {
      if (pw) pw[c] = sum;
    } else if (pb) {
      pb[c - a.cols] = sum;
    }
  }
}

// dweight / dbias = sum of the blocks' partial sums, in block order within
// each of 16 interleaved chains.  V neighbouring columns per lane; all of a
// warp's loads are in flight together.
constexpr int kSumWarps = 16;
template <int V>
__global__ void __launch_bounds__(kSumWarps * 32) ln_param_sum_kernel(const float* __restrict__ part, int blocks,
                                                                      int cols, float* dw, float* db) {
  constexpr int kLoads = (kBwdMaxBlocks + kSumWarps - 1) / kSumWarps;
  __shared__ float red[kSumWarps][32 * V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + lane) * V;
  float* out = blockIdx.y ? db : dw;
  griddep_wait();
  if (!out) return;
  float x[kLoads][V];
  const float* p = part + (static_cast<int64_t>(warp) * 2 + blockIdx.y) * cols + c;
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[k][v] = 0.0f;
    if (c < cols && warp + k * kSumWarps < blocks) {
      const float* q = p + static_cast<int64_t>(k) * kSumWarps * 2 * cols;
      if constexpr (V == 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(q));
        x[k][0] = f.x; x[k][1] = f.y; x[k][2] = f.z; x[k][3] = f.w;
      } else {
        x[k][0] = __ldcg(q);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) s += x[k][v];
    red[warp][lane * V + v] = s;
  }
  __syncthreads();
  const int col = blockIdx.x * 32 * V + threadIdx.x;
  if (threadIdx.x < 32 * V && col < cols) {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kSumWarps; ++k) sum += red[k][threadIdx.x];
    out[col] = sum;
  }
}

// Rows too long for the ring kernel's registers: one block per row for the
// input gradient, reading the row twice.
template <typename T, typename W, int VEC, bool FUSED>
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
  for (int c0 = warp * 256; c0 < a.cols; c0 += 32 * 256) {
    const Raw8<T> dy = load_cols<VEC>(dyr, c0, a.cols, lane);
    const Raw8<T> z = load_cols<VEC>(zr, c0, a.cols, lane);
    Raw8<W> w;
    if (wr) w = load_cols<VEC>(wr, c0, a.cols, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float h = (raw_f32(z, e) - mean) * rstd;  // past the end dY = 0
      const float gr = wr ? raw_f32(dy, e) * raw_f32(w, e) : raw_f32(dy, e);
      s1 += gr;
      s2 = fmaf(gr, h, s2);
    }
  }
  s1 = row_sum(s1, red[0], warp, 0, 32) * a.inv_n;
  s2 = row_sum(s2, red[1], warp, 0, 32) * a.inv_n;
  for (int c0 = warp * 256; c0 < a.cols; c0 += 32 * 256) {
    const Raw8<T> dy = load_cols<VEC>(dyr, c0, a.cols, lane);
    const Raw8<T> z = load_cols<VEC>(zr, c0, a.cols, lane);
    Raw8<W> w;
    if (wr) w = load_cols<VEC>(wr, c0, a.cols, lane);
    Raw8<T> dz;
    if (FUSED && a.dz) dz = load_cols<VEC>(static_cast<const T*>(a.dz) + at, c0, a.cols, lane);
    F2 v[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const F2 h = mul2(add2(raw_f2(z, p), f2_all(-mean)), f2_all(rstd));
      const F2 g = fma2(raw_f2(dy, p), wr ? raw_f2(w, p) : f2_all(1.0f), f2_all(-s1));
      v[p] = mul2(fma2(h, f2_all(-s2), g), f2_all(rstd));
      if (FUSED && a.dz) v[p] = add2(v[p], raw_f2(dz, p));
    }
    store_grad<T, VEC, FUSED>(a, row, at, c0, lane, base, v);
  }
}

// The parameter gradients of such rows: block (x, y) sums 256 columns over
// the rows y, y + gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(256) ln_param_long_kernel(const LnBwdArgs a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float sw = 0.0f, sb = 0.0f;
#pragma unroll 8
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

template <typename T, typename W, int VEC, bool FUSED>
cudaError_t launch_fwd(LnFwdArgs a, const FwdDrop<FUSED>& drop, cudaStream_t stream) {
  if (a.cols > kFwdWarps * 256 * kFwdMaxGroups) {
    constexpr int kLong = VEC == kRagged ? kRagged : kAligned;
    ln_fwd_long_kernel<T, W, kLong, FUSED><<<static_cast<unsigned>(a.rows), 1024, 0, stream>>>(a, drop);
    return cudaGetLastError();
  }
  // Few rows: one step per warp where 32 warps allow it, for latency (bf16,
  // 1 x 8192: 3.0 us, 3.4 with four; 290 x 4096: 2.9 against 3.5; 290 x 8192, the
  // rule's edge: 4.1 against 4.0).  Otherwise four steps, so that several rows
  // share an SM.
  int groups = kFwdMaxGroups;
  if (a.rows <= 2 * device_sm_count() && a.cols <= 2 * kFwdWarps * 256) groups = 1;
  a.wpr = warps_for(a.cols, groups);
  while (groups > 1 && static_cast<int64_t>(a.wpr) * 256 * (groups / 2) >= a.cols) groups /= 2;
  const int warps = std::max(a.wpr, 4);
  const int64_t rpb = warps / a.wpr;
  const unsigned grid = static_cast<unsigned>((a.rows + rpb - 1) / rpb);
  if (groups == 1) ln_fwd_kernel<T, W, 1, VEC, FUSED><<<grid, warps * 32, 0, stream>>>(a, drop);
  else if (groups == 2) ln_fwd_kernel<T, W, 2, VEC, FUSED><<<grid, warps * 32, 0, stream>>>(a, drop);
  else ln_fwd_kernel<T, W, 4, VEC, FUSED><<<grid, warps * 32, 0, stream>>>(a, drop);
  return cudaGetLastError();
}

template <typename T, typename W, bool FUSED>
cudaError_t launch_fwd_layout(const LnFwdArgs& a, const FwdDrop<FUSED>& drop, bool vec, cudaStream_t stream) {
  if (!vec) return launch_fwd<T, W, kRagged, FUSED>(a, drop, stream);
  return aligned_layout(a.cols) == kWhole ? launch_fwd<T, W, kWhole, FUSED>(a, drop, stream)
                                          : launch_fwd<T, W, kAligned, FUSED>(a, drop, stream);
}

template <typename T, typename W>
cudaError_t launch_fwd_any(const LnFwdArgs& a, const DropArgs* drop, bool vec, cudaStream_t stream) {
  return drop ? launch_fwd_layout<T, W, true>(a, *drop, vec, stream)
              : launch_fwd_layout<T, W, false>(a, NoDrop{}, vec, stream);
}

cudaError_t launch_ln_fwd(const LnFwdArgs& a, const DropArgs* drop, int32_t dtype, int32_t wdtype,
                          cudaStream_t stream) {
  const bool vec = vector_rows(a.x, a.cols) && vector_rows(a.y, a.cols) && vector_rows(a.w, a.cols) &&
                   vector_rows(a.b, a.cols) &&
                   (!drop || (vector_rows(a.residual, a.cols) && vector_rows(a.z, a.cols)));
  if (dtype == QLORA_DTYPE_FP32) return launch_fwd_any<float, float>(a, drop, vec, stream);
  if (dtype == QLORA_DTYPE_BF16)
    return wdtype == dtype ? launch_fwd_any<__nv_bfloat16, __nv_bfloat16>(a, drop, vec, stream)
                           : launch_fwd_any<__nv_bfloat16, float>(a, drop, vec, stream);
  return wdtype == dtype ? launch_fwd_any<__half, __half>(a, drop, vec, stream)
                         : launch_fwd_any<__half, float>(a, drop, vec, stream);
}

template <typename T, typename W, int VEC, bool FUSED, int R>
cudaError_t launch_bwd_rows(const LnBwdArgs& a, int grid, size_t smem, cudaStream_t stream) {
  auto kern = ln_bwd_kernel<T, W, VEC, FUSED, R>;
  const cudaError_t e = allow_shared_memory(kern, kRingBytes);
  if (e != cudaSuccess) return e;
  kern<<<grid, kBwdThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, typename W, bool FUSED>
cudaError_t launch_bwd(LnBwdArgs a, bool vec, float* dw, float* db, cudaStream_t stream) {
  int blocks;
  cudaError_t e;
  a.wpr = warps_for(std::min(a.cols, kBwdCols), kBwdGroups);
  const int slots = kBwdWarps / a.wpr;
  // Rows a warp takes per step: two, where their stages still leave three in the
  // ring and there are steps enough.  That pays for narrow and ragged rows (bf16,
  // 32768 x 64: 15.4 us, 18.2 with one; 20000 x 250: 16.1 against 17.3;
  // 4096 x 4095: 36.1 against 38.8) and costs a little for some wide aligned ones
  // (4096 x 2048: 18.2 against 17.3; 4096 x 8192: 46.8 against 45.7).
  const auto plan = [&](int r) {
    // Room for a stage's rows at any alignment.
    const int64_t row_bytes = static_cast<int64_t>(std::min(a.cols, kBwdCols)) * sizeof(T);
    a.tensor_bytes = static_cast<uint32_t>((slots * r * row_bytes + 15 + 127) / 128 * 128);
    a.stages = static_cast<int>(
        std::min<int64_t>(kMaxStages, kRingBytes / (static_cast<int64_t>(a.tensor_bytes) * (FUSED && a.dz ? 3 : 2))));
  };
  plan(2);
  int rows_per_warp = 2;
  if (a.stages < 3 || a.rows < static_cast<int64_t>(device_sm_count()) * slots * 4) {
    rows_per_warp = 1;
    plan(1);
  }
  const int rpi = slots * rows_per_warp;
  const int64_t stage = static_cast<int64_t>(a.tensor_bytes) * (FUSED && a.dz ? 3 : 2);
  // The step loop needs two stages: one tensor's rows of a step are at most
  // kBwdCols values, whatever the columns.
  static_assert(2 * 3 * ((kBwdCols * 4 + 15 + 127) / 128 * 128) <= kRingBytes, "two stages fit");
  if (a.cols > kBwdCols) {
    if (vec) ln_bwd_long_kernel<T, W, kAligned, FUSED><<<static_cast<unsigned>(a.rows), 1024, 0, stream>>>(a);
    else ln_bwd_long_kernel<T, W, kRagged, FUSED><<<static_cast<unsigned>(a.rows), 1024, 0, stream>>>(a);
    e = cudaGetLastError();
    blocks = static_cast<int>(std::min<int64_t>(a.rows, 64));
    if (e == cudaSuccess && a.part) {
      const dim3 grid(static_cast<unsigned>((a.cols + 255) / 256), static_cast<unsigned>(blocks));
      ln_param_long_kernel<T><<<grid, 256, 0, stream>>>(a);
      e = cudaGetLastError();
    }
  } else {
    const int64_t steps = (a.rows + rpi - 1) / rpi;
    blocks = static_cast<int>(std::min<int64_t>(steps, std::min(device_sm_count(), kBwdMaxBlocks)));
    if (blocks == 1) {  // its sums are the result
      a.part = nullptr;
      a.dw = dw;
      a.db = db;
    }
    const size_t acc = static_cast<size_t>(slots) * a.cols * 8;  // sums of the row slots
    const size_t smem = std::max<size_t>(a.stages * stage, acc);
    const int layout = vec ? aligned_layout(a.cols) : kRagged;
    if (rows_per_warp == 2) {
      if (layout == kRagged) e = launch_bwd_rows<T, W, kRagged, FUSED, 2>(a, blocks, smem, stream);
      else if (layout == kWhole) e = launch_bwd_rows<T, W, kWhole, FUSED, 2>(a, blocks, smem, stream);
      else e = launch_bwd_rows<T, W, kAligned, FUSED, 2>(a, blocks, smem, stream);
    } else {
      if (layout == kRagged) e = launch_bwd_rows<T, W, kRagged, FUSED, 1>(a, blocks, smem, stream);
      else if (layout == kWhole) e = launch_bwd_rows<T, W, kWhole, FUSED, 1>(a, blocks, smem, stream);
      else e = launch_bwd_rows<T, W, kAligned, FUSED, 1>(a, blocks, smem, stream);
    }
  }
  if (e != cudaSuccess || !a.part) return e;
  const int v = a.cols % 4 == 0 ? 4 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.cols + 32 * v - 1) / (32 * v)), 2, 1);
  cfg.blockDim = dim3(kSumWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const float* part = a.part;
  return v == 4 ? cudaLaunchKernelEx(&cfg, ln_param_sum_kernel<4>, part, blocks, a.cols, dw, db)
                : cudaLaunchKernelEx(&cfg, ln_param_sum_kernel<1>, part, blocks, a.cols, dw, db);
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

qlora_status fwd_call(LnFwdArgs& a, const DropArgs* drop, int64_t rows, int64_t cols, int32_t dtype, int32_t wdtype,
                      float eps, const char* name, void* stream) {
  qlora_status s = check_types(dtype, wdtype);
  if (s == QLORA_OK) s = check_rows(rows, cols);
  if (s != QLORA_OK) return s;
  if (!std::isfinite(eps) || eps < 0.0f) return QLORA_ERR_INVALID_ARG;
  const int es = dtype_bytes(dtype), ws = dtype_bytes(wdtype);
  if (!aligned_to(a.x, es) || !aligned_to(a.y, es) || !aligned_to(a.residual, es) || !aligned_to(a.z, es) ||
      !aligned_to(a.w, ws) || !aligned_to(a.b, ws) || !aligned_to(a.mean, 4) || !aligned_to(a.rstd, 4))
    return QLORA_ERR_ALIGNMENT;
  const int64_t n = rows * cols * es;
  if (!disjoint({{a.y, n}, {a.z, n}, {a.mean, rows * 4}, {a.rstd, rows * 4}},
                {{a.x, n}, {a.residual, n}, {a.w, cols * ws}, {a.b, cols * ws}}))
    return QLORA_ERR_INVALID_ARG;
  a.rows = rows;
  a.cols = static_cast<int>(cols);
  a.eps = eps;
  a.inv_n = static_cast<float>(1.0 / static_cast<double>(cols));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope prof(st, name, 1);
  const cudaError_t e = launch_ln_fwd(a, drop, dtype, wdtype, st);
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
  const int64_t n = rows * cols * es;
  if (!disjoint({{a.dx, n}, {a.dres, n}, {dweight, cols * 4}, {dbias, cols * 4}},
                {{a.dy, n}, {a.dz, n}, {a.z, n}, {a.mean, rows * 4}, {a.rstd, rows * 4},
                 {a.w, cols * dtype_bytes(wdtype)}}))
    return QLORA_ERR_INVALID_ARG;
  a.rows = rows;
  a.cols = static_cast<int>(cols);
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
  return fwd_call(a, nullptr, rows, cols, dtype, wdtype, eps, "layernorm_fwd", stream);
}

qlora_status qlora_dropout_add_layernorm_fwd(const void* X, const void* residual, const void* weight,
                                             const void* bias, void* Z, void* Y, float* mean, float* rstd,
                                             int64_t rows, int64_t cols, int32_t dtype, int32_t wdtype, float eps,
                                             double p, uint64_t seed, uint64_t offset, const uint64_t* offset_dev,
                                             void* stream) {
  if (!X || !residual || !Z || !Y || !(p >= 0.0 && p <= 1.0)) return QLORA_ERR_INVALID_ARG;
  LnFwdArgs a{};
  DropArgs drop;
  if (!make_drop_args(p, seed, offset, offset_dev, cols, &drop)) return QLORA_ERR_ALIGNMENT;
  a.x = X;
  a.residual = residual;
  a.w = weight;
  a.b = bias;
  a.z = Z;
  a.y = Y;
  a.mean = mean;
  a.rstd = rstd;
  return fwd_call(a, &drop, rows, cols, dtype, wdtype, eps, "dropout_add_layernorm_fwd", stream);
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
