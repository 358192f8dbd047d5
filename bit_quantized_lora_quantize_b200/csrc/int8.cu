// The linear layer on an 8-bit integer weight, for serving: inputs quantized
// per token, the weight per output channel, the product in whole numbers.
//
//   s_row = fp32(max|x| / 127),  code = x / s_row to the nearest whole number
//   (ties to even, of the real quotient),  Y = sx[m] sw[n] sum_k xq[m,k] wq[n,k]
//
// Sums are exact in 32-bit integers (codes in -127 .. 127, depth up to 133144),
// so no split of the depth and no order of work changes a result; float32
// enters in the epilogue.
//
// Three kernels:
// - quantization: one pass, rows in registers (4096 x 8192 in bf16 20.3 us, 0.76
//   of the copy bandwidth, with issue slots 71 % busy; ragged, by scalar
//   accesses, 4096 x 8191 30.4 us);
// - up to 16 tokens, bound by reading the weight: `token_kernel` streams it
//   straight into the register fragments of mma.sync (one token, 8192 x 8192:
//   16.2 us with the quantization, 10.3 are the weight at the copy bandwidth; four
//   tokens, 22016 x 8192: 35.3 us, 0.78 of it).  Against the other kernel: 12
//   tokens, 4096 x 4096 8.4 us and 16.5; 16 tokens, 8192 x 8192 23.2 and 23.0,
//   22016 x 8192 56.7 and 50.9;
// - more tokens: `pair_kernel`, CTA pairs (cta_group::2) with 256 x 256 tiles
//   fed by a TMA ring; persistent, with two accumulators in TMEM so that a
//   tile's epilogue runs under the next tile's products (4096 x 8192 x 8192:
//   177 us, 3.1 P operations/s; tensor pipe 83 % busy; 196 us in a row of calls
//   under the power cap), or, where the tiles fill less than half of the SMs,
//   several pairs to a tile, each a part of the depth (300 x 11003 x 4099:
//   30.3 us).
//   Narrower tiles do not help: a tcgen05.mma over 128 rows per SM costs about
//   the same for 16 columns as for 256 (8192 x 8192 with one token on that
//   path: 24.8 us).
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "abi_internal.h"
#include "kernels.h"
#include "ptx.cuh"
#include "rows_host.h"
#include "tensor_map.h"

namespace qlora {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int64_t kMaxDepth = 2147483647 / (127 * 127);  // int32 sums of codes in -127 .. 127 stay exact
constexpr int kDepth = 128;                              // bytes of K per stage: one swizzle row

// ================================================================ quantization
constexpr int kQuantGroups = 4;  // steps of 256 columns a warp holds

struct QuantArgs {
  const void* x;
  int8_t* codes;
  float* scale;
  int64_t rows, ld;
  int cols, wpr;
};

// Largest magnitude of a lane's eight values, as the bits of the float32:
// NaN orders above infinity, so both survive.  16-bit types compare in pairs.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <typename T>
__device__ __forceinline__ uint32_t abs_max(const Raw8<T>& x) {
  uint32_t m = 0;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, x.w[e] & 0x7FFFFFFFu);
    return m;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) m = max_u16x2(m, x.w[e] & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    Raw8<T> top;
    top.w[0] = m;
    return __float_as_uint(raw_f32(top, 0));
  }
}

// Codes of a row with this largest magnitude.  x times the reciprocal of the
// scale is off by far less than a half; adding 1.5 * 2^23 rounds it to a whole
// number q, ties to even, whose low byte is the code.  The remainder x - q s is
// exact in float32 (a multiple of the smaller of the two last places, no
// larger than s / 2 but for the error of q), so one comparison with s / 2 tells
// the few codes that may need mending.
struct RowScale {
  float scale, up, s, inv, half;
  bool plain;  // neither zero, tiny nor non-finite
  __device__ explicit RowScale(uint32_t bits) {
    scale = __fdiv_rn(__uint_as_float(bits), 127.0f);
    plain = bits < 0x7F800000u && scale >= 0x1p-100f;
    // A tiny scale is lifted by an exact power of two, so that its
    // reciprocal stays finite.
    up = plain ? 1.0f : 0x1p64f;
    s = scale * up;
    inv = __fdiv_rn(1.0f, s);
    half = 0.5f * s;
    if (!(bits < 0x7F800000u) || scale == 0.0f) s = 0.0f;  // all codes 0
  }
  __device__ __noinline__ uint32_t exact_code(float x) const {
    if (s == 0.0f) return 0;
    x *= up;
    float q = rintf(x * inv);
    const float r = fmaf(-q, s, x);
    const bool odd = static_cast<int>(q) & 1;
    if (r > half || (r == half && odd)) q += 1.0f;
    else if (r < -half || (r == -half && odd)) q -= 1.0f;
    return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(q, -127.0f), 127.0f))) & 0xFFu;
  }
  // The codes of eight values, in the low bytes of `c`.  Near ties are not
  // rare: 127 x / max|x| of two short mantissas often is a half.
  template <typename T>
  __device__ __forceinline__ void codes(const Raw8<T>& x, uint32_t (&c)[8]) const {
    if (!plain) {
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = exact_code(raw_f32(x, e));
      return;
    }
    float r[8], worst = 0.0f;
    const F2 magic = f2_all(12582912.0f), inv2 = f2_all(inv), neg = f2_all(-s);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const F2 v = raw_f2(x, p), b = fma2(v, inv2, magic);
      const float2 bits = f2_get(b), rest = f2_get(fma2(add2(b, f2_all(-12582912.0f)), neg, v));
      c[2 * p] = __float_as_uint(bits.x);
      c[2 * p + 1] = __float_as_uint(bits.y);
      r[2 * p] = rest.x;
      r[2 * p + 1] = rest.y;
      worst = fmaxf(worst, fmaxf(fabsf(rest.x), fabsf(rest.y)));
    }
    if (worst < half) return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (fabsf(r[e]) > half || (fabsf(r[e]) == half && (c[e] & 1u))) c[e] += r[e] > 0.0f ? 1u : ~0u;
  }
};

template <int VEC, typename T>
__device__ __forceinline__ void store_codes(const QuantArgs& a, int64_t row, int c0, int lane, const RowScale& rs,
                                            const Raw8<T>& x) {
  const int padded = (a.cols + 15) / 16 * 16;  // columns past the end hold 0
  int8_t* out = a.codes + row * a.ld;
  uint32_t k[8];
  rs.codes(x, k);
  if constexpr (VEC) {
    const int c = c0 + lane * 8;
    if (VEC == kWhole || c < padded)
      *reinterpret_cast<uint2*>(out + c) =
          make_uint2(prmt(prmt(k[0], k[1], 0x0040), prmt(k[2], k[3], 0x0040), 0x5410),
                     prmt(prmt(k[4], k[5], 0x0040), prmt(k[6], k[7], 0x0040), 0x5410));
  } else {
    int8_t* p = out + (c0 + lane);
    if (c0 + 256 <= padded) {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[32 * e] = static_cast<int8_t>(k[e]);
    } else {
      const int n = padded - c0 - lane;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (32 * e < n) p[32 * e] = static_cast<int8_t>(k[e]);
    }
  }
}

__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* buf, int warp, int first, int wpr) {
  v = __reduce_max_sync(kAll, v);
  if (wpr == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  return __reduce_max_sync(kAll, buf[first + (lane & (wpr - 1))]);
}

// Three blocks of 16 warps per SM where rows take four steps: 300 rows of 11003
// need no second wave (10.1 -> 7.0 us, 5.1 with accesses at fixed distances).
template <typename T, int G, int VEC>
__global__ void __launch_bounds__(G == 1 ? 1024 : 512, G == 1 || sizeof(T) == 4 ? 2 : 3)
    quantize_rows_kernel(const QuantArgs a) {
  griddep_launch_dependents();  // a product that follows may load its weight meanwhile
  __shared__ uint32_t red[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp & (a.wpr - 1), first = warp - part, shift = __ffs(a.wpr) - 1;  // wpr is a power of two
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> (5 + shift)) + (warp >> shift);
  const bool valid = row < a.rows;
  const T* xr = static_cast<const T*>(a.x) + row * a.cols;
  Raw8<T> x[G];
  uint32_t m = 0;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c0 = (part + g * a.wpr) * 256;
    if (valid && c0 < a.cols) x[g] = load_cols<VEC>(xr, c0, a.cols, lane);
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c0 = (part + g * a.wpr) * 256;
    if (valid && c0 < a.cols) m = max(m, abs_max(x[g]));
  }
  m = row_max(m, red, warp, first, a.wpr);
  if (!valid) return;
  const RowScale rs(m);
  if (part == 0 && lane == 0) a.scale[row] = rs.scale;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int c0 = (part + g * a.wpr) * 256;
    if (c0 < a.cols) store_codes<VEC>(a, row, c0, lane, rs, x[g]);
  }
}

// Rows too long for a block's registers: read twice.
template <typename T>
__global__ void __launch_bounds__(1024) quantize_long_rows_kernel(const QuantArgs a) {
  griddep_launch_dependents();
  __shared__ uint32_t red[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const T* xr = static_cast<const T*>(a.x) + row * a.cols;
  uint32_t m = 0;
  for (int c0 = warp * 256; c0 < a.cols; c0 += 32 * 256)
    m = max(m, abs_max(load_cols<kRagged>(xr, c0, a.cols, lane)));
  const RowScale rs(row_max(m, red, warp, 0, 32));
  if (threadIdx.x == 0) a.scale[row] = rs.scale;
  for (int c0 = warp * 256; c0 < a.cols; c0 += 32 * 256)
    store_codes<kRagged>(a, row, c0, lane, rs, load_cols<kRagged>(xr, c0, a.cols, lane));
}

template <typename T>
cudaError_t launch_quantize_rows(QuantArgs a, cudaStream_t stream) {
  if (a.cols > 16 * 256 * kQuantGroups) {
    quantize_long_rows_kernel<T><<<static_cast<unsigned>(a.rows), 1024, 0, stream>>>(a);
    return cudaGetLastError();
  }
  const bool vec = vector_rows(a.x, a.cols);
  // Few rows: as many warps per row as its columns allow; else four steps each
  // (bf16, 1 x 1024: 1.7 us, 2.1 with four; 290 x 4096: 2.6 against 2.7; at the
  // rule's edge, 290 x 8192, 3.6 against 3.3).
  const int groups = a.rows <= 2 * device_sm_count() && a.cols <= 32 * 256 ? 1 : kQuantGroups;
  a.wpr = 1;
  while (static_cast<int64_t>(a.wpr) * 256 * groups < a.cols) a.wpr *= 2;
  const int warps = std::max(a.wpr, 4);
  const unsigned grid = static_cast<unsigned>((a.rows + warps / a.wpr - 1) / (warps / a.wpr));
  const int layout = vec ? aligned_layout(a.cols) : kRagged;
  if (groups == 1) {
    if (layout == kWhole) quantize_rows_kernel<T, 1, kWhole><<<grid, warps * 32, 0, stream>>>(a);
    else if (layout == kAligned) quantize_rows_kernel<T, 1, kAligned><<<grid, warps * 32, 0, stream>>>(a);
    else quantize_rows_kernel<T, 1, kRagged><<<grid, warps * 32, 0, stream>>>(a);
  } else {
    if (layout == kWhole) quantize_rows_kernel<T, kQuantGroups, kWhole><<<grid, warps * 32, 0, stream>>>(a);
    else if (layout == kAligned) quantize_rows_kernel<T, kQuantGroups, kAligned><<<grid, warps * 32, 0, stream>>>(a);
    else quantize_rows_kernel<T, kQuantGroups, kRagged><<<grid, warps * 32, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_quantize_int8(int32_t dtype, const QuantArgs& a, cudaStream_t stream) {
  if (dtype == QLORA_DTYPE_BF16) return launch_quantize_rows<__nv_bfloat16>(a, stream);
  if (dtype == QLORA_DTYPE_FP16) return launch_quantize_rows<__half>(a, stream);
  return launch_quantize_rows<float>(a, stream);
}

// ================================================================ up to 16 tokens
// Register-fragment products (mma.sync m16n8k32): tokens on the M side, eight
// weight rows on the N side, the weight straight from global memory into the
// fragments.  A lane holds 16 consecutive codes of its row for two products;
// both operands take the same order along the depth, so the sums are the same.
// The 16 warps of a block share the depth and walk over the block's groups of
// eight rows together; each group's partial sums meet in shared memory.
constexpr int kTokenMax = 16;
constexpr int kTokenWarps = 16;
constexpr int kTokenBatch = 4;   // 64-deep steps of two row groups in flight per warp, twice
constexpr int kTokenSlots = 4;   // row groups between two exchanges
static_assert(kTokenSlots % 2 == 0, "pairs of groups");

struct TokenArgs {
  const int8_t* x;
  const int8_t* w;
  const float* sx;
  const float* sw;
  void* y;
  int64_t ldx, ldw;
  int M, K, N, groups;
  int chained;
};

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 codes from position k of a row; where the row ends inside them, nothing
// past it is read.
__device__ __noinline__ uint4 load_tail(const int8_t* row, int k, int K) {
  uint32_t w[4] = {0, 0, 0, 0};
  for (int i = 0; i < 16 && k + i < K; ++i)
    w[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k + i])) << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load_stream(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <typename T>
__device__ __forceinline__ T scaled(int v, float sx, float sw) {
  return from_f32<T>(__fmul_rn(__fmul_rn(static_cast<float>(v), sx), sw));
}

// TWO: tokens 8 .. 15 exist.
template <typename T, bool TWO>
__global__ void __launch_bounds__(kTokenWarps * 32, 1) token_kernel(const TokenArgs a) {
  constexpr int kTokens = TWO ? 16 : 8;
  __shared__ int sums[kTokenSlots][kTokenWarps][kTokens * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int g0 = static_cast<int>(static_cast<int64_t>(a.groups) * blockIdx.x / gridDim.x);
  const int g1 = static_cast<int>(static_cast<int64_t>(a.groups) * (blockIdx.x + 1) / gridDim.x);
  // Whole 64-deep steps, dealt to the warps; the last warp also takes what is
  // left of the depth.
  const int steps = a.K / 64;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * warp / kTokenWarps);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (warp + 1) / kTokenWarps);
  const int batches = (s1 - s0 + kTokenBatch - 1) / kTokenBatch;
  const bool tail = a.K % 64 != 0 && warp == kTokenWarps - 1;
  // Lanes past the last row or token repeat it; their sums are not stored.
  const auto row_of = [&](int group) { return a.w + static_cast<int64_t>(min(group * 8 + g, a.N - 1)) * a.ldw; };
  const int8_t* x0 = a.x + static_cast<int64_t>(min(g, a.M - 1)) * a.ldx;
  const int8_t* x1 = a.x + static_cast<int64_t>(min(g + 8, a.M - 1)) * a.ldx;

  uint4 next[2][kTokenBatch] = {};
  const auto fetch = [&](int group, int batch) {
    const int s = s0 + batch * kTokenBatch;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (group + h < g1) {
        const int8_t* p = row_of(group + h) + s * 64 + q * 16;
#pragma unroll
        for (int i = 0; i < kTokenBatch; ++i)
          if (s + i < s1) next[h][i] = load_stream(p + i * 64);
      }
    }
  };
  // The weight is ready before the kernel that quantizes the tokens started.
  if (!a.chained) griddep_wait();
  if (g0 < g1) fetch(g0, 0);
  if (a.chained) griddep_wait();

  int c[2][4] = {};
  for (int from = g0; from < g1; from += kTokenSlots) {
    const int to = min(g1, from + kTokenSlots);
    // Two groups at a time share the tokens' fragments (one token, 4096 x 4096:
    // 6.8 -> 5.5 us; 16 tokens, 11008 x 4096: 19.2 -> 15.9).
    for (int group = from; group < to; group += 2) {
      const bool pair = group + 1 < to;
      for (int batch = 0; batch < batches; ++batch) {
        uint4 w[2][kTokenBatch];
#pragma unroll
        for (int i = 0; i < kTokenBatch; ++i) {
          w[0][i] = next[0][i];
          w[1][i] = next[1][i];
        }
        if (batch + 1 < batches) fetch(group, batch + 1);
        else if (group + 2 < g1) fetch(group + 2, 0);
        const int s = s0 + batch * kTokenBatch, at = s * 64 + q * 16;
#pragma unroll
        for (int i = 0; i < kTokenBatch; ++i) {
          if (s + i < s1) {
            const uint4 x = *reinterpret_cast<const uint4*>(x0 + at + i * 64);
            const uint4 z = TWO ? *reinterpret_cast<const uint4*>(x1 + at + i * 64) : make_uint4(0, 0, 0, 0);
            mma_s8(c[0], x.x, z.x, x.y, z.y, w[0][i].x, w[0][i].y);
            mma_s8(c[0], x.z, z.z, x.w, z.w, w[0][i].z, w[0][i].w);
            if (pair) {
              mma_s8(c[1], x.x, z.x, x.y, z.y, w[1][i].x, w[1][i].y);
              mma_s8(c[1], x.z, z.z, x.w, z.w, w[1][i].z, w[1][i].w);
            }
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !pair) break;
        if (tail) {
          const int at = steps * 64 + q * 16;
          const uint4 w = load_tail(row_of(group + h), at, a.K), x = load_tail(x0, at, a.K);
          const uint4 z = TWO ? load_tail(x1, at, a.K) : make_uint4(0, 0, 0, 0);
          mma_s8(c[h], x.x, z.x, x.y, z.y, w.x, w.y);
          mma_s8(c[h], x.z, z.z, x.w, z.w, w.z, w.w);
        }
        // c[h][0], c[h][1]: token g, rows 2 q and 2 q + 1 of the group; c[h][2], c[h][3]: token g + 8
        int* out = sums[group + h - from][warp];
        *reinterpret_cast<int2*>(out + g * 8 + 2 * q) = make_int2(c[h][0], c[h][1]);
        if (TWO) *reinterpret_cast<int2*>(out + (g + 8) * 8 + 2 * q) = make_int2(c[h][2], c[h][3]);
        c[h][0] = c[h][1] = c[h][2] = c[h][3] = 0;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (to - from) * 8 * a.M; i += kTokenWarps * 32) {
      const int rows = (to - from) * 8, m = i / rows, r = i - m * rows, row = from * 8 + r;
      int sum = 0;
#pragma unroll
      for (int v = 0; v < kTokenWarps; ++v) sum += sums[r >> 3][v][m * 8 + (r & 7)];
      if (row < a.N)
        static_cast<T*>(a.y)[static_cast<int64_t>(m) * a.N + row] = scaled<T>(sum, __ldg(a.sx + m), __ldg(a.sw + row));
    }
    if (to < g1) __syncthreads();
  }
}

template <typename T>
cudaError_t launch_token(const TokenArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(a.groups, device_sm_count())), 1, 1);
  cfg.blockDim = dim3(kTokenWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.attrs = &attr;
  cfg.numAttrs = a.chained ? 1 : 0;
  return a.M > 8 ? cudaLaunchKernelEx(&cfg, token_kernel<T, true>, a)
                 : cudaLaunchKernelEx(&cfg, token_kernel<T, false>, a);
}

// ================================================================ more tokens
constexpr int kPairTokens = 256;  // rows of a pair's tile (tokens), 128 per CTA
constexpr int kPairCols = 256;    // its columns (weight rows), 128 per CTA
constexpr int kMaxPairs = 80;     // of a launch that splits its tiles

struct PairGemmArgs {
  int M, N, nkb, tiles_m, tiles_n, tiles, group_rows;
  const float* sx;
  const float* sw;
  void* y;
  int vec;        // rows of Y are whole 16-byte vectors
  int split;      // pairs that share a tile
  int* ctr;       // [tiles][2] parts of a split tile that are done; left at zero
  int32_t* part;  // [tiles][split][2] partial sums of 128 rows, [column][row]
  int* status;
  uint64_t wait_ns;
};

struct PairGemmSmem {
  static constexpr int kHalf = 128 * kDepth;  // this CTA's tokens; as many bytes of its weight rows follow
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = 6;
  static constexpr int offBar = kStages * kStage;
  static constexpr int kNumBars = 2 * kStages + 5;
  static constexpr int offSlot = offBar + kNumBars * 8;
  static constexpr int offTurn = (offSlot + 16 + 15) / 16 * 16;  // per epilogue warp 32 x 33 floats
  static constexpr int offScale = offTurn + 4 * 32 * 33 * 4;  // per epilogue warp the tile's column scales
  static constexpr int kTotal = offScale + 4 * kPairCols * 4;
  static constexpr int kDynamic = kTotal + 1024;
};

// Tiles in groups of `group_rows` token blocks, column by column inside a
// group, so that the tiles in flight share both operands in L2.
__device__ __forceinline__ void pair_tile(const PairGemmArgs& a, int tile, int& tm, int& tn) {
  const int per = a.group_rows * a.tiles_n, g = tile / per, at = tile - g * per;
  const int rows = min(a.group_rows, a.tiles_m - g * a.group_rows);
  tn = at / rows;
  tm = g * a.group_rows + at - tn * rows;
}

// The scales of columns col0 .. col0 + n - 1 into a warp's shared memory.
__device__ __forceinline__ void load_scales(const PairGemmArgs& a, int col0, int n, float* to) {
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int c = lane; c < n; c += 32) to[c] = col0 + c < a.N ? __ldg(a.sw + col0 + c) : 0.0f;
}

// 32 columns of a warp's 32 rows of Y from their whole-number sums; `sw` holds
// the columns' scales.
template <typename T>
__device__ __forceinline__ void store_scaled(const PairGemmArgs& a, int row, int col0, const uint32_t (&v)[32],
                                             float sx, const float* sw, float* turn) {
  const int lane = threadIdx.x & 31;
  float f[32];
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float4 s = *reinterpret_cast<const float4*>(sw + e);
    f[e] = __fmul_rn(__fmul_rn(static_cast<float>(static_cast<int>(v[e])), sx), s.x);
    f[e + 1] = __fmul_rn(__fmul_rn(static_cast<float>(static_cast<int>(v[e + 1])), sx), s.y);
    f[e + 2] = __fmul_rn(__fmul_rn(static_cast<float>(static_cast<int>(v[e + 2])), sx), s.z);
    f[e + 3] = __fmul_rn(__fmul_rn(static_cast<float>(static_cast<int>(v[e + 3])), sx), s.w);
  }
  if (a.vec) {
    if (row < a.M) {
      T* out = static_cast<T*>(a.y) + static_cast<int64_t>(row) * a.N;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (col0 + g * 8 < a.N) {
          const float w8[8] = {f[g * 8],     f[g * 8 + 1], f[g * 8 + 2], f[g * 8 + 3],
                               f[g * 8 + 4], f[g * 8 + 5], f[g * 8 + 6], f[g * 8 + 7]};
          store_group(out + col0 + g * 8, raw_from<T>(w8));
        }
      }
    }
  } else {
    // Ragged rows: turn the 32 x 32 block in shared memory, so that a warp
    // stores 32 neighbours of one row at a time.
#pragma unroll
    for (int e = 0; e < 32; ++e) turn[lane * 33 + e] = f[e];
    __syncwarp();
    T* to = static_cast<T*>(a.y) + static_cast<int64_t>(row - lane) * a.N + col0 + lane;
    const int rows = min(32, a.M - (row - lane));
    if (col0 + lane < a.N)
      for (int r = 0; r < rows; ++r) to[static_cast<int64_t>(r) * a.N] = from_f32<T>(turn[r * 33 + lane]);
    __syncwarp();
  }
}

// Without SPLIT: persistent pairs, one tile after the other.  With it: `split`
// pairs on each tile, each a part of the depth; every CTA leaves its partial
// sums in the workspace and the last of a tile's `split` CTAs of one rank adds
// them up.  Nobody waits for another pair.
template <typename T, bool SPLIT>
__global__ void __launch_bounds__(256, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                const PairGemmArgs a) {
  using L = PairGemmSmem;
  constexpr int kStages = L::kStages;
  constexpr uint32_t kTmemCols = 2 * kPairCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::offBar);  // leader: both CTAs' bytes
  uint64_t* empty = full + kStages;                                // local: products done with the stage
  uint64_t* acc_full = empty + kStages;                            // local
  uint64_t* acc_empty = acc_full + 2;                              // leader: both CTAs' epilogue warps
  uint64_t* drain = acc_empty + 2;                                 // leader
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::offSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();  // 0 = leader
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 2) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the leader's barriers exist before the peer uses them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  const int first = SPLIT ? pair / a.split : pair, stride = SPLIT ? a.tiles : pairs;
  const int share = SPLIT ? pair - first * a.split : 0;
  const int kb0 = SPLIT ? a.nkb * share / a.split : 0, kb1 = SPLIT ? a.nkb * (share + 1) / a.split : a.nkb;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const WaitCtx ctx{abort_flag, a.status, 54, a.wait_ns};
      int i = 0;
      bool ok = true;
      griddep_wait();
      for (int tile = first; tile < a.tiles && ok; tile += stride) {
        int tm, tn;
        pair_tile(a, tile, tm, tn);
        const int x_row = tm * kPairTokens + static_cast<int>(rank) * 128;
        const int w_row = tn * kPairCols + static_cast<int>(rank) * 128;
        for (int kb = kb0; kb < kb1; ++kb, ++i) {
          const int s = i % kStages;
          if (!(ok = mbar_wait(&empty[s], ((i / kStages) & 1) ^ 1, ctx))) break;
          const uint32_t bar = map_rank(&full[s], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * L::kStage);
          tma_load_2d_pair(&tmX, bar, smem + s * L::kStage, kb * kDepth, x_row);
          tma_load_2d_pair(&tmW, bar, smem + s * L::kStage + L::kHalf, kb * kDepth, w_row);
        }
      }
      if (*abort_flag && rank == 0)
        for (int k = max(0, i - kStages); k < i; ++k) mbar_drain(&full[k % kStages], (k / kStages) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA (leader)
    if (lane == 0 && rank == 0) {
      const WaitCtx ctx{abort_flag, a.status, 55, a.wait_ns};
      constexpr uint32_t idesc = idesc_s8_s32(kPairTokens, kPairCols);
      int i = 0, seg = 0;
      bool ok = true;
      for (int tile = first; tile < a.tiles && ok; tile += stride, ++seg) {
        if (!(ok = mbar_wait(&acc_empty[seg & 1], ((seg >> 1) & 1) ^ 1, ctx))) break;
        tc_fence_after();
        for (int kb = kb0; kb < kb1; ++kb, ++i) {
          const int s = i % kStages;
          if (!(ok = mbar_wait(&full[s], (i / kStages) & 1, ctx))) break;
          tc_fence_after();
          const uint32_t x = smem_u32(smem + s * L::kStage), w = x + L::kHalf;
#pragma unroll
          for (int k = 0; k < kDepth / 32; ++k)
            umma_s8_pair(tmem + (seg & 1) * kPairCols, smem_desc_sw128(x + k * 32, 16, 1024),
                         smem_desc_sw128(w + k * 32, 16, 1024), idesc, kb > kb0 || k > 0);
          umma_commit_pair(&empty[s]);
        }
        if (ok) umma_commit_pair(&acc_full[seg & 1]);
      }
      if (!ok) {
        umma_commit_pair(drain);
        mbar_drain(drain, 0);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const WaitCtx ctx{abort_flag, a.status, 56, a.wait_ns};
    const int q = warp & 3;
    float* turn = reinterpret_cast<float*>(smem + L::offTurn) + q * 32 * 33;
    float* sw = reinterpret_cast<float*>(smem + L::offScale) + q * kPairCols;
    griddep_wait();
    int seg = 0;
    for (int tile = first; tile < a.tiles && !SPLIT; tile += stride, ++seg) {
      int tm, tn;
      pair_tile(a, tile, tm, tn);
      const int row = tm * kPairTokens + static_cast<int>(rank) * 128 + q * 32 + lane;
      const float sx = row < a.M ? __ldg(a.sx + row) : 0.0f;
      __syncwarp();
      load_scales(a, tn * kPairCols, kPairCols, sw);
      __syncwarp();
      if (!__all_sync(kAll, mbar_wait(&acc_full[seg & 1], (seg >> 1) & 1, ctx))) break;
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + (seg & 1) * kPairCols;
      // Columns of this tile that exist, for warps with rows that do.
      const int cols = row - lane < a.M ? min(kPairCols, a.N - tn * kPairCols) : 0;
#pragma unroll 1
      for (int c = 0; c < cols; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(acc + c, v);
        tmem_wait_ld();
        store_scaled<T>(a, row, tn * kPairCols + c, v, sx, sw + c, turn);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_rank(&acc_empty[seg & 1], 0));
    }
    if (SPLIT) mbar_wait(&acc_full[0], 0, ctx);
  }
  if (SPLIT) {
    // The products are done: all eight warps hand over or add up, each 32 rows
    // of half of the columns.
    __syncthreads();
    tc_fence_after();
    constexpr int kPart = kPairCols * 128;
    const bool ok = *abort_flag == 0;
    const int q = warp & 3;
    int tm, tn;
    pair_tile(a, first, tm, tn);
    const int row = tm * kPairTokens + static_cast<int>(rank) * 128 + q * 32 + lane;
    const int half = (warp >> 2) * (kPairCols / 2);
    const int cols = row - lane < a.M ? min(kPairCols / 2, a.N - tn * kPairCols - half) : 0;
    const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + half;
    int32_t* part = a.part + (static_cast<int64_t>(first) * a.split * 2 + rank) * kPart + half * 128 + q * 32 + lane;
    const float sx = row < a.M ? __ldg(a.sx + row) : 0.0f;
    float* sw = reinterpret_cast<float*>(smem + L::offScale) + warp * (kPairCols / 2);
    load_scales(a, tn * kPairCols + half, kPairCols / 2, sw);
#pragma unroll 1
    for (int c = 0; c < cols; c += 32) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(acc + c, v);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) __stcg(part + share * 2 * kPart + (c + e) * 128, static_cast<int32_t>(v[e]));
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      const bool last = ok && atomicAdd(a.ctr + first * 2 + rank, 1) + 1 == a.split;
      if (last) a.ctr[first * 2 + rank] = 0;  // nobody else adds to it
      *last_flag = last;
      __threadfence();
    }
    __syncthreads();
    if (*last_flag) {
      float* turn = reinterpret_cast<float*>(smem) + warp * 32 * 33;  // the ring is free
#pragma unroll 1
      for (int c = 0; c < cols; c += 64) {
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(acc + c, v[0]);
        tmem_ld_32x32b_x32(acc + c + 32, v[1]);
        tmem_wait_ld();
#pragma unroll 1
        for (int d = 1; d < a.split; ++d) {
          const int p = share + d < a.split ? share + d : share + d - a.split;
          int32_t o[64];
#pragma unroll
          for (int e = 0; e < 64; ++e) o[e] = __ldcg(part + p * 2 * kPart + (c + e) * 128);
#pragma unroll
          for (int e = 0; e < 64; ++e) v[e >> 5][e & 31] += static_cast<uint32_t>(o[e]);
        }
        store_scaled<T>(a, row, tn * kPairCols + half + c, v[0], sx, sw + c, turn);
        if (c + 32 < cols)
          store_scaled<T>(a, row, tn * kPairCols + half + c + 32, v[1], sx, sw + c + 32, turn);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the pair's products or signals may touch it
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

template <typename T, bool SPLIT>
cudaError_t launch_pair_gemm(const CUtensorMap& x, const CUtensorMap& w, const PairGemmArgs& a, int pairs, bool chained,
                             cudaStream_t stream) {
  using L = PairGemmSmem;
  static_assert(L::kDynamic <= 232448, "shared memory budget");
  static_assert(L::offBar % 8 == 0 && L::offScale % 16 == 0, "barriers, and scales read as vectors");
  auto kern = pair_kernel<T, SPLIT>;
  const cudaError_t e = allow_shared_memory(kern, L::kDynamic);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = L::kDynamic;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = pdl_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = chained ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, x, w, a);
}

// Pairs per tile.  A 128-deep block takes a pair about 0.33 us and handing
// over and adding partial sums about 7 us.  Measured with the split chosen here
// against one pair a tile: 64 x 8192 x 8192 21.8 against 24.9 us, 300 x 11003 x
// 4099 30.3 against 39.2, 200 x 8192 x 8192 26.2 against 26.7; a depth of 2048
// stays with one (15.8 us with two, 11.7 with one).
int pair_split(int64_t tiles, int nkb, int sms) {
  const int pairs = std::min(std::max(1, sms / 2), kMaxPairs);
  int best = 1;
  double best_us = 0.33 * nkb;
  for (int s = 2; s * tiles <= pairs && s <= nkb; ++s) {
    const double us = 0.33 * ((nkb + s - 1) / s) + 7.0;
    if (us < best_us) {
      best = s;
      best_us = us;
    }
  }
  return best;
}

// ================================================================ host
constexpr size_t kStatusBytes = 256;

size_t round256(size_t v) { return (v + 255) / 256 * 256; }
int64_t padded_depth(int64_t K) { return (K + 15) / 16 * 16; }

// [status][counters of split tiles][codes and scales of X][partial sums of
// split tiles].  Only the first two, of one size for all shapes, need zeros.
struct Int8Layout {
  size_t ctr, codes, scale, part, total;
};

Int8Layout int8_layout(int64_t M, int64_t K, int64_t N) {
  Int8Layout l{};
  l.ctr = kStatusBytes;
  l.codes = l.ctr + 768;
  static_assert(kMaxPairs * 2 * 4 <= 768, "a counter per tile and rank");
  l.scale = l.codes + round256(static_cast<size_t>(M) * padded_depth(K));
  l.part = l.scale + round256(static_cast<size_t>(M) * 4);
  l.total = l.part;
  const int64_t tiles = ((M + kPairTokens - 1) / kPairTokens) * ((N + kPairCols - 1) / kPairCols);
  if (M > kTokenMax && 2 * tiles <= kMaxPairs) l.total += static_cast<size_t>(kMaxPairs) * kPairTokens * kPairCols * 4;
  return l;
}

qlora_status check_int8_shape(int64_t M, int64_t K, int64_t N) {
  if (M <= 0 || K <= 0 || N <= 0) return QLORA_ERR_INVALID_ARG;
  if (M >= (int64_t(1) << 31) - 32768 || N >= (int64_t(1) << 31) - 32768 || K > kMaxDepth) return QLORA_ERR_UNSUPPORTED;
  // tiles and rows are counted in 32 bits
  if ((M / 128 + 1) * (N / 128 + 1) >= (int64_t(1) << 31)) return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

template <typename T>
cudaError_t launch_product(const int8_t* xq, int64_t ldx, const float* sx, int64_t M, int64_t K, int64_t N,
                           const int8_t* wq, int64_t ldw, const float* sw, T* y, uint8_t* ws, bool chained,
                           cudaStream_t stream) {
  const int nkb = static_cast<int>((K + kDepth - 1) / kDepth);
  if (M <= kTokenMax) {
    const TokenArgs a{xq,  wq,  sx, sw, y, ldx, ldw, static_cast<int>(M), static_cast<int>(K), static_cast<int>(N),
                      static_cast<int>((N + 7) / 8), chained ? 1 : 0};
    return launch_token<T>(a, stream);
  }
  CUtensorMap mx, mw;
  if (!make_map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, K, M, ldx, kDepth, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, wq, K, N, ldw, kDepth, 128, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const int sms = device_sm_count();
  PairGemmArgs a{};
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.nkb = nkb;
  a.tiles_m = static_cast<int>((M + kPairTokens - 1) / kPairTokens);
  a.tiles_n = static_cast<int>((N + kPairCols - 1) / kPairCols);
  a.tiles = a.tiles_m * a.tiles_n;
  a.group_rows = std::min(a.tiles_m, 8);
  a.sx = sx;
  a.sw = sw;
  a.y = y;
  a.vec = N % 8 == 0 && aligned_to(y, 16);
  a.status = reinterpret_cast<int*>(ws);
  a.wait_ns = wait_limit_ns();
  const Int8Layout l = int8_layout(M, K, N);
  a.split = pair_split(a.tiles, nkb, sms);
  a.ctr = reinterpret_cast<int*>(ws + l.ctr);
  a.part = reinterpret_cast<int32_t*>(ws + l.part);
  if (a.split > 1) return launch_pair_gemm<T, true>(mx, mw, a, a.tiles * a.split, chained, stream);
  return launch_pair_gemm<T, false>(mx, mw, a, std::min(a.tiles, std::max(1, sms / 2)), chained, stream);
}

cudaError_t launch_matmul_int8(int32_t dtype, const int8_t* xq, int64_t ldx, const float* sx, int64_t M, int64_t K,
                               int64_t N, const int8_t* wq, int64_t ldw, const float* sw, void* y, uint8_t* ws,
                               bool chained, cudaStream_t st) {
  if (dtype == QLORA_DTYPE_BF16)
    return launch_product(xq, ldx, sx, M, K, N, wq, ldw, sw, static_cast<__nv_bfloat16*>(y), ws, chained, st);
  if (dtype == QLORA_DTYPE_FP16)
    return launch_product(xq, ldx, sx, M, K, N, wq, ldw, sw, static_cast<__half*>(y), ws, chained, st);
  return launch_product(xq, ldx, sx, M, K, N, wq, ldw, sw, static_cast<float*>(y), ws, chained, st);
}

// Row strides in bytes: multiples of 16 that hold a row, below TMA's 2^40.
int64_t code_bytes(int64_t rows, int64_t ld, int64_t used) {  // from the first row to the end of the last
  return rows - 1 > (int64_t(1) << 61) / ld ? int64_t(1) << 61 : (rows - 1) * ld + used;
}
bool bad_stride(int64_t ld, int64_t K) { return ld < K || ld % 16 != 0 || ld >= (int64_t(1) << 40); }

}  // namespace

}  // namespace qlora

using namespace qlora;

extern "C" {

qlora_status qlora_quantize_int8(const void* X, int64_t rows, int64_t cols, int32_t dtype, int8_t* codes, int64_t ld,
                                 float* scale, void* stream) {
  if (!X || !codes || !scale || !known_dtype(dtype)) return QLORA_ERR_INVALID_ARG;
  const qlora_status sh = check_rows(rows, cols);
  if (sh != QLORA_OK) return sh;
  if (bad_stride(ld, cols)) return QLORA_ERR_INVALID_ARG;
  if (!aligned_to(X, dtype_bytes(dtype)) || !aligned16(codes) || !aligned_to(scale, 4)) return QLORA_ERR_ALIGNMENT;
  if (!disjoint({{codes, code_bytes(rows, ld, padded_depth(cols))}, {scale, rows * 4}},
                {{X, rows * cols * dtype_bytes(dtype)}}))
    return QLORA_ERR_INVALID_ARG;
  const QuantArgs a{X, codes, scale, rows, ld, static_cast<int>(cols), 1};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope prof(st, "quantize_int8", 1);
  const cudaError_t e = launch_quantize_int8(dtype, a, st);
  prof.done();
  return e == cudaSuccess ? QLORA_OK : cuda_fail(e);
}

size_t qlora_int8_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  return check_int8_shape(M, K, N) == QLORA_OK ? int8_layout(M, K, N).total : 0;
}

qlora_status qlora_matmul_int8(const int8_t* Xq, int64_t ldx, const float* x_scale, int64_t M, int64_t K, int64_t N,
                               const int8_t* Wq, int64_t ldw, const float* w_scale, void* Y, int32_t dtype,
                               void* workspace, size_t ws_bytes, void* stream) {
  if (!Xq || !x_scale || !Wq || !w_scale || !Y || !known_dtype(dtype)) return QLORA_ERR_INVALID_ARG;
  const qlora_status sh = check_int8_shape(M, K, N);
  if (sh != QLORA_OK) return sh;
  if (bad_stride(ldx, K) || bad_stride(ldw, K)) return QLORA_ERR_INVALID_ARG;
  if (!aligned16(Xq) || !aligned16(Wq) || !aligned_to(x_scale, 4) || !aligned_to(w_scale, 4) ||
      !aligned_to(Y, dtype_bytes(dtype)))
    return QLORA_ERR_ALIGNMENT;
  if (!workspace || ws_bytes < int8_layout(M, K, N).total) return QLORA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return QLORA_ERR_ALIGNMENT;
  if (!disjoint({{Y, M * N * dtype_bytes(dtype)}}, {{Xq, code_bytes(M, ldx, K)}, {Wq, code_bytes(N, ldw, K)},
                                                   {x_scale, M * 4}, {w_scale, N * 4}}))
    return QLORA_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope prof(st, "matmul_int8", 1);
  const cudaError_t e = launch_matmul_int8(dtype, Xq, ldx, x_scale, M, K, N, Wq, ldw, w_scale, Y,
                                           static_cast<uint8_t*>(workspace), false, st);
  prof.done();
  return e == cudaSuccess ? QLORA_OK : cuda_fail(e);
}

qlora_status qlora_linear_int8_fwd(const void* X, int64_t M, int64_t K, int64_t N, int32_t dtype, const int8_t* Wq,
                                   int64_t ldw, const float* w_scale, void* Y, void* workspace, size_t ws_bytes,
                                   void* stream) {
  if (!X || !Wq || !w_scale || !Y || !known_dtype(dtype)) return QLORA_ERR_INVALID_ARG;
  qlora_status sh = check_int8_shape(M, K, N);
  if (sh == QLORA_OK) sh = check_rows(M, K);
  if (sh != QLORA_OK) return sh;
  if (bad_stride(ldw, K)) return QLORA_ERR_INVALID_ARG;
  const int es = dtype_bytes(dtype);
  if (!aligned_to(X, es) || !aligned_to(Y, es) || !aligned16(Wq) || !aligned_to(w_scale, 4)) return QLORA_ERR_ALIGNMENT;
  const Int8Layout l = int8_layout(M, K, N);
  if (!workspace || ws_bytes < l.total) return QLORA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return QLORA_ERR_ALIGNMENT;
  if (!disjoint({{Y, M * N * es}}, {{X, M * K * es}, {Wq, code_bytes(N, ldw, K)}, {w_scale, N * 4}}))
    return QLORA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int8_t* codes = reinterpret_cast<int8_t*>(ws + l.codes);
  float* scale = reinterpret_cast<float*>(ws + l.scale);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope prof(st, "linear_int8_fwd", 2);
  const QuantArgs quant{X, codes, scale, M, padded_depth(K), static_cast<int>(K), 1};
  cudaError_t e = launch_quantize_int8(dtype, quant, st);
  if (e == cudaSuccess)
    e = launch_matmul_int8(dtype, codes, padded_depth(K), scale, M, K, N, Wq, ldw, w_scale, Y, ws, true, st);
  prof.done();
  return e == cudaSuccess ? QLORA_OK : cuda_fail(e);
}

}  // extern "C"
