// The linear layer on an 8-bit integer weight, for serving: inputs quantized
// per token, the weight per output channel, the product in whole numbers.
//
//   s_row = fp32(max|x| / 127),  code = x / s_row to the nearest whole number
//   (ties to even, of the real quotient),  Y = sx[m] sw[n] sum_k xq[m,k] wq[n,k]
//
// Sums are exact in 32-bit integers (depth up to 133144), so no split of the
// depth and no order of work changes a result; float32 enters in the epilogue.
//
// Three kernels:
// - quantization: one pass, rows in registers, HBM-bound;
// - up to 128 tokens, bound by reading the weight once: `stream_kernel` takes
//   128 weight rows as the M side of tcgen05.mma (kind::i8) and the tokens,
//   padded to 16, 32, 64 or 128, as its N side.  The (row tile, 128-deep
//   block) units are dealt to one block per SM in equal contiguous runs, so
//   every SM streams the same number of bytes whatever the shape; a tile whose
//   units lie in several blocks is summed by the block that finishes last,
//   from int32 partial tiles in the workspace;
// - more tokens: `pair_kernel`, persistent CTA pairs (cta_group::2), a 256 x
//   256 or 256 x 128 tile per pair, TMA ring, two accumulators in TMEM so that
//   a tile's epilogue runs under the next tile's products.
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
constexpr int64_t kMaxDepth = 2147483647 / (127 * 127);  // int32 sums stay exact
constexpr int kDepth = 128;                              // bytes of K per stage: one swizzle row

// ================================================================ quantization
constexpr int kQuantGroups = 4;  // steps of 256 columns a warp holds

struct QuantArgs {
  const void* x;
  int8_t* codes;
  float* scale;
  int64_t rows, cols, ld;
  int wpr;
};

// Largest magnitude as bits: NaN orders above infinity, so both survive.
template <typename T>
__device__ __forceinline__ uint32_t abs_bits(const Raw8<T>& x, int e) {
  return __float_as_uint(raw_f32(x, e)) & 0x7FFFFFFFu;
}

struct RowScale {
  float scale, up, s, inv, half;
  __device__ explicit RowScale(uint32_t bits) {
    scale = __fdiv_rn(__uint_as_float(bits), 127.0f);
    // A tiny scale is lifted by an exact power of two, so that its
    // reciprocal stays finite.
    up = scale < 0x1p-100f ? 0x1p64f : 1.0f;
    s = scale * up;
    inv = __fdiv_rn(1.0f, s);
    half = 0.5f * s;
    if (!(bits < 0x7F800000u) || scale == 0.0f) up = s = inv = half = 0.0f;  // all codes 0
  }
  // Nearest whole number to x / scale, ties to even.  The product with the
  // reciprocal is off by far less than a half, and the remainder x - q s is
  // exact in float32 (a multiple of the smaller of the two last places, no
  // larger than s / 2 but for the error of q), so one comparison settles it.
  __device__ __forceinline__ int code(float x) const {
    if (s == 0.0f) return 0;
    x *= up;
    float q = rintf(x * inv);
    const float r = fmaf(-q, s, x);
    const bool odd = static_cast<int>(q) & 1;
    if (r > half || (r == half && odd)) q += 1.0f;
    else if (r < -half || (r == -half && odd)) q -= 1.0f;
    return static_cast<int>(fminf(fmaxf(q, -127.0f), 127.0f));
  }
};

template <bool VEC, typename T>
__device__ __forceinline__ void store_codes(const QuantArgs& a, int64_t row, int64_t c0, int lane, const RowScale& rs,
                                            const Raw8<T>& x) {
  const int64_t padded = (a.cols + 15) / 16 * 16;  // columns past the end hold 0
  int8_t* out = a.codes + row * a.ld;
  if constexpr (VEC) {
    const int64_t c = c0 + lane * 8;
    if (c >= padded) return;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e >> 2] |= (static_cast<uint32_t>(rs.code(raw_f32(x, e))) & 0xFFu) << (8 * (e & 3));
    *reinterpret_cast<uint2*>(out + c) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = c0 + lane + 32 * e;
      if (c < padded) out[c] = static_cast<int8_t>(rs.code(raw_f32(x, e)));
    }
  }
}

__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* buf, int warp, int first, int wpr) {
  v = __reduce_max_sync(kAll, v);
  if (wpr == 1) return v;
  if ((threadIdx.x & 31) == 0) buf[warp] = v;
  __syncthreads();
  uint32_t m = 0;
  for (int i = 0; i < wpr; ++i) m = max(m, buf[first + i]);
  return m;
}

template <typename T, int G, bool VEC>
__global__ void __launch_bounds__(1024) quantize_rows_kernel(const QuantArgs a) {
  griddep_launch_dependents();  // a product that follows may load its weight meanwhile
  __shared__ uint32_t red[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % a.wpr, first = warp - part;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32 / a.wpr) + warp / a.wpr;
  const bool valid = row < a.rows;
  const T* xr = static_cast<const T*>(a.x) + row * a.cols;
  Raw8<T> x[G];
  uint32_t m = 0;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t c0 = static_cast<int64_t>(part + g * a.wpr) * 256;
    if (valid && c0 < a.cols) x[g] = load_cols<VEC>(xr, c0, a.cols, lane);
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t c0 = static_cast<int64_t>(part + g * a.wpr) * 256;
    if (valid && c0 < a.cols) {
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, abs_bits(x[g], e));
    }
  }
  m = row_max(m, red, warp, first, a.wpr);
  if (!valid) return;
  const RowScale rs(m);
  if (part == 0 && lane == 0) a.scale[row] = rs.scale;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int64_t c0 = static_cast<int64_t>(part + g * a.wpr) * 256;
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
  for (int64_t c0 = static_cast<int64_t>(warp) * 256; c0 < a.cols; c0 += 32 * 256) {
    const Raw8<T> x = load_cols<false>(xr, c0, a.cols, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, abs_bits(x, e));
  }
  const RowScale rs(row_max(m, red, warp, 0, 32));
  if (threadIdx.x == 0) a.scale[row] = rs.scale;
  for (int64_t c0 = static_cast<int64_t>(warp) * 256; c0 < a.cols; c0 += 32 * 256)
    store_codes<false>(a, row, c0, lane, rs, load_cols<false>(xr, c0, a.cols, lane));
}

template <typename T>
cudaError_t launch_quantize_rows(QuantArgs a, cudaStream_t stream) {
  if (a.cols > 32 * 256 * kQuantGroups) {
    quantize_long_rows_kernel<T><<<static_cast<unsigned>(a.rows), 1024, 0, stream>>>(a);
    return cudaGetLastError();
  }
  const bool vec = vector_rows(a.x, a.cols);
  // Few rows: as many warps per row as its columns allow; else four steps each.
  const int groups = a.rows <= 2 * device_sm_count() && a.cols <= 32 * 256 ? 1 : kQuantGroups;
  a.wpr = 1;
  while (static_cast<int64_t>(a.wpr) * 256 * groups < a.cols) a.wpr *= 2;
  const int warps = std::max(a.wpr, 4);
  const unsigned grid = static_cast<unsigned>((a.rows + warps / a.wpr - 1) / (warps / a.wpr));
  if (groups == 1) {
    if (vec) quantize_rows_kernel<T, 1, true><<<grid, warps * 32, 0, stream>>>(a);
    else quantize_rows_kernel<T, 1, false><<<grid, warps * 32, 0, stream>>>(a);
  } else {
    if (vec) quantize_rows_kernel<T, kQuantGroups, true><<<grid, warps * 32, 0, stream>>>(a);
    else quantize_rows_kernel<T, kQuantGroups, false><<<grid, warps * 32, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_quantize_int8(int32_t dtype, const QuantArgs& a, cudaStream_t stream) {
  if (dtype == QLORA_DTYPE_BF16) return launch_quantize_rows<__nv_bfloat16>(a, stream);
  if (dtype == QLORA_DTYPE_FP16) return launch_quantize_rows<__half>(a, stream);
  return launch_quantize_rows<float>(a, stream);
}

// ================================================================ few tokens
constexpr int kStreamMax = 128;   // tokens
constexpr int kStreamRows = 128;  // weight rows of a tile
constexpr int kMaxStreamBlocks = 160;
constexpr int kMinRun = 4;        // units a block takes at least

struct StreamArgs {
  int M, N, nkb, tiles;
  int64_t units;
  const float* sx;
  const float* sw;
  void* y;
  int32_t* part;  // [blocks][2][NT][128] partial tiles
  int* ctr;       // [blocks] units done of the split tile that begins in a block; left at zero
  int* status;
  uint64_t wait_ns;
  int chained;    // the previous kernel quantizes the tokens: the weight may be loaded before it ends
};

template <int NT>
struct StreamSmem {
  static constexpr int kW = kStreamRows * kDepth;
  static constexpr int kX = NT * kDepth;
  static constexpr int kStage = kW + kX;
  static constexpr int kStages = std::min(10, 200 * 1024 / kStage);
  static constexpr int offBar = kStages * kStage;
  static constexpr int kNumBars = 2 * kStages + 5;  // full, empty; acc full/empty x 2; drain
  static constexpr int offSlot = offBar + kNumBars * 8;
  static constexpr int kTotal = offSlot + 16;  // tmem address, abort flag, last flag
  static constexpr int kDynamic = kTotal + 1024;
};

__device__ __forceinline__ int64_t run_start(int64_t units, int block, int blocks) { return units * block / blocks; }

template <typename T>
__device__ __forceinline__ T scaled(int v, float sx, float sw) {
  return from_f32<T>(__fmul_rn(__fmul_rn(static_cast<float>(v), sx), sw));
}

template <typename T, int NT>
__global__ void __launch_bounds__(256, 1)
    stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                  const StreamArgs a) {
  using L = StreamSmem<NT>;
  constexpr int kStages = L::kStages;
  constexpr uint32_t kTmemCols = 2 * NT < 32 ? 32 : 2 * NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::offBar);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::offSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int64_t u0 = run_start(a.units, blockIdx.x, gridDim.x), u1 = run_start(a.units, blockIdx.x + 1, gridDim.x);
  const int n = static_cast<int>(u1 - u0);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const WaitCtx ctx{abort_flag, a.status, 51, a.wait_ns};
      const auto load_w = [&](int i) {
        const int64_t u = u0 + i;
        const int tile = static_cast<int>(u / a.nkb), kb = static_cast<int>(u - static_cast<int64_t>(tile) * a.nkb);
        mbar_arrive_expect_tx(&full[i % kStages], L::kStage);
        tma_load_2d(&tmW, &full[i % kStages], smem + (i % kStages) * L::kStage, kb * kDepth, tile * kStreamRows);
      };
      const auto load_x = [&](int i) {
        const int kb = static_cast<int>((u0 + i) % a.nkb);
        tma_load_2d(&tmX, &full[i % kStages], smem + (i % kStages) * L::kStage + L::kW, kb * kDepth, 0);
      };
      // The weight is ready before the kernel that quantizes the tokens
      // started; the codes only once it has ended.
      const int ahead = min(n, kStages);
      if (!a.chained) griddep_wait();
      for (int i = 0; i < ahead; ++i) load_w(i);
      if (a.chained) griddep_wait();
      for (int i = 0; i < ahead; ++i) load_x(i);
      int issued = ahead;
      for (int i = ahead; i < n; ++i) {
        if (!mbar_wait(&empty[i % kStages], ((i / kStages) & 1) ^ 1, ctx)) break;
        load_w(i);
        load_x(i);
        ++issued;
      }
      if (*abort_flag)
        for (int i = max(0, issued - kStages); i < issued; ++i) mbar_drain(&full[i % kStages], (i / kStages) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    if (lane == 0) {
      const WaitCtx ctx{abort_flag, a.status, 52, a.wait_ns};
      constexpr uint32_t idesc = idesc_s8_s32(kStreamRows, NT);
      bool ok = true;
      int seg = -1, prev = -1;
      for (int i = 0; i < n && ok; ++i) {
        const int tile = static_cast<int>((u0 + i) / a.nkb);
        const bool first = tile != prev;
        if (first) {
          prev = tile;
          ++seg;
          if (!(ok = mbar_wait(&acc_empty[seg & 1], ((seg >> 1) & 1) ^ 1, ctx))) break;
        }
        if (!(ok = mbar_wait(&full[i % kStages], (i / kStages) & 1, ctx))) break;
        tc_fence_after();
        const uint32_t w = smem_u32(smem + (i % kStages) * L::kStage), x = w + L::kW;
#pragma unroll
        for (int k = 0; k < kDepth / 32; ++k)
          umma_s8(tmem + (seg & 1) * NT, smem_desc_sw128(w + k * 32, 16, 1024), smem_desc_sw128(x + k * 32, 16, 1024),
                  idesc, !first || k > 0);
        umma_commit(&empty[i % kStages]);
        if (i + 1 == n || static_cast<int>((u0 + i + 1) / a.nkb) != tile) umma_commit(&acc_full[seg & 1]);
      }
      if (!ok) {  // the products already issued must end before the block leaves
        umma_commit(drain);
        mbar_drain(drain, 0);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const WaitCtx ctx{abort_flag, a.status, 53, a.wait_ns};
    const int q = warp & 3, t = q * 32 + lane;  // weight row of the tile
    griddep_wait();                             // sx, the partial tiles and Y
    int seg = 0;
    bool ok = true;  // after a wait that gave up the warp only keeps the barriers below
    for (int64_t u = u0; u < u1; ++seg) {
      const int tile = static_cast<int>(u / a.nkb);
      const int64_t t0 = static_cast<int64_t>(tile) * a.nkb, t1 = t0 + a.nkb;
      const int64_t end = min(u1, t1);
      ok = __all_sync(kAll, ok && mbar_wait(&acc_full[seg & 1], (seg >> 1) & 1, ctx));
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + (seg & 1) * NT;
      const int row = tile * kStreamRows + t;
      const float sw = row < a.N ? __ldg(a.sw + row) : 0.0f;
      T* y = static_cast<T*>(a.y) + row;
      const bool whole = u == t0 && end == t1;
      int32_t* mine = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + (u == t0)) * NT * kStreamRows + t;
#pragma unroll
      for (int c = 0; c < NT / 16; ++c) {
        if (!ok || c * 16 >= a.M) break;
        uint32_t v[16];
        tmem_ld_32x32b_x16(acc + c * 16, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int m = c * 16 + e;
          if (m >= a.M) break;
          if (!whole) mine[m * kStreamRows] = static_cast<int32_t>(v[e]);
          else if (row < a.N) y[static_cast<int64_t>(m) * a.N] = scaled<T>(static_cast<int>(v[e]), __ldg(a.sx + m), sw);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[seg & 1]);
      if (!whole) {
        // The block whose units complete the tile adds up all partial tiles.
        __threadfence();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        // The block this tile begins in: the last whose run starts at or
        // before t0.  It begins no other tile that it does not finish, so the
        // tile's counter is that block's.
        int b0 = static_cast<int>(t0 * gridDim.x / a.units);
        while (b0 + 1 < static_cast<int>(gridDim.x) && run_start(a.units, b0 + 1, gridDim.x) <= t0) ++b0;
        while (b0 > 0 && run_start(a.units, b0, gridDim.x) > t0) --b0;
        if (t == 0) {
          const int add = static_cast<int>(end - u);
          const bool last = ok && atomicAdd(a.ctr + b0, add) + add == a.nkb;
          *last_flag = last;
          if (last) a.ctr[b0] = 0;  // nobody else adds to this tile
          __threadfence();
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (*last_flag) {
          for (int m0 = 0; m0 < a.M; m0 += 8) {
            int sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            for (int b = b0; b < static_cast<int>(gridDim.x); ++b) {
              const int64_t s = run_start(a.units, b, gridDim.x);
              if (s >= t1) break;
              const int32_t* p = a.part + (static_cast<int64_t>(b) * 2 + (s <= t0)) * NT * kStreamRows + t;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (m0 + e < a.M) sum[e] += __ldcg(p + (m0 + e) * kStreamRows);
            }
            if (row < a.N) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (m0 + e < a.M) y[static_cast<int64_t>(m0 + e) * a.N] = scaled<T>(sum[e], __ldg(a.sx + m0 + e), sw);
            }
          }
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");  // last_flag is free again
      }
      u = end;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

int stream_width(int64_t M) { return M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : 128)); }

template <typename T, int NT>
cudaError_t launch_stream_width(const CUtensorMap& w, const CUtensorMap& x, const StreamArgs& a, int grid,
                                cudaStream_t stream) {
  using L = StreamSmem<NT>;
  static_assert(L::kDynamic <= 232448, "shared memory budget");
  auto kern = stream_kernel<T, NT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kDynamic);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = L::kDynamic;
  cfg.stream = stream;
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.attrs = &attr;
  cfg.numAttrs = a.chained ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, w, x, a);
}

template <typename T>
cudaError_t launch_stream(const CUtensorMap& w, const CUtensorMap& x, const StreamArgs& a, int grid, int width,
                          cudaStream_t stream) {
  switch (width) {
    case 16: return launch_stream_width<T, 16>(w, x, a, grid, stream);
    case 32: return launch_stream_width<T, 32>(w, x, a, grid, stream);
    case 64: return launch_stream_width<T, 64>(w, x, a, grid, stream);
    default: return launch_stream_width<T, 128>(w, x, a, grid, stream);
  }
}

// ================================================================ many tokens
constexpr int kPairTokens = 256;  // rows of a pair's tile (tokens), 128 per CTA

struct PairGemmArgs {
  int M, N, nkb, tiles_m, tiles_n, tiles, group_rows;
  const float* sx;
  const float* sw;
  void* y;
  int vec;        // rows of Y are whole 16-byte vectors
  int* status;
  uint64_t wait_ns;
};

template <int BN>
struct PairGemmSmem {
  static constexpr int kX = 128 * kDepth;       // this CTA's tokens
  static constexpr int kW = BN / 2 * kDepth;    // this CTA's half of the weight rows
  static constexpr int kStage = kX + kW;
  static constexpr int kStages = std::min(8, 200 * 1024 / kStage);
  static constexpr int offBar = kStages * kStage;
  static constexpr int kNumBars = 2 * kStages + 5;
  static constexpr int offSlot = offBar + kNumBars * 8;
  static constexpr int kTotal = offSlot + 16;
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

template <typename T, int BN>
__global__ void __launch_bounds__(256, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                const PairGemmArgs a) {
  using L = PairGemmSmem<BN>;
  constexpr int kStages = L::kStages;
  constexpr uint32_t kTmemCols = 2 * BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::offBar);  // leader: both CTAs' bytes
  uint64_t* empty = full + kStages;                                // local: products done with the stage
  uint64_t* acc_full = empty + kStages;                            // local
  uint64_t* acc_empty = acc_full + 2;                              // leader: both CTAs' epilogue warps
  uint64_t* drain = acc_empty + 2;                                 // leader
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::offSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

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
  const int pairs = static_cast<int>(gridDim.x >> 1), first = static_cast<int>(blockIdx.x >> 1);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const WaitCtx ctx{abort_flag, a.status, 54, a.wait_ns};
      int i = 0;
      bool ok = true;
      for (int tile = first; tile < a.tiles && ok; tile += pairs) {
        int tm, tn;
        pair_tile(a, tile, tm, tn);
        const int x_row = tm * kPairTokens + static_cast<int>(rank) * 128;
        const int w_row = tn * BN + static_cast<int>(rank) * (BN / 2);
        for (int kb = 0; kb < a.nkb; ++kb, ++i) {
          const int s = i % kStages;
          if (!(ok = mbar_wait(&empty[s], ((i / kStages) & 1) ^ 1, ctx))) break;
          const uint32_t bar = map_rank(&full[s], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * L::kStage);
          tma_load_2d_pair(&tmX, bar, smem + s * L::kStage, kb * kDepth, x_row);
          tma_load_2d_pair(&tmW, bar, smem + s * L::kStage + L::kX, kb * kDepth, w_row);
        }
      }
      if (*abort_flag && rank == 0)
        for (int k = max(0, i - kStages); k < i; ++k) mbar_drain(&full[k % kStages], (k / kStages) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA (leader)
    if (lane == 0 && rank == 0) {
      const WaitCtx ctx{abort_flag, a.status, 55, a.wait_ns};
      constexpr uint32_t idesc = idesc_s8_s32(kPairTokens, BN);
      int i = 0, seg = 0;
      bool ok = true;
      for (int tile = first; tile < a.tiles && ok; tile += pairs, ++seg) {
        if (!(ok = mbar_wait(&acc_empty[seg & 1], ((seg >> 1) & 1) ^ 1, ctx))) break;
        tc_fence_after();
        for (int kb = 0; kb < a.nkb; ++kb, ++i) {
          const int s = i % kStages;
          if (!(ok = mbar_wait(&full[s], (i / kStages) & 1, ctx))) break;
          tc_fence_after();
          const uint32_t x = smem_u32(smem + s * L::kStage), w = x + L::kX;
#pragma unroll
          for (int k = 0; k < kDepth / 32; ++k)
            umma_s8_pair(tmem + (seg & 1) * BN, smem_desc_sw128(x + k * 32, 16, 1024),
                         smem_desc_sw128(w + k * 32, 16, 1024), idesc, kb > 0 || k > 0);
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
    int seg = 0;
    for (int tile = first; tile < a.tiles; tile += pairs, ++seg) {
      int tm, tn;
      pair_tile(a, tile, tm, tn);
      const int row = tm * kPairTokens + static_cast<int>(rank) * 128 + q * 32 + lane;
      const bool in = row < a.M;
      const float sx = in ? __ldg(a.sx + row) : 0.0f;
      T* out = static_cast<T*>(a.y) + static_cast<int64_t>(row) * a.N;
      if (!__all_sync(kAll, mbar_wait(&acc_full[seg & 1], (seg >> 1) & 1, ctx))) break;
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + (seg & 1) * BN;
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        const int col0 = tn * BN + c * 32;
        if (col0 >= a.N) break;
        uint32_t v[32];
        tmem_ld_32x32b_x32(acc + c * 32, v);
        const float my = col0 + lane < a.N ? __ldg(a.sw + col0 + lane) : 0.0f;
        tmem_wait_ld();
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
          f[e] = __fmul_rn(__fmul_rn(static_cast<float>(static_cast<int>(v[e])), sx), __shfl_sync(kAll, my, e));
        if (in) {
          if (a.vec) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              if (col0 + g * 8 < a.N) {
                const float w8[8] = {f[g * 8], f[g * 8 + 1], f[g * 8 + 2], f[g * 8 + 3],
                                     f[g * 8 + 4], f[g * 8 + 5], f[g * 8 + 6], f[g * 8 + 7]};
                store_group(out + col0 + g * 8, raw_from<T>(w8));
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (col0 + e < a.N) out[col0 + e] = from_f32<T>(f[e]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_rank(&acc_empty[seg & 1], 0));
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

template <typename T, int BN>
cudaError_t launch_pair_gemm(const CUtensorMap& x, const CUtensorMap& w, const PairGemmArgs& a, int pairs,
                             cudaStream_t stream) {
  using L = PairGemmSmem<BN>;
  static_assert(L::kDynamic <= 232448, "shared memory budget");
  auto kern = pair_kernel<T, BN>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kDynamic);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = L::kDynamic;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, x, w, a);
}

// ================================================================ host
constexpr size_t kStatusBytes = 256;

size_t round256(size_t v) { return (v + 255) / 256 * 256; }
int64_t padded_depth(int64_t K) { return (K + 15) / 16 * 16; }

// [status][counters of the few-token tiles][codes and scales of X][partial
// tiles].  Only the first two, of one size for all shapes, need zeros.
struct Int8Layout {
  size_t ctr, part, codes, scale, total;
};

Int8Layout int8_layout(int64_t M, int64_t K) {
  Int8Layout l{};
  l.ctr = kStatusBytes;
  l.codes = l.ctr + round256(kMaxStreamBlocks * 4);
  l.scale = l.codes + round256(static_cast<size_t>(M) * padded_depth(K));
  l.part = l.scale + round256(static_cast<size_t>(M) * 4);
  l.total = l.part;
  if (M <= kStreamMax) l.total += static_cast<size_t>(kMaxStreamBlocks) * 2 * stream_width(M) * kStreamRows * 4;
  return l;
}

qlora_status check_int8_shape(int64_t M, int64_t K, int64_t N) {
  if (M <= 0 || K <= 0 || N <= 0) return QLORA_ERR_INVALID_ARG;
  if (M >= (int64_t(1) << 31) - 512 || N >= (int64_t(1) << 31) - 512 || K > kMaxDepth) return QLORA_ERR_UNSUPPORTED;
  // tiles and rows are counted in 32 bits
  if ((M / 128 + 1) * (N / 128 + 1) >= (int64_t(1) << 31)) return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

template <typename T>
cudaError_t launch_product(const int8_t* xq, int64_t ldx, const float* sx, int64_t M, int64_t K, int64_t N,
                           const int8_t* wq, int64_t ldw, const float* sw, T* y, uint8_t* ws, bool chained,
                           cudaStream_t stream) {
  const Int8Layout l = int8_layout(M, K);
  const int nkb = static_cast<int>((K + kDepth - 1) / kDepth);
  CUtensorMap mx, mw;
  if (M <= kStreamMax) {
    const int width = stream_width(M);
    if (!make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, wq, K, N, ldw, kDepth, kStreamRows,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, K, M, ldx, kDepth, width, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
    StreamArgs a{};
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.nkb = nkb;
    a.tiles = static_cast<int>((N + kStreamRows - 1) / kStreamRows);
    a.units = static_cast<int64_t>(a.tiles) * nkb;
    a.sx = sx;
    a.sw = sw;
    a.y = y;
    a.ctr = reinterpret_cast<int*>(ws + l.ctr);
    a.part = reinterpret_cast<int32_t*>(ws + l.part);
    a.status = reinterpret_cast<int*>(ws);
    a.wait_ns = wait_limit_ns();
    a.chained = chained ? 1 : 0;
    const int64_t want = (a.units + kMinRun - 1) / kMinRun;
    const int grid = static_cast<int>(std::min<int64_t>(want, std::min(device_sm_count(), kMaxStreamBlocks)));
    return launch_stream<T>(mw, mx, a, grid, width, stream);
  }
  PairGemmArgs a{};
  const int tiles_m = static_cast<int>((M + kPairTokens - 1) / kPairTokens);
  const int pairs = std::max(1, device_sm_count() / 2);
  // The narrower tile when it fills the last wave of pairs better.
  const auto waves = [&](int bn) {
    const int64_t tiles = static_cast<int64_t>(tiles_m) * ((N + bn - 1) / bn);
    return (tiles + pairs - 1) / pairs * bn;
  };
  const int bn = waves(128) < waves(256) ? 128 : 256;
  if (!make_map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, K, M, ldx, kDepth, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, wq, K, N, ldw, kDepth, bn / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.nkb = nkb;
  a.tiles_m = tiles_m;
  a.tiles_n = static_cast<int>((N + bn - 1) / bn);
  a.tiles = a.tiles_m * a.tiles_n;
  a.group_rows = std::min(tiles_m, 8);
  a.sx = sx;
  a.sw = sw;
  a.y = y;
  a.vec = N % 8 == 0 && aligned_to(y, 16);
  a.status = reinterpret_cast<int*>(ws);
  a.wait_ns = wait_limit_ns();
  const int grid = std::min(a.tiles, pairs);
  return bn == 128 ? launch_pair_gemm<T, 128>(mx, mw, a, grid, stream)
                   : launch_pair_gemm<T, 256>(mx, mw, a, grid, stream);
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
  const QuantArgs a{X, codes, scale, rows, cols, ld, 1};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope prof(st, "quantize_int8", 1);
  const cudaError_t e = launch_quantize_int8(dtype, a, st);
  prof.done();
  return e == cudaSuccess ? QLORA_OK : cuda_fail(e);
}

size_t qlora_int8_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  return check_int8_shape(M, K, N) == QLORA_OK ? int8_layout(M, K).total : 0;
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
  if (!workspace || ws_bytes < int8_layout(M, K).total) return QLORA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return QLORA_ERR_ALIGNMENT;
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
  const Int8Layout l = int8_layout(M, K);
  if (!workspace || ws_bytes < l.total) return QLORA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return QLORA_ERR_ALIGNMENT;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int8_t* codes = reinterpret_cast<int8_t*>(ws + l.codes);
  float* scale = reinterpret_cast<float*>(ws + l.scale);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope prof(st, "linear_int8_fwd", 2);
  cudaError_t e = launch_quantize_int8(dtype, QuantArgs{X, codes, scale, M, K, padded_depth(K), 1}, st);
  if (e == cudaSuccess)
    e = launch_matmul_int8(dtype, codes, padded_depth(K), scale, M, K, N, Wq, ldw, w_scale, Y, ws, true, st);
  prof.done();
  return e == cudaSuccess ? QLORA_OK : cuda_fail(e);
}

}  // extern "C"
