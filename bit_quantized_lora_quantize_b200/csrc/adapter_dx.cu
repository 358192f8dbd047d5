// The adapter's part of the input gradient under adapter dropout:
//   dX[m, k] = bf16(base[m, k] + keep[m, k] * sum_j U[m, j] A[k, j])
// (base is dY W' as the GEMM accumulated it, in float32, so that dX is rounded
// once; U carries the LoRA scale and the dropout's gain; the mask is drawn again).
// Base lies as groups of eight columns, [K / 8][M][8]: the GEMM's lanes hold one
// row each, so a warp of them writes whole lines.
//
// A pass over dX: 6 bytes of HBM traffic per element against 4 r operations,
// so HBM would allow 30.7 us for 4096 x 8192 at rank 64; measured 56 us (50 with
// base in bf16, which rounds dX twice), a seventh of the input-gradient GEMM of
// an 8192 x 8192 layer before it.  A block takes a 64 x 128 tile; U enters as its
// bf16 pair (hi + lo, about 16 significant bits), 64 ranks at a time by
// asynchronous copies.
//
// The weight rows are handed to the tensor cores in an order that leaves each
// lane with eight consecutive columns of dX: output column c of the 8-wide
// block b of a warp's 32 columns is column 8 (c / 2) + 2 b + c % 2 of them.
// So one 16-byte load, one Philox output and one 16-byte store serve a lane's
// eight sums, straight from the accumulators.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "ptx.cuh"
#include "rows_host.h"

namespace qlora {

namespace {

constexpr int kTileM = 64;
constexpr int kTileK = 128;
constexpr int kThreads = 256;  // 2 x 4 warps of 32 x 32
constexpr int kRanks = 64;     // ranks per step
constexpr int kUBytes = kTileM * kRanks * 2;
constexpr int kABytes = kTileK * kRanks * 2;

// 16 bytes to shared memory; zeros when `in` is false (nothing is read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offsets of 16-byte chunk `c` of a 128-byte row.  Rows of U are read
// eight consecutive ones at a time; rows of A by the permutation above, eight
// that share bits 1 and 2.
__device__ __forceinline__ uint32_t u_offset(int row, int c) { return row * 128 + ((c ^ (row & 7)) << 4); }
__device__ __forceinline__ uint32_t a_offset(int row, int c) {
  return row * 128 + ((c ^ (((row >> 3) & 3) * 2 + (row & 1))) << 4);
}

__global__ void __launch_bounds__(kThreads, 3)
    adapter_dx_kernel(const uint16_t* __restrict__ U, const uint16_t* __restrict__ A, const float* __restrict__ base,
                      uint16_t* __restrict__ dX, int64_t M, int64_t base_rows, int64_t K, int r, int rp,
                      const DropArgs d) {
  __shared__ __align__(1024) uint8_t smem[2 * kUBytes + kABytes];
  const uint32_t s_hi = smem_u32(smem), s_lo = s_hi + kUBytes, s_a = s_lo + kUBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = (warp & 1) * 32, wn = (warp >> 1) * 32;
  const int64_t k0 = static_cast<int64_t>(blockIdx.x) * kTileK, m0 = static_cast<int64_t>(blockIdx.y) * kTileM;

  // Thread t copies 16-byte chunk t % 8 of rows t / 8, t / 8 + 32, ...
  const int crow = threadIdx.x >> 3, chunk = threadIdx.x & 7;
  const int rows_m = static_cast<int>(min(static_cast<int64_t>(kTileM), M - m0));
  const int rows_k = static_cast<int>(min(static_cast<int64_t>(kTileK), K - k0));
  const uint16_t* u_src = U + (m0 + crow) * 2 * rp + chunk * 8;
  const uint16_t* a_src = A + (k0 + crow) * r + chunk * 8;
  const auto fetch_a = [&](int j0) {
#pragma unroll
    for (int t = 0; t < kTileK / 32; ++t) {
      const int row = crow + t * 32;
      const bool in = row < rows_k && j0 + chunk * 8 < r;
      copy16(s_a + a_offset(row, chunk), in ? a_src + t * 32 * r + j0 : A, in);
    }
  };
  const auto fetch_u = [&](int j0) {
#pragma unroll
    for (int t = 0; t < kTileM / 32; ++t) {
      const int row = crow + t * 32;
      const bool in = row < rows_m;
      const uint16_t* p = in ? u_src + t * 64 * rp + j0 : U;
      copy16(s_hi + u_offset(row, chunk), p, in);
      copy16(s_lo + u_offset(row, chunk), p + (in ? rp : 0), in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // A is ready before the GEMM that computes U and the rest of dX starts.
  fetch_a(0);
  griddep_wait();
  fetch_u(0);

  float acc[2][4][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][b][e] = 0.0f;

  for (int j0 = 0; j0 < rp; j0 += kRanks) {
    if (j0) {
      __syncthreads();  // the previous step's fragments have been read
      fetch_a(j0);
      fetch_u(j0);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kRanks / 16; ++kk) {
      uint32_t uh[2][4], ul[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // matrices: rows 0-7 and 8-15 of the first eight ranks, then of the next
        const int row = wm + 16 * i + (lane & 15), c = 2 * kk + (lane >> 4);
        ldmatrix_x4(s_hi + u_offset(row, c), uh[i]);
        ldmatrix_x4(s_lo + u_offset(row, c), ul[i]);
      }
#pragma unroll
      for (int bb = 0; bb < 2; ++bb) {
        // two 8-wide blocks: matrices (block 2 bb, ranks 0-7), (ranks 8-15), (block 2 bb + 1, ...)
        uint32_t w[4];
        const int b = 2 * bb + (lane >> 4), n = lane & 7;
        const int row = wn + (n >> 1) * 8 + b * 2 + (n & 1);
        ldmatrix_x4(s_a + a_offset(row, 2 * kk + ((lane >> 3) & 1)), w);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma_bf16(acc[i][2 * bb], uh[i], w[0], w[1]);
          mma_bf16(acc[i][2 * bb + 1], uh[i], w[2], w[3]);
          mma_bf16(acc[i][2 * bb], ul[i], w[0], w[1]);
          mma_bf16(acc[i][2 * bb + 1], ul[i], w[2], w[3]);
        }
      }
    }
  }

  // This lane's groups of eight: rows wm + 16 i + 8 h + lane / 4, columns
  // wn + 8 (lane % 4).  K % 64 == 0, so a group is whole or outside.  Three
  // blocks per SM hide these loads and the draws better than registers held
  // for them across the products did (4096 x 8192 at rank 64, with base in bf16:
  // 49 us, 57 with two blocks).
  const int64_t k = k0 + wn + 8 * (lane & 3);
  const int row0 = wm + (lane >> 2);
  if (k >= K) return;
  uint16_t* at = dX + (m0 + row0) * K + k;
  const float* from = base + (k / 8 * base_rows + m0 + row0) * 8;
  uint64_t counter = drop_base(d) + (m0 + row0) * d.groups + k / 8;
  const int64_t step = 8 * K, steps = 8 * d.groups;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    Raw8<float> x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (row0 + 16 * i + 8 * h < rows_m) x[h] = load_group_stream(from + (2 * i + h) * 64);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (row0 + 16 * i + 8 * h < rows_m) {
        const KeepGroup keep = keep_group(d, counter);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = raw_f32(x[h], e) + (keep(e) ? acc[i][e >> 1][2 * h + (e & 1)] : 0.0f);
        store_group_stream(reinterpret_cast<__nv_bfloat16*>(at), raw_from<__nv_bfloat16>(v));
      }
      at += step;
      counter += steps;
    }
  }
}

}  // namespace

cudaError_t launch_adapter_dx(const uint16_t* Upair, const uint16_t* A, const float* base, uint16_t* dX, int64_t M,
                              int64_t K, int r, const DropArgs& d, cudaStream_t stream) {
  // Row blocks beyond a grid's second dimension go to further launches.
  constexpr int64_t kMaxRowBlocks = 65535;
  const int64_t row_blocks = (M + kTileM - 1) / kTileM;
  for (int64_t b = 0; b < row_blocks; b += kMaxRowBlocks) {
    const int64_t m0 = b * kTileM;
    DropArgs part = d;
    part.offset += static_cast<uint64_t>(m0) * d.groups;
    const dim3 grid(static_cast<unsigned>((K + kTileK - 1) / kTileK),
                    static_cast<unsigned>(row_blocks - b < kMaxRowBlocks ? row_blocks - b : kMaxRowBlocks));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr = pdl_attribute();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, adapter_dx_kernel, Upair + m0 * 2 * lora_pad(r), A, base + m0 * 8,
                                             dX + m0 * K, M - m0, M, K, r, lora_pad(r), part);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace qlora
