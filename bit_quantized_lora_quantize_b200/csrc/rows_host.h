// Host side of the row-wise kernels: argument checks shared by their entry
// points, and the dropout launch that the linear with adapter dropout uses.
// Not part of the public header.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>
#include <initializer_list>

#include "../../include/qlora.h"
#include "rows_device.cuh"

namespace qlora {

constexpr int64_t kMaxRowElements = int64_t(1) << 40;

inline int dtype_bytes(int32_t dtype) { return dtype == QLORA_DTYPE_FP32 ? 4 : 2; }
inline bool known_dtype(int32_t dtype) {
  return dtype == QLORA_DTYPE_BF16 || dtype == QLORA_DTYPE_FP16 || dtype == QLORA_DTYPE_FP32;
}
inline bool aligned_to(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
// Layout that aligned rows of this many columns have.  Rows of whole 256-column
// steps have kernels of their own, without a test per lane: 4096 x 8192 in bf16
// takes 28.7 us in the norm's forward against 32.0 by the aligned ones, 48.2
// against 51.8 fused, 70.9 against 79.0 in the fused backward with dZ, and 20.4
// against 21.7 in the quantization (norm's backward alone 46.7 against 46.9).
inline int aligned_layout(int64_t cols) { return cols % 256 == 0 ? kWhole : kAligned; }
// Rows of whole 16-byte vectors: eight-element groups never straddle rows.
inline bool vector_rows(const void* p, int64_t cols) { return cols % 8 == 0 && aligned_to(p, 16); }

// Memory a call reads or writes; none where the pointer is null.
struct Span {
  const void* p;
  int64_t bytes;
};
// The outputs share no byte with an input or with one another.
inline bool disjoint(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
  const auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && (x < y ? y - x < static_cast<uintptr_t>(a.bytes) : x - y < static_cast<uintptr_t>(b.bytes));
  };
  for (const Span* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Span& i : inputs)
      if (meet(*o, i)) return false;
    for (const Span* other = outputs.begin(); other != o; ++other)
      if (meet(*o, *other)) return false;
  }
  return true;
}

inline qlora_status check_rows(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return QLORA_ERR_INVALID_ARG;
  if (rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31) - 65536 || rows > kMaxRowElements / cols)
    return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

// Threshold and gain of a dropout probability (0 <= p <= 1); false when p is
// outside that range or the counter pointer is misaligned.
inline bool make_drop_args(double p, uint64_t seed, uint64_t offset, const uint64_t* offset_dev, int64_t cols,
                           DropArgs* d) {
  if (!(p >= 0.0 && p <= 1.0) || !aligned_to(offset_dev, 8)) return false;
  d->offset = offset;
  d->offset_dev = offset_dev;
  for (uint32_t i = 0; i < 10; ++i) {
    d->keys[i][0] = static_cast<uint32_t>(seed) + i * 0x9E3779B9u;
    d->keys[i][1] = static_cast<uint32_t>(seed >> 32) + i * 0xBB67AE85u;
  }
  const uint32_t threshold = static_cast<uint32_t>(std::nearbyint(65536.0 * p));
  d->above = (threshold << 16) - 1u;
  d->all = threshold == 0;
  d->gain = threshold < 65536u ? 65536.0f / static_cast<float>(65536u - threshold) : 0.0f;
  d->groups = (cols + 7) / 8;
  return true;
}

// Y = keep * (X * gain) + residual (residual may be null).
cudaError_t launch_dropout(int32_t dtype, const void* X, const void* residual, void* Y, int64_t rows, int64_t cols,
                           const DropArgs& d, cudaStream_t stream);

// dX = bf16(base + keep * (U A^T)): U as its bf16 pair [M x 2 rp], A [K x r] with
// r a multiple of 8, base float32 [K / 8][M][8], dX bf16 [M x K].
cudaError_t launch_adapter_dx(const uint16_t* Upair, const uint16_t* A, const float* base, uint16_t* dX, int64_t M,
                              int64_t K, int r, const DropArgs& d, cudaStream_t stream);

}  // namespace qlora
