// Element types, row addressing and random draws shared by the row-wise
// kernels (dropout, layer norm, 8-bit row quantization).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace qlora {

// Eight consecutive elements as loaded: one 16-byte vector of bf16 or fp16,
// two of float32.
template <typename T>
struct Raw8 {
  uint32_t w[sizeof(T) * 2];
};

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// Value e (0..7) of a loaded group.
template <typename T>
__device__ __forceinline__ float raw_f32(const Raw8<T>& r, int e);
template <>
__device__ __forceinline__ float raw_f32<__nv_bfloat16>(const Raw8<__nv_bfloat16>& r, int e) {
  const uint32_t w = r.w[e >> 1];
  return __uint_as_float((e & 1) ? (w & 0xFFFF0000u) : (w << 16));
}
template <>
__device__ __forceinline__ float raw_f32<__half>(const Raw8<__half>& r, int e) {
  const uint32_t w = r.w[e >> 1];
  return __half2float(__ushort_as_half(static_cast<unsigned short>((e & 1) ? (w >> 16) : (w & 0xFFFFu))));
}
template <>
__device__ __forceinline__ float raw_f32<float>(const Raw8<float>& r, int e) { return __uint_as_float(r.w[e]); }

// A group from eight float32 values, each rounded once to T.
template <typename T>
__device__ __forceinline__ Raw8<T> raw_from(const float (&v)[8]);
template <>
__device__ __forceinline__ Raw8<__nv_bfloat16> raw_from<__nv_bfloat16>(const float (&v)[8]) {
  Raw8<__nv_bfloat16> r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    r.w[e] = __bfloat16_as_ushort(p.x) | (static_cast<uint32_t>(__bfloat16_as_ushort(p.y)) << 16);
  }
  return r;
}
template <>
__device__ __forceinline__ Raw8<__half> raw_from<__half>(const float (&v)[8]) {
  Raw8<__half> r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 p = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
    r.w[e] = __half_as_ushort(p.x) | (static_cast<uint32_t>(__half_as_ushort(p.y)) << 16);
  }
  return r;
}
template <>
__device__ __forceinline__ Raw8<float> raw_from<float>(const float (&v)[8]) {
  Raw8<float> r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r.w[e] = __float_as_uint(v[e]);
  return r;
}

// Group transfers through 16-byte vectors (the address is 16-byte aligned).
// "Stream" marks data that is touched once.
template <typename T>
__device__ __forceinline__ Raw8<T> load_group(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
    const uint4 v = *(reinterpret_cast<const uint4*>(p) + i);
    r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
  }
  return r;
}
template <typename T>
__device__ __forceinline__ Raw8<T> load_group_stream(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void store_group(T* p, const Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
    *(reinterpret_cast<uint4*>(p) + i) = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
}
template <typename T>
__device__ __forceinline__ void store_group_stream(T* p, const Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
    __stcs(reinterpret_cast<uint4*>(p) + i, make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]));
}

// ---------------------------------------------------------------- columns of a warp
// A warp owns 256 consecutive columns of a row at a time, eight per lane.
// With aligned rows lane l holds columns 8 l .. 8 l + 7 (one group); with
// ragged rows it holds l, l + 32, ... so that scalar accesses coalesce.
template <bool VEC>
__device__ __forceinline__ int warp_col(int lane, int e) { return VEC ? lane * 8 + e : lane + 32 * e; }

// The warp's 8 values per lane of row[c0 ..], `fill` past the end.
template <bool VEC, typename T>
__device__ __forceinline__ Raw8<T> load_cols(const T* row, int64_t c0, int64_t cols, int lane) {
  if constexpr (VEC) {
    const int64_t c = c0 + lane * 8;
    if (c < cols) return load_group(row + c);
    Raw8<T> z;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) * 2; ++i) z.w[i] = 0;
    return z;
  } else {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = c0 + lane + 32 * e;
      v[e] = c < cols ? to_f32(row[c]) : 0.0f;
    }
    return raw_from<T>(v);  // exact: the values came from T
  }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store_cols(T* row, int64_t c0, int64_t cols, int lane, const float (&v)[8]) {
  if constexpr (VEC) {
    const int64_t c = c0 + lane * 8;
    if (c < cols) store_group(row + c, raw_from<T>(v));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = c0 + lane + 32 * e;
      if (c < cols) row[c] = from_f32<T>(v[e]);
    }
  }
}

// ---------------------------------------------------------------- random draws
// Philox4x32-10: Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3" (SC 2011): ten rounds of two 32 x 32 -> 64 bit products
// over a 128-bit counter, with a key that grows by a Weyl constant per round.
struct Draws {
  uint32_t w[4];
};

__device__ __forceinline__ Draws philox(uint64_t counter, uint64_t key) {
  uint32_t c0 = static_cast<uint32_t>(counter), c1 = static_cast<uint32_t>(counter >> 32), c2 = 0, c3 = 0;
  uint32_t k0 = static_cast<uint32_t>(key), k1 = static_cast<uint32_t>(key >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Draws{{c0, c1, c2, c3}};
}

// What a dropout needs: an element is dropped when its 16-bit draw is below
// `threshold` = round(65536 p); what is kept is multiplied by `gain`.
struct DropArgs {
  uint64_t seed;
  uint64_t offset;
  const uint64_t* offset_dev;  // added to offset when not null
  uint32_t threshold;          // 0 .. 65536
  float gain;
  int64_t groups;              // counters per row: ceil(cols / 8)
};

__device__ __forceinline__ uint64_t drop_base(const DropArgs& d) {
  return d.offset + (d.offset_dev ? *d.offset_dev : 0);
}

// Bit e is set when element e of the group with this counter is kept.
__device__ __forceinline__ uint32_t keep_bits(const DropArgs& d, uint64_t counter) {
  const Draws r = philox(counter, d.seed);
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t draw = (e & 1) ? (r.w[e >> 1] >> 16) : (r.w[e >> 1] & 0xFFFFu);
    m |= (draw >= d.threshold ? 1u : 0u) << e;
  }
  return m;
}

// The same for the eight columns a lane holds (warp_col) of the 256 at
// `counter0` (the counter of the warp's first group).  All lanes take part.
template <bool VEC>
__device__ __forceinline__ uint32_t keep_bits_cols(const DropArgs& d, uint64_t counter0, int lane) {
  const uint32_t own = keep_bits(d, counter0 + lane);
  if constexpr (VEC) {
    return own;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int col = lane + 32 * e;
      m |= ((__shfl_sync(0xFFFFFFFFu, own, col >> 3) >> (col & 7)) & 1u) << e;
    }
    return m;
  }
}

}  // namespace qlora
