// Element types, row addressing and random draws shared by the row-wise
// kernels (dropout, layer norm, 8-bit row quantization).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

namespace qlora {

// Eight consecutive elements as loaded: one 16-byte vector of bf16 or fp16,
// two of float32.
template <typename T>
struct Raw8 {
  uint32_t w[sizeof(T) * 2];
};

// Single elements.
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
    r.w[e] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return r;
}
template <>
__device__ __forceinline__ Raw8<__half> raw_from<__half>(const float (&v)[8]) {
  Raw8<__half> r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 p = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
    r.w[e] = *reinterpret_cast<const uint32_t*>(&p);
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

__device__ __forceinline__ bool aligned_group(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

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

// ---------------------------------------------------------------- pairs of float32
// Two float32 values in a 64-bit register: one instruction adds, multiplies or
// multiply-adds both.
using F2 = unsigned long long;

__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ F2 f2_all(float v) { return f2(v, v); }
__device__ __forceinline__ float2 f2_get(F2 a) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
  return d;
}
__device__ __forceinline__ float f2_sum(F2 a) {
  const float2 d = f2_get(a);
  return d.x + d.y;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Elements 2 p and 2 p + 1 of a group.
template <typename T>
__device__ __forceinline__ F2 raw_f2(const Raw8<T>& r, int p) { return f2(raw_f32(r, 2 * p), raw_f32(r, 2 * p + 1)); }

// All four pairs.
template <typename T>
__device__ __forceinline__ void raw_pairs(const Raw8<T>& r, F2 (&v)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) v[p] = raw_f2(r, p);
}

// A group from four pairs, each value rounded once to T.
template <typename T>
__device__ __forceinline__ Raw8<T> raw_from_pairs(const F2 (&v)[4]) {
  float f[8];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 d = f2_get(v[p]);
    f[2 * p] = d.x;
    f[2 * p + 1] = d.y;
  }
  return raw_from<T>(f);
}

// ---------------------------------------------------------------- columns of a warp
// A warp owns 256 consecutive columns of a row at a time, eight per lane.
// With aligned rows lane l holds columns 8 l .. 8 l + 7 (one group); with
// ragged rows it holds l, l + 32, ... so that scalar accesses coalesce.  The
// template argument tells how rows lie:
enum RowLayout {
  kRagged = 0,   // anything
  kAligned = 1,  // whole groups on 16-byte boundaries
  kWhole = 2,    // the same, and a multiple of 256 columns: no lane is past the end
};
// Column numbers stay below 2^31 (check_rows leaves room for the last step).
template <int VEC>
__device__ __forceinline__ int warp_col(int lane, int e) { return VEC ? lane * 8 + e : lane + 32 * e; }

template <typename T>
__device__ __forceinline__ Raw8<T> raw_zero() {
  Raw8<T> z;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) * 2; ++i) z.w[i] = 0;
  return z;
}

template <typename T>
__device__ __forceinline__ Raw8<T> raw_ones() {
  const float v[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
  return raw_from<T>(v);
}

// The lane's eight columns of row[c0 ..] (global or shared memory), zeros past
// the end.
template <int VEC, bool SPLIT = true, typename T>
__device__ __forceinline__ Raw8<T> load_cols(const T* row, int c0, int cols, int lane) {
  if constexpr (VEC) {
    const int c = c0 + lane * 8;
    return VEC == kWhole || c < cols ? load_group(row + c) : raw_zero<T>();
  } else {
    // No column is past the end but in a row's last step: unconditional
    // accesses at fixed distances otherwise (layer norm of 4096 x 4095 in bf16
    // 41.2 -> 24.2 us).  SPLIT = false takes one path for both.
    using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
    const Bits* p = reinterpret_cast<const Bits*>(row) + (c0 + lane);
    uint32_t h[8];
    if (SPLIT && c0 + 256 <= cols) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = p[32 * e];
    } else {
      const int n = cols - c0 - lane;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = 32 * e < n ? p[32 * e] : 0u;
    }
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.w[e] = h[e];
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) r.w[q] = __byte_perm(h[2 * q], h[2 * q + 1], 0x5410);
    }
    return r;
  }
}

template <int VEC, bool SPLIT = true, typename T>
__device__ __forceinline__ void store_cols(T* row, int c0, int cols, int lane, const Raw8<T>& r) {
  if constexpr (VEC) {
    const int c = c0 + lane * 8;
    if (VEC == kWhole || c < cols) store_group(row + c, r);
  } else {
    using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
    Bits* p = reinterpret_cast<Bits*>(row) + (c0 + lane);
    const auto bits = [&](int e) {
      return sizeof(T) == 4 ? static_cast<Bits>(r.w[e % (sizeof(T) * 2)])
                            : static_cast<Bits>(r.w[e >> 1] >> (16 * (e & 1)));
    };
    if (SPLIT && c0 + 256 <= cols) {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[32 * e] = bits(e);
    } else {
      const int n = cols - c0 - lane;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (32 * e < n) p[32 * e] = bits(e);
    }
  }
}

// ---------------------------------------------------------------- random draws
// Philox4x32-10: Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3" (SC 2011): ten rounds of two 32 x 32 -> 64 bit products
// over a 128-bit counter, with a key that grows by a Weyl constant per round.
// The draws are most of what a drawing kernel issues (the dropout of 4096 x 8192
// in bf16: ALU pipe 62 %, issue slots 61 % busy), so the rounds' keys come from
// the host as constants (25.9 -> 20.9 us there, together with the comparison
// below).
struct Draws {
  uint32_t w[4];
};

// What a dropout needs: an element is dropped when its 16-bit draw is below
// threshold = round(65536 p); what is kept is multiplied by `gain`.
struct DropArgs {
  uint64_t offset;
  const uint64_t* offset_dev;  // added to offset when not null
  uint32_t keys[10][2];        // of the rounds
  uint32_t above;              // (threshold << 16) - 1: a draw in the upper half word is kept when the word is above
  bool all;                    // threshold 0: everything is kept
  float gain;
  int64_t groups;              // counters per row: ceil(cols / 8)
};

__device__ __forceinline__ Draws philox(uint64_t counter, const DropArgs& d) {
  uint32_t c0 = static_cast<uint32_t>(counter), c1 = static_cast<uint32_t>(counter >> 32), c2 = 0, c3 = 0;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ d.keys[i][0];
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ d.keys[i][1];
    c3 = static_cast<uint32_t>(a);
  }
  return Draws{{c0, c1, c2, c3}};
}

__device__ __forceinline__ uint64_t drop_base(const DropArgs& d) {
  return d.offset + (d.offset_dev ? *d.offset_dev : 0);
}

// Which of a lane's eight elements are kept.
struct KeepGroup {  // of one group, straight from its draws
  Draws r;
  uint32_t above;
  bool all;
  __device__ __forceinline__ bool operator()(int e) const {
    // Draws compare in the upper half word; what lies below it cannot change
    // the outcome.
    return ((e & 1) ? r.w[e >> 1] : (r.w[e >> 1] << 16)) > above || all;
  }
};
struct KeepBits {  // bit 4 e: element e
  uint32_t bits;
  __device__ __forceinline__ bool operator()(int e) const { return (bits >> (4 * e)) & 1u; }
};

__device__ __forceinline__ KeepGroup keep_group(const DropArgs& d, uint64_t counter) {
  return KeepGroup{philox(counter, d), d.above, d.all};
}

// The same for the eight columns a lane holds (warp_col) of the 256 at
// `counter0` (the counter of the warp's first group).  All lanes take part.
template <int VEC>
__device__ __forceinline__ auto keep_cols(const DropArgs& d, uint64_t counter0, int lane) {
  const KeepGroup own = keep_group(d, counter0 + lane);
  if constexpr (VEC) {
    return own;
  } else {
    // Column lane + 32 e is element lane % 8 of the group of lane (lane / 8 + 4 e):
    // of the eight ballots a lane needs the one of its element.
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t all = __ballot_sync(0xFFFFFFFFu, own(e));
      if ((lane & 7) == e) m = all >> (lane >> 3);
    }
    return KeepBits{m};
  }
}

}  // namespace qlora
