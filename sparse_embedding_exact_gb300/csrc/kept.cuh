// Values kept in 8 bits: e4m3 codes with a power of two for every 32 of a row.
//
//   e = the smallest with max|x| <= 448 2^e over the group's finite values, and
//       not below the type's least
//   code = x 2^-e to the nearest e4m3 (ties to even),  value = code 2^e
//
// The scale's byte is e + 127.  A power of two makes the value exact in the
// type it came from (the least exponent keeps its smallest codes above that
// type's smallest value), so that nothing is rounded a second time, and 32
// values are what one thread of a product's epilogue holds.  An infinity or a
// NaN becomes NaN and leaves its group's other values as they are.
#pragma once

#include "dense.cuh"

namespace dense {

constexpr int kGroup = SS_KEPT_GROUP;

// Exponents from which code 2^e is a value of the type: e4m3's smallest is 2^-9.
__host__ __device__ constexpr int least_exponent(int32_t type) {
  return type == SS_VALUES_F32 ? -126 : type == SS_VALUES_BF16 ? -124 : -15;
}
constexpr uint32_t kInfBits = 0x7F800000u;
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t u = abs_bits(v);
  return u < kInfBits ? u : 0u;
}
// e of a group whose largest finite |x| has these bits: 448 = 1.75 2^8.
__device__ __forceinline__ int exponent_of(uint32_t most, int least) {
  return max(least, (int)(most >> 23) - 135 + ((most & 0x7FFFFFu) > 0x600000u ? 1 : 0));
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float power_of(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// The scale that a byte holds: 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float scale_of_byte(uint32_t b) {
  return __uint_as_float(b == 255 ? 0x7FC00000u : b == 0 ? 0x00400000u : b << 23);
}
// Two codes (the first in the low byte); infinities have been made NaN.
__device__ __forceinline__ uint32_t codes2(float x, float y) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 widen_codes2(uint32_t two) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)));
}
__device__ __forceinline__ float widen_code(uint8_t c) { return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3))); }
// x 2^-e with infinities made NaN.
__device__ __forceinline__ float scaled_down(float x, float down) {
  return abs_bits(x) == kInfBits ? __uint_as_float(0x7FC00000u) : x * down;
}

// A type's largest value: what stands for more becomes that.
template <typename T>
__device__ __forceinline__ constexpr float largest() {
  return sizeof(T) == 4 ? 3.40282347e38f : std::is_same<T, __half>::value ? 65504.0f : 3.38953139e38f;
}
template <typename T>
__device__ __forceinline__ float within(float v) {
  return v > largest<T>() ? largest<T>() : v < -largest<T>() ? -largest<T>() : v;
}
// Bytes of scales up to which no code reaches beyond the type: 448 2^e = 1.75 2^(e + 8).
template <typename T>
__device__ __forceinline__ constexpr uint32_t safe_byte() {
  return std::is_same<T, __half>::value ? 127 + 6 : 127 + 118;
}

// Of these bytes every code stands for a value of the type: none is beyond its
// largest, or between two of its smallest.
template <typename T>
__device__ __forceinline__ constexpr bool exact_byte(uint32_t b) {
  constexpr uint32_t low = sizeof(T) == 4 ? 0 : 127 + least_exponent(std::is_same<T, __half>::value ? SS_VALUES_F16 : SS_VALUES_BF16);
  return b - low <= safe_byte<T>() - low;
}
// What a kept value is to the gradients: the type's nearest, as expand has it.
// Only of a scale that is not exact_byte is that another value.
template <typename T>
__device__ __forceinline__ float as_type(float v) {
  return Type<T>::up(Type<T>::down(within<T>(v)));
}

// kN codes of a row (8, 4 or 1) as a load leaves them.
template <int kN>
struct Codes {
  static_assert(kN == 8 || kN == 4 || kN == 1, "codes of one load");
  uint32_t w[(kN + 3) / 4];
  __device__ __forceinline__ void load(const uint8_t *p) {
    if constexpr (kN == 8) {
      const uint2 q = *reinterpret_cast<const uint2 *>(p);
      w[0] = q.x;
      w[1] = q.y;
    } else if constexpr (kN == 4) {
      w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
      w[0] = *p;
    }
  }
  __device__ __forceinline__ void load_shared(uint32_t at) {
    if constexpr (kN == 8)
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
    else
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
  }
  // Codes 2 i and 2 i + 1.
  __device__ __forceinline__ float2 pair(int i) const { return widen_codes2(w[i / 2] >> i % 2 * 16 & 0xFFFFu); }
  __device__ __forceinline__ float one() const { return widen_code((uint8_t)w[0]); }
};
inline bool kept_aligned(const ss_kept &m, int64_t unit) {
  return reinterpret_cast<uintptr_t>(m.codes) % (uintptr_t)unit == 0 && (m.n_rows <= 1 || m.ld % unit == 0);
}

}  // namespace dense
