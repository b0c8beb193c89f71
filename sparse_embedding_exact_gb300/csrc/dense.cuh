// Shared by the dense operators (rmsnorm.cu, linear.cu, distill.cu): value
// types, vector loads and stores, reductions, and the launchers the ABI calls.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "internal.cuh"

namespace dense {

constexpr float kF8Max = 448.0f;  // largest finite e4m3 value

// ---------------------------------------------------------------- values
template <typename T>
struct Type;
template <>
struct Type<float> {
  static constexpr int kVec = 4;  // values in 16 bytes
  static __device__ __forceinline__ float up(float v) { return v; }
  static __device__ __forceinline__ float down(float v) { return v; }
};
template <>
struct Type<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float up(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Type<__half> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float up(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half down(float v) { return __float2half_rn(v); }
};

// kN consecutive values read as one access of kN * sizeof(T) bytes, and their
// float32 values.
template <typename T, int kN>
struct alignas(sizeof(T) * kN) Pack {
  T v[kN];
};
// Eight 16-bit values stay in the words that a load fills and a conversion of
// two values makes: taken apart into halves they cost the norm's gradient
// three times its instructions.
template <>
struct alignas(16) Pack<__nv_bfloat16, 8> {
  uint32_t w[4];
};
template <>
struct alignas(16) Pack<__half, 8> {
  uint32_t w[4];
};
template <typename T, int kN>
__device__ __forceinline__ T item(const Pack<T, kN> &p, int i) {
  if constexpr (kN == 8) {
    const uint16_t h = (uint16_t)(p.w[i / 2] >> i % 2 * 16);
    T v;
    memcpy(&v, &h, 2);
    return v;
  } else {
    return p.v[i];
  }
}
// Value i set to 0.
template <typename T, int kN>
__device__ __forceinline__ void clear_item(Pack<T, kN> &p, int i) {
  if constexpr (kN == 8)
    p.w[i / 2] &= i % 2 ? 0x0000FFFFu : 0xFFFF0000u;
  else
    p.v[i] = Type<T>::down(0.0f);
}
__device__ __forceinline__ float2 widen2(const Pack<__nv_bfloat16, 8> &p, int i) {
  return make_float2(__uint_as_float(p.w[i] << 16), __uint_as_float(p.w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ float2 widen2(const Pack<__half, 8> &p, int i) {
  __half2 h;
  memcpy(&h, &p.w[i], 4);
  return __half22float2(h);
}
template <typename T, int kN>
__device__ __forceinline__ void widen(const Pack<T, kN> &p, float (&f)[kN]) {
  if constexpr (kN == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q = widen2(p, i);
      f[2 * i] = q.x;
      f[2 * i + 1] = q.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = Type<T>::up(p.v[i]);
  }
}
// Each value rounded once, to the nearest (ties to even).
__device__ __forceinline__ uint32_t narrow2(__nv_bfloat16, float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}
__device__ __forceinline__ uint32_t narrow2(__half, float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}
template <typename T, int kN>
__device__ __forceinline__ Pack<T, kN> narrow(const float (&f)[kN]) {
  Pack<T, kN> p;
  if constexpr (kN == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p.w[i] = narrow2(T(), f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) p.v[i] = Type<T>::down(f[i]);
  }
  return p;
}
template <typename T, int kN>
__device__ __forceinline__ Pack<T, kN> load_pack(const T *p) {
  return *reinterpret_cast<const Pack<T, kN> *>(p);
}
template <typename T, int kN>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, kN> &v) {
  *reinterpret_cast<Pack<T, kN> *>(p) = v;
}
// kN values rounded to e4m3 (to the nearest, beyond 448 to 448; NaN kept).
template <int kN>
__device__ __forceinline__ void store_f8(uint8_t *p, const float (&f)[kN]) {
  if constexpr (kN == 1) {
    *p = (uint8_t)__nv_cvt_float_to_fp8(f[0], __NV_SATFINITE, __NV_E4M3);
  } else {
    Pack<uint16_t, kN / 2> q;
#pragma unroll
    for (int i = 0; i < kN / 2; ++i)
      q.v[i] = (uint16_t)__nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<Pack<uint16_t, kN / 2> *>(p) = q;
  }
}

// Two float32 values in one register pair: one instruction for both.
struct Two {
  unsigned long long v;
};
__device__ __forceinline__ Two two(float x, float y) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 both(Two a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma_of(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Values 2 i and 2 i + 1 of a vector.
__device__ __forceinline__ Two pair_of(const Pack<float, 4> &p, int i) { return two(p.v[2 * i], p.v[2 * i + 1]); }
template <typename T>
__device__ __forceinline__ Two pair_of(const Pack<T, 8> &p, int i) {
  const float2 f = widen2(p, i);
  return two(f.x, f.y);
}
// The larger of two values, NaN when either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

__device__ __forceinline__ void flag(int32_t *status, int32_t code) { atomicCAS(status, DEV_OK, code); }

inline int64_t size_of(int32_t type) {
  return type == SS_VALUES_F32 ? 4 : type == SS_VALUES_F8 ? 1 : 2;
}
// Whether the rows of m can be read in aligned units of `unit` bytes.
inline bool rows_aligned(const ss_dense &m, int64_t unit) {
  return (reinterpret_cast<uintptr_t>(m.data) % (uintptr_t)unit) == 0 &&
         (m.n_rows <= 1 || (m.ld * size_of(m.type)) % unit == 0);
}

}  // namespace dense

// Launchers (all asynchronous on `s`; *queued gets the kernels queued).  The
// matrices have been checked; absent ones have a null data pointer.
struct rms_args {
  ss_dense x, residual, weight, total, y;
  float *scale;  // with y in 8 bits: one scale a row
  float *rstd;   // or null
  float eps;
};
cudaError_t launch_rms_norm(ss_handle *h, const rms_args &a, cudaStream_t s, int *queued);

struct rms_grad_args {
  ss_dense grad_y, total, weight, grad_total, grad_x, grad_weight;
  const float *rstd;
  float *scratch;  // rms_grad_scratch bytes
};
int64_t rms_grad_scratch(const ss_handle *h, int64_t rows, int64_t cols);
cudaError_t launch_rms_norm_grad(ss_handle *h, const rms_grad_args &a, cudaStream_t s, int *queued);

// out[c] = the sum of column c over the n rows of part (one kernel; a fixed
// order), rounded to `type`.
cudaError_t launch_sum_rows(const ss_handle *h, const float *part, int64_t n, int64_t cols, void *out, int32_t type, cudaStream_t s);

struct distill_args {
  ss_dense logits, grad_logits;
  const float *scores;   // [rows][k]
  const int64_t *items;  // [rows][k]
  int32_t k;
  float temperature, teacher_temperature;
  const float *weight;     // [rows] or null: 1
  const float *grad_loss;  // [rows] or null: 1
  float *loss;             // [rows]
  float *stats;            // [rows][2]: {max, sum of exp((z - max) / T)}
};
enum : int32_t { DISTILL_FORWARD = 0, DISTILL_BACKWARD = 1, DISTILL_STEP = 2 };
cudaError_t launch_distill(ss_handle *h, const distill_args &a, int32_t mode, cudaStream_t s, int *queued);

struct linear_args {
  ss_dense x, w, residual, pre, y;
  const float *x_scale, *w_scale, *bias;
  int32_t activation;
  unsigned char *scratch;  // linear_scratch bytes
};
int64_t linear_scratch(const ss_handle *h, const ss_dense &x, const ss_dense &w);
cudaError_t launch_linear(ss_handle *h, const linear_args &a, cudaStream_t s, int *queued);

struct linear_grad_args {
  ss_dense grad_y, x, w, pre, grad_x, grad_w;  // grad_x, grad_w: or null
  float *grad_bias;                            // or null
  int32_t activation;
  unsigned char *scratch;  // linear_grad_scratch bytes
};
int64_t linear_grad_scratch(const ss_handle *h, const ss_dense &grad_y, const ss_dense &x, const ss_dense &w,
                            int32_t activation);
cudaError_t launch_linear_grad(ss_handle *h, const linear_grad_args &a, cudaStream_t s, int *queued);
