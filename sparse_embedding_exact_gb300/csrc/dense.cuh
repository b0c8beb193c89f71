// Shared by the dense operators (rmsnorm.cu, linear.cu, distill.cu): value
// types, vector loads and stores, reductions, and the launchers the ABI calls.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

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
// kBytes (16 or 8) bytes at p, which may lie anywhere that holds the values of
// kSize bytes whole: from the aligned units that hold them where these lie within
// [begin, end), the memory of the whole matrix; else value by value, zeros from
// `end` on.
template <int kBytes, int kSize>
__device__ __forceinline__ void load_anywhere(const void *at, const void *begin, const void *end, uint32_t (&v)[kBytes / 4]) {
  const unsigned char *p = static_cast<const unsigned char *>(at);
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & (kBytes - 1)), bits = 8 * (off & 3);
  if (p - off >= begin && p - off + 2 * kBytes <= end) {
    constexpr int kW = kBytes / 4;
    uint32_t w[2 * kW];
    if constexpr (kBytes == 16) {
      const uint4 a = *reinterpret_cast<const uint4 *>(p - off), b = *reinterpret_cast<const uint4 *>(p - off + 16);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
      const uint2 a = *reinterpret_cast<const uint2 *>(p - off), b = *reinterpret_cast<const uint2 *>(p - off + 8);
      w[0] = a.x, w[1] = a.y, w[2] = b.x, w[3] = b.y;
    }
    auto from = [&](auto first) {
      constexpr int k = decltype(first)::value;
#pragma unroll
      for (int i = 0; i < kW; ++i) v[i] = __funnelshift_r(w[k + i], w[(k + i + 1) % (2 * kW)], bits);
    };
    switch (off >> 2) {  // the same for the threads of a row
      case 0: from(std::integral_constant<int, 0>()); break;
      case 1: from(std::integral_constant<int, 1>()); break;
      case 2: from(std::integral_constant<int, kBytes == 16 ? 2 : 0>()); break;
      default: from(std::integral_constant<int, kBytes == 16 ? 3 : 1>()); break;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i) v[i] = 0;
#pragma unroll
    for (int i = 0; i < kBytes; i += kSize) {
      uint32_t x = 0;
      if (p + i + kSize <= end) {
        if constexpr (kSize == 1)
          x = p[i];
        else if constexpr (kSize == 2)
          x = *reinterpret_cast<const uint16_t *>(p + i);
        else
          x = *reinterpret_cast<const uint32_t *>(p + i);
      }
      v[i / 4] |= x << i % 4 * 8;
    }
  }
}
// The end of a matrix's memory.
__device__ __forceinline__ const void *end_of(const void *data, int64_t rows, int64_t cols, int64_t ld, int size) {
  return static_cast<const unsigned char *>(data) + ((rows - 1) * ld + cols) * size;
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
  float *scratch;      // rms_grad_scratch bytes
  ss_kept total_kept;  // in total's place (which keeps its sizes and type, with null data), or null codes
};
int64_t rms_grad_scratch(const ss_handle *h, int64_t rows, int64_t cols);
int64_t rms_kept_grad_scratch(const ss_handle *h, int64_t rows, int64_t cols, int32_t type);
cudaError_t launch_rms_norm_grad(ss_handle *h, const rms_grad_args &a, cudaStream_t s, int *queued);

// Values to codes and scales, and back (kept.cuh).
cudaError_t launch_compress(const ss_dense &x, const ss_kept &out, cudaStream_t s, int *queued);
// beside: at the end of the kernel before, which is of the same call.
cudaError_t launch_expand(const ss_kept &x, const ss_dense &y, cudaStream_t s, int *queued, bool beside = false);

// out[c] = the sum of column c over the n rows of part (one kernel; a fixed
// order), rounded to `type`; beside: at the end of the kernel before, which is of
// the same call.
cudaError_t launch_sum_rows(const ss_handle *h, const float *part, int64_t n, int64_t cols, void *out, int32_t type, cudaStream_t s,
                            bool beside = false);

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
  ss_kept keep;            // in pre's place, or null codes
};
int64_t linear_scratch(const ss_handle *h, const ss_dense &x, const ss_dense &w, bool keep);
cudaError_t launch_linear(ss_handle *h, const linear_args &a, cudaStream_t s, int *queued);

struct linear_grad_args {
  ss_dense grad_y, x, w, pre, grad_x, grad_w;  // grad_x, grad_w: or null
  float *grad_bias;                            // or null
  int32_t activation;
  unsigned char *scratch;    // linear_grad_scratch bytes
  ss_kept x_kept, pre_kept;  // in x's and pre's place (x keeps its sizes and type, with null data), or null codes
};
int64_t linear_grad_scratch(const ss_handle *h, const ss_dense &grad_y, const ss_dense &x, const ss_dense &w,
                            int32_t activation, bool x_kept);
cudaError_t launch_linear_grad(ss_handle *h, const linear_grad_args &a, cudaStream_t s, int *queued);

// Each matrix itself, or its copy with padded rows at *scratch (advanced past
// it, copy_bytes of each); `other` may be null.
cudaError_t launch_aligned_rows(ss_handle *h, ss_dense *m, ss_dense *other, unsigned char **scratch, cudaStream_t s, int *queued);

// A layer's two gradient products in one launch, all matrices of 16 bits with
// 16-byte aligned rows:
//   grad_x (+)= diag(row_factor) gz wide  and  grad_w = factor gz^T x
// grad_x may come in several calls (`begun`: an earlier one added to acc;
// `ends`: grad_x is written), each of another gz and wide of the same sizes or
// less.  Its sum is split over `parts` (grad_product_parts of the largest gz)
// shares of the summed dimension, each in its own float32 matrix of acc
// (grad_part_bytes each; none is needed for one part in one call).
struct grad_products {
  ss_dense gz, wide, x;     // [M][N], [N][K], [M][K]
  ss_dense grad_x, grad_w;  // [M][K], [N][K], of x's type or float32, or null data
  float *acc;
  const float *factor;  // device float or null: 1
  int32_t parts;
  bool begun, ends;
  bool beside;  // the kernel before is of the same call
  // with it, sum_to[c] = the sum of column c of sums[sum_rows][sum_cols], or null
  const float *sums;
  int64_t sum_rows, sum_cols;
  float *sum_to;
  const float *row_factor;  // float r row_step of it for row r, or null: 1
  int32_t row_step;
};
int64_t grad_product_parts(const ss_handle *h, int64_t M, int64_t N, int64_t K, int64_t *clocks = nullptr);
int64_t grad_part_bytes(int64_t M, int64_t K);
cudaError_t launch_grad_products(ss_handle *h, const grad_products &g, cudaStream_t s, int *queued);

struct xent_args {
  ss_dense x, w, grad_x, grad_w;  // grad_x, grad_w: or null
  const float *bias;              // [items] or null
  const int64_t *targets;         // [rows]
  const float *weight;            // [rows] or null: 1
  const float *grad_loss;         // [rows] or null: 1
  float *loss;                    // [rows]
  float *stats;                   // [rows][2]: {largest logit, sum of exp((logit - it) / T)}
  float *grad_bias;               // [items] or null
  float temperature;
  unsigned char *scratch;  // xent_scratch bytes
};
enum : int32_t { XENT_LOSS = 0, XENT_BACKWARD = 1, XENT_STEP = 2 };
int64_t xent_scratch(const ss_handle *h, const ss_dense &x, const ss_dense &w, int32_t mode);
cudaError_t launch_xent(ss_handle *h, const xent_args &a, int32_t mode, cudaStream_t s, int *queued);
