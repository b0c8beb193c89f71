// Activations kept in 8 bits (kept.cuh has the format): to codes and scales, and
// back.
//
// Bound by memory: each value is read once and written once.  Four threads share
// a group of 32, eight values each (16 bytes in, 8 out), and find its largest by
// two shuffles; rows that start anywhere take a warp a group, a value a lane.
#include <algorithm>

#include "kept.cuh"

namespace {

using namespace dense;

constexpr int kThreads = 256;

template <typename T, int kN>
__device__ __forceinline__ void load_values(const T *p, float (&f)[kN]) {
  if constexpr (sizeof(T) == 4 && kN == 8) {
    float a[4], b[4];
    widen(load_pack<T, 4>(p), a);
    widen(load_pack<T, 4>(p + 4), b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i];
      f[4 + i] = b[i];
    }
  } else {
    widen(load_pack<T, kN>(p), f);
  }
}
// Values to T, beyond its largest to that.
template <typename T>
__device__ __forceinline__ constexpr float largest() {
  return sizeof(T) == 4 ? 3.40282347e38f : std::is_same<T, __half>::value ? 65504.0f : 3.38953139e38f;
}
template <typename T, int kN>
__device__ __forceinline__ void store_values(T *p, float (&f)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) f[i] = f[i] > largest<T>() ? largest<T>() : f[i] < -largest<T>() ? -largest<T>() : f[i];
  if constexpr (sizeof(T) == 4 && kN == 8) {
    float a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = f[i];
      b[i] = f[4 + i];
    }
    store_pack(p, narrow<T, 4>(a));
    store_pack(p + 4, narrow<T, 4>(b));
  } else {
    store_pack(p, narrow<T, kN>(f));
  }
}

// Blocks of blockDim.x threads along a row and blockDim.y rows.
template <typename T, int kN>
__global__ void __launch_bounds__(kThreads) k_compress(const ss_dense x, const ss_kept out, int least) {
  constexpr int kShare = kGroup / kN;  // threads of a group
  const int64_t units = (x.n_cols + kN - 1) / kN;
  const int64_t padded = (units + kShare - 1) / kShare * kShare;  // every thread of a warp takes part in its shuffles
  for (int64_t row0 = (int64_t)blockIdx.x * blockDim.y; row0 < x.n_rows; row0 += (int64_t)gridDim.x * blockDim.y) {
    const int64_t row = row0 + threadIdx.y;
    for (int64_t u0 = 0; u0 < padded; u0 += blockDim.x) {
      const int64_t u = u0 + threadIdx.x;
      const bool in = row < x.n_rows && u < units;
      float f[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) f[i] = 0.0f;
      if (in) load_values<T, kN>(static_cast<const T *>(x.data) + row * x.ld + u * kN, f);
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < kN; ++i) most = max(most, finite_bits(f[i]));
#pragma unroll
      for (int o = kShare / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
      const int e = exponent_of(most, least);
      const float down = power_of(-e);
      if (!in) continue;
      uint8_t *to = static_cast<uint8_t *>(out.codes) + row * out.ld + u * kN;
#pragma unroll
      for (int i = 0; i < kN; ++i) f[i] = scaled_down(f[i], down);
      if constexpr (kN == 8) {
        uint2 q;
        q.x = codes2(f[0], f[1]) | codes2(f[2], f[3]) << 16;
        q.y = codes2(f[4], f[5]) | codes2(f[6], f[7]) << 16;
        *reinterpret_cast<uint2 *>(to) = q;
      } else {
        *to = (uint8_t)codes2(f[0], 0.0f);
      }
      if (u % kShare == 0) out.scale[row * out.ld_scale + u / kShare] = (uint8_t)(e + 127);
    }
  }
}

template <typename T, int kN>
__global__ void __launch_bounds__(kThreads) k_expand(const ss_kept x, const ss_dense y) {
  const int64_t units = (y.n_cols + kN - 1) / kN;
  for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < y.n_rows; row += (int64_t)gridDim.x * blockDim.y)
    for (int64_t u = threadIdx.x; u < units; u += blockDim.x) {
      float f[kN];
      load_kept<kN>(x, row, u * kN, f);
      store_values<T, kN>(static_cast<T *>(y.data) + row * y.ld + u * kN, f);
    }
}

// The threads along a row (a power of two, whole groups and, one value a
// thread, whole warps) and the rows of a block.
dim3 block_for(int64_t units, int least) {
  int64_t x = least;
  while (x < units && x < kThreads) x *= 2;
  return dim3((unsigned)x, (unsigned)(kThreads / x));
}
unsigned blocks_for(int64_t rows, const dim3 &block) {
  return (unsigned)std::min<int64_t>((rows + block.y - 1) / block.y, (int64_t)1 << 30);
}

template <typename T>
cudaError_t compress_typed(const ss_dense &x, const ss_kept &out, cudaStream_t s) {
  const int least = least_exponent(x.type);
  if (x.n_cols % 8 == 0 && rows_aligned(x, 16) && kept_aligned(out, 8)) {
    const dim3 block = block_for(x.n_cols / 8, 4);
    k_compress<T, 8><<<blocks_for(x.n_rows, block), block, 0, s>>>(x, out, least);
  } else {
    const dim3 block = block_for(x.n_cols, 32);
    k_compress<T, 1><<<blocks_for(x.n_rows, block), block, 0, s>>>(x, out, least);
  }
  return cudaGetLastError();
}
template <typename T>
cudaError_t expand_typed(const ss_kept &x, const ss_dense &y, cudaStream_t s) {
  if (y.n_cols % 8 == 0 && rows_aligned(y, 16) && kept_aligned(x, 8)) {
    const dim3 block = block_for(y.n_cols / 8, 4);
    k_expand<T, 8><<<blocks_for(y.n_rows, block), block, 0, s>>>(x, y);
  } else {
    const dim3 block = block_for(y.n_cols, 32);
    k_expand<T, 1><<<blocks_for(y.n_rows, block), block, 0, s>>>(x, y);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_compress(const ss_dense &x, const ss_kept &out, cudaStream_t s, int *queued) {
  *queued = x.n_rows > 0 && x.n_cols > 0;
  if (!*queued) return cudaSuccess;
  switch (x.type) {
    case SS_VALUES_F32: return compress_typed<float>(x, out, s);
    case SS_VALUES_BF16: return compress_typed<__nv_bfloat16>(x, out, s);
    default: return compress_typed<__half>(x, out, s);
  }
}

cudaError_t launch_expand(const ss_kept &x, const ss_dense &y, cudaStream_t s, int *queued) {
  *queued = y.n_rows > 0 && y.n_cols > 0;
  if (!*queued) return cudaSuccess;
  switch (y.type) {
    case SS_VALUES_F32: return expand_typed<float>(x, y, s);
    case SS_VALUES_BF16: return expand_typed<__nv_bfloat16>(x, y, s);
    default: return expand_typed<__half>(x, y, s);
  }
}
