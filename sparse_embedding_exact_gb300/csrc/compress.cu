// Activations kept in 8 bits (kept.cuh has the format): to codes and scales, and
// back.
//
// Bound by memory: each value is read once and written once.  Four threads share
// a group of 32, eight values each (16 bytes in, 8 out), and find its largest by
// two shuffles; rows that start anywhere take a warp a group, a value a lane.
#include <algorithm>

#include "kept.cuh"
#include "tc.cuh"

namespace {

using namespace dense;

constexpr int kThreads = 256;

// A unit of a row: 8 values as the words that the loads fill, or one value.
template <typename T, int kN>
struct Unit {
  static constexpr int kWords = kN * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 q = reinterpret_cast<const uint4 *>(p)[i];
      w[4 * i] = q.x;
      w[4 * i + 1] = q.y;
      w[4 * i + 2] = q.z;
      w[4 * i + 3] = q.w;
    }
  }
  // From anywhere; zeros after `left` of the values.
  __device__ __forceinline__ void load_any(const T *p, const void *begin, const void *end, int left) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      uint32_t q[4];
      load_anywhere<16, (int)sizeof(T)>(reinterpret_cast<const uint4 *>(p) + i, begin, end, q);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[4 * i + k] = q[k];
    }
    if (left < kN) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (sizeof(T) == 4)
          w[i] = i < left ? w[i] : 0;
        else
          w[i] = 2 * i + 1 < left ? w[i] : 2 * i < left ? w[i] & 0xFFFFu : 0;
      }
    }
  }
  __device__ __forceinline__ T value(int i) const {
    const float2 f = pair(i / 2);
    return Type<T>::down(i % 2 ? f.y : f.x);
  }
  __device__ __forceinline__ void store(T *p) const {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  // Values 2 i and 2 i + 1.
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (sizeof(T) == 4) {
      return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else if constexpr (std::is_same<T, __half>::value) {
      __half2 h;
      memcpy(&h, &w[i], 4);
      return __half22float2(h);
    } else {
      return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
  }
  __device__ __forceinline__ void set_pair(int i, float2 f) {
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(f.x);
      w[2 * i + 1] = __float_as_uint(f.y);
    } else {
      w[i] = narrow2(T(), f.x, f.y);
    }
  }
  // The largest |value|, as float32 bits.  Absolute values order as the
  // integers that hold them, infinities and NaN last.
  __device__ __forceinline__ uint32_t most() const {
    if constexpr (sizeof(T) == 4) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
      return m;
    } else {
      uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
      for (int i = 1; i < kWords; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
      m = max(m >> 16, m & 0xFFFFu);
      if constexpr (std::is_same<T, __half>::value)
        return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
      else
        return m << 16;
    }
  }
};
template <typename T>
struct Unit<T, 1> {
  T v;
  __device__ __forceinline__ void clear() { v = Type<T>::down(0.0f); }
  __device__ __forceinline__ void load(const T *p) { v = *p; }
  __device__ __forceinline__ void load_any(const T *p, const void *, const void *, int) { v = *p; }
  __device__ __forceinline__ uint32_t most() const { return abs_bits(Type<T>::up(v)); }
};

// Where a thread's four units of kN values lie: kAlong of them along a row, a
// block's width apart, in each of kDown rows, a block's rows apart.  All four
// are asked for before the first is used: with one at a time too few bytes were
// under way (16,384 x 4096 bf16: 44 us to codes and 48 back).
template <int kAlong>
struct Place {
  static constexpr int kDown = 4 / kAlong;
  int64_t row;
  int32_t unit;  // of a row: fewer than 2^28
  __device__ Place()
      : row((int64_t)blockIdx.x * (blockDim.y * kDown) + threadIdx.y), unit((int32_t)(blockIdx.y * (blockDim.x * kAlong) + threadIdx.x)) {}
  __device__ __forceinline__ int64_t row_of(int down) const { return row + (int64_t)(down * (int)blockDim.y); }
  __device__ __forceinline__ int32_t unit_of(int along) const { return unit + along * (int32_t)blockDim.x; }
};

// kAny: x's rows start anywhere, or end within a unit (codes' rows start on
// 8-byte boundaries all the same).
template <typename T, int kN, int kAlong, bool kAny>
__global__ void __launch_bounds__(kThreads) k_compress(const ss_dense x, const ss_kept out, int least) {
  constexpr int kShare = kGroup / kN;  // threads of a group: neighbours in a warp
  const int32_t units = (int32_t)((x.n_cols + kN - 1) / kN);
  const Place<kAlong> at;
  const void *end = end_of(x.data, x.n_rows, x.n_cols, x.ld, sizeof(T));
  Unit<T, kN> v[4];
#pragma unroll
  for (int d = 0; d < at.kDown; ++d) {
    const bool there = at.row_of(d) < x.n_rows;
    const T *p = static_cast<const T *>(x.data) + at.row_of(d) * x.ld;
#pragma unroll
    for (int k = 0; k < kAlong; ++k) {
      v[d * kAlong + k].clear();
      if (there && at.unit_of(k) < units) {
        if (kAny)
          v[d * kAlong + k].load_any(p + (int64_t)at.unit_of(k) * kN, x.data, end, (int)min((int64_t)kN, x.n_cols - (int64_t)at.unit_of(k) * kN));
        else
          v[d * kAlong + k].load(p + (int64_t)at.unit_of(k) * kN);
      }
    }
  }
#pragma unroll
  for (int d = 0; d < at.kDown; ++d) {
    const bool there = at.row_of(d) < x.n_rows;
    uint8_t *codes = static_cast<uint8_t *>(out.codes) + at.row_of(d) * out.ld, *scale = out.scale + at.row_of(d) * out.ld_scale;
#pragma unroll
    for (int k = 0; k < kAlong; ++k) {
      const Unit<T, kN> &f = v[d * kAlong + k];
      const int32_t u = at.unit_of(k);
      uint32_t most = f.most();
      const bool odd = most >= kInfBits;  // an infinity or a NaN here: rare
      if (odd) {
        most = 0;
        if constexpr (kN == 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) most = max(most, max(finite_bits(f.pair(i).x), finite_bits(f.pair(i).y)));
      }
#pragma unroll
      for (int o = kShare / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
      const int e = exponent_of(most, least);
      const float down = power_of(-e);
      if (!there || u >= units) continue;
      if constexpr (kN == 8) {
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 g = f.pair(i);
          q[i] = codes2(g.x * down, g.y * down);
        }
        if (odd) {
#pragma unroll
          for (int i = 0; i < 4; ++i) q[i] = codes2(scaled_down(f.pair(i).x, down), scaled_down(f.pair(i).y, down));
        }
        if (kAny && (int64_t)u * kN + kN > x.n_cols) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if ((int64_t)u * kN + i < x.n_cols) codes[(int64_t)u * kN + i] = (uint8_t)(q[i / 2] >> i % 2 * 8);
        } else {
          *reinterpret_cast<uint2 *>(codes + (int64_t)u * kN) = make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
        }
      } else {
        codes[u] = (uint8_t)codes2(scaled_down(Type<T>::up(f.v), down), 0.0f);
      }
      if (u % kShare == 0) scale[u / kShare] = (uint8_t)(e + 127);
    }
  }
}

template <typename T, int kAlong>
__global__ void __launch_bounds__(kThreads) k_expand(const ss_kept x, const ss_dense y) {
  constexpr int kN = 8;
  tc::let_next();
  const int32_t units = (int32_t)(y.n_cols / kN);
  const Place<kAlong> at;
  uint2 q[4];
  uint32_t byte[4];
#pragma unroll
  for (int d = 0; d < at.kDown; ++d) {
    const uint8_t *codes = static_cast<const uint8_t *>(x.codes) + at.row_of(d) * x.ld, *scale = x.scale + at.row_of(d) * x.ld_scale;
#pragma unroll
    for (int k = 0; k < kAlong; ++k)
      if (at.row_of(d) < y.n_rows && at.unit_of(k) < units) {
        const int32_t u = at.unit_of(k);
        q[d * kAlong + k] = *reinterpret_cast<const uint2 *>(codes + (int64_t)u * kN);
        byte[d * kAlong + k] = scale[u / (kGroup / kN)];
      }
  }
#pragma unroll
  for (int d = 0; d < at.kDown; ++d) {
    T *to = static_cast<T *>(y.data) + at.row_of(d) * y.ld;
#pragma unroll
    for (int k = 0; k < kAlong; ++k) {
      const int i = d * kAlong + k;
      const int32_t u = at.unit_of(k);
      if (at.row_of(d) >= y.n_rows || u >= units) continue;
      const float s = scale_of_byte(byte[i]);
      Unit<T, 8> out;
      float2 f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 c = widen_codes2((j < 2 ? q[i].x : q[i].y) >> j % 2 * 16 & 0xFFFFu);
        f[j] = both(two(c.x, c.y) * two(s, s));
      }
      if (byte[i] > safe_byte<T>()) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = make_float2(within<T>(f[j].x), within<T>(f[j].y));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) out.set_pair(j, f[j]);
      out.store(to + (int64_t)u * kN);
    }
  }
  tc::wait_before();  // what follows waits for this kernel, and so for the one before it
}

// The same for rows that start anywhere: a thread's units of 8 values lie from
// the row's first 16-byte boundary in y on (unit 0 before it), and take their
// codes from anywhere.
template <typename T, int kAlong>
__global__ void __launch_bounds__(kThreads) k_expand_any(const ss_kept x, const ss_dense y) {
  tc::let_next();
  const Place<kAlong> at;
  const void *end = end_of(x.codes, x.n_rows, x.n_cols, x.ld, 1);
  const int32_t cols = (int32_t)y.n_cols;
#pragma unroll
  for (int d = 0; d < at.kDown; ++d) {
    if (at.row_of(d) >= y.n_rows) break;
    T *to = static_cast<T *>(y.data) + at.row_of(d) * y.ld;
    const uint8_t *codes = static_cast<const uint8_t *>(x.codes) + at.row_of(d) * x.ld, *scale = x.scale + at.row_of(d) * x.ld_scale;
    const int32_t head = (int32_t)((16 - (reinterpret_cast<uintptr_t>(to) & 15)) % 16 / sizeof(T)) - 8;
#pragma unroll
    for (int k = 0; k < kAlong; ++k) {
      const int32_t first = head + 8 * at.unit_of(k), c0 = max(first, 0), c1 = min(first + 8, cols);
      if (c0 >= c1) continue;
      uint32_t q[2];
      load_anywhere<8, 1>(codes + c0, x.codes, end, q);
      if (first < 0) {  // codes of what lies before the row are none
        const uint64_t v = ((uint64_t)q[1] << 32 | q[0]) << -8 * first;
        q[0] = (uint32_t)v;
        q[1] = (uint32_t)(v >> 32);
      }
      const uint32_t b0 = scale[c0 / kGroup], b1 = scale[(c1 - 1) / kGroup];
      const float s0 = scale_of_byte(b0), s1 = scale_of_byte(b1);
      const int32_t border = (c0 / kGroup + 1) * kGroup - first;  // values before it have s0
      Unit<T, 8> out;
      float2 f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 c = widen_codes2((j < 2 ? q[0] : q[1]) >> j % 2 * 16 & 0xFFFFu);
        f[j] = make_float2(c.x * (2 * j < border ? s0 : s1), c.y * (2 * j + 1 < border ? s0 : s1));
      }
      if (max(b0, b1) > safe_byte<T>()) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = make_float2(within<T>(f[j].x), within<T>(f[j].y));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) out.set_pair(j, f[j]);
      if (c1 - c0 == 8) {
        out.store(to + first);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (first + j >= c0 && first + j < c1) to[first + j] = out.value(j);
      }
    }
  }
  tc::wait_before();
}

// Calls run(kAlong, grid, block) for `rows` rows of `units` units; a block's
// width is a power of two of at least `least` threads, so that a group's (one
// value a thread: a warp's) threads are neighbours of one row.
template <typename F>
void laid_out(int64_t rows, int64_t units, int least, F run) {
  int64_t x = least;
  while (x < units && x < kThreads) x *= 2;
  const int64_t y = kThreads / x;
  const dim3 block((unsigned)x, (unsigned)y);
  auto grid = [&](int64_t along) {
    return dim3((unsigned)((rows + y * (4 / along) - 1) / (y * (4 / along))), (unsigned)((units + x * along - 1) / (x * along)));
  };
  if (units <= x)
    run(std::integral_constant<int, 1>(), grid(1), block);
  else if (units <= 2 * x)
    run(std::integral_constant<int, 2>(), grid(2), block);
  else
    run(std::integral_constant<int, 4>(), grid(4), block);
}
// Columns of a call, as a grid has at most 65,535 blocks that way: whole groups.
constexpr int64_t kMostCols = (int64_t)65535 * kThreads * 4;

template <typename T>
cudaError_t compress_typed(const ss_dense &x, const ss_kept &out, cudaStream_t s) {
  const int least = least_exponent(x.type);
  const bool whole = x.n_cols % 8 == 0 && rows_aligned(x, 16);
  if (kept_aligned(out, 8))
    laid_out(x.n_rows, (x.n_cols + 7) / 8, 4, [&](auto along, dim3 grid, dim3 block) {
      if (whole)
        k_compress<T, 8, decltype(along)::value, false><<<grid, block, 0, s>>>(x, out, least);
      else
        k_compress<T, 8, decltype(along)::value, true><<<grid, block, 0, s>>>(x, out, least);
    });
  else
    laid_out(x.n_rows, x.n_cols, 32, [&](auto along, dim3 grid, dim3 block) {
      k_compress<T, 1, decltype(along)::value, false><<<grid, block, 0, s>>>(x, out, least);
    });
  return cudaGetLastError();
}
template <typename T>
cudaError_t expand_typed(const ss_kept &x, const ss_dense &y, cudaStream_t s, bool beside) {
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = beside ? 1 : 0;
  cudaError_t e = cudaSuccess;
  if (y.n_cols % 8 == 0 && rows_aligned(y, 16) && kept_aligned(x, 8))
    laid_out(y.n_rows, y.n_cols / 8, 4, [&](auto along, dim3 grid, dim3 block) {
      cfg.gridDim = grid;
      cfg.blockDim = block;
      e = cudaLaunchKernelEx(&cfg, k_expand<T, decltype(along)::value>, x, y);
    });
  else
    laid_out(y.n_rows, (y.n_cols + 7) / 8 + 1, 4, [&](auto along, dim3 grid, dim3 block) {
      cfg.gridDim = grid;
      cfg.blockDim = block;
      e = cudaLaunchKernelEx(&cfg, k_expand_any<T, decltype(along)::value>, x, y);
    });
  return e;
}

}  // namespace

cudaError_t launch_compress(const ss_dense &x, const ss_kept &out, cudaStream_t s, int *queued) {
  *queued = x.n_rows > 0 && x.n_cols > 0;
  if (!*queued) return cudaSuccess;
  if (x.n_cols > kMostCols) {  // in slices: 64 million columns a row
    for (int64_t c = 0; c < x.n_cols; c += kMostCols) {
      ss_dense part = x;
      ss_kept to = out;
      part.n_cols = to.n_cols = std::min(kMostCols, x.n_cols - c);
      part.data = static_cast<unsigned char *>(x.data) + c * size_of(x.type);
      to.codes = static_cast<uint8_t *>(out.codes) + c;
      to.scale += c / kGroup;
      int one;
      const cudaError_t e = launch_compress(part, to, s, &one);
      if (e != cudaSuccess) return e;
      *queued += c > 0;
    }
    return cudaSuccess;
  }
  switch (x.type) {
    case SS_VALUES_F32: return compress_typed<float>(x, out, s);
    case SS_VALUES_BF16: return compress_typed<__nv_bfloat16>(x, out, s);
    default: return compress_typed<__half>(x, out, s);
  }
}

cudaError_t launch_expand(const ss_kept &x, const ss_dense &y, cudaStream_t s, int *queued, bool beside) {
  *queued = y.n_rows > 0 && y.n_cols > 0;
  if (!*queued) return cudaSuccess;
  if (y.n_cols > kMostCols) {
    for (int64_t c = 0; c < y.n_cols; c += kMostCols) {
      ss_dense part = y;
      ss_kept from = x;
      part.n_cols = from.n_cols = std::min(kMostCols, y.n_cols - c);
      part.data = static_cast<unsigned char *>(y.data) + c * size_of(y.type);
      from.codes = static_cast<uint8_t *>(x.codes) + c;
      from.scale += c / kGroup;
      int one;
      const cudaError_t e = launch_expand(from, part, s, &one, beside || c > 0);
      if (e != cudaSuccess) return e;
      *queued += c > 0;
    }
    return cudaSuccess;
  }
  switch (y.type) {
    case SS_VALUES_F32: return expand_typed<float>(x, y, s, beside);
    case SS_VALUES_BF16: return expand_typed<__nv_bfloat16>(x, y, s, beside);
    default: return expand_typed<__half>(x, y, s, beside);
  }
}
