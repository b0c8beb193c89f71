// Root-mean-square norm with the residual's addition, and its gradient.
//
//   s = x + r,  rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w
//
// over each row, in float32, each output rounded once.  With y in 8 bits
// (e4m3) a row has one scale: scale = max|y| / 448 and y / scale is what is
// rounded.  rstd cancels there, y / scale = 448 s w / max|s w|, so the sum of
// squares and the maximum of |s w| are one reduction, and a row is read once.
//
// Gradient, with xh = s rstd and g = grad_y w:
//   grad_x = rstd (g - xh mean(g xh)) + grad_s,   grad_w = sum_rows grad_y xh
//
// Both are bound by memory: every value is read once, held in registers
// across the row's reduction, and written once.  A block takes a row at a
// time, every thread the same columns of each row, so the weights (and the
// gradient's sums over rows) stay in registers; the next row is loaded before
// the current row's reduction, which hides the reduction's barrier.  The sums
// over a block's rows go to scratch, one row of it a block, and a second
// kernel adds them in a fixed order: no atomics, the same bits every time.
#include <algorithm>

#include "dense.cuh"

namespace {

using namespace dense;

constexpr int kWideThreads = 1024;
constexpr int kMostThreads = 512;  // of a block that holds its row in registers (up to 128 a thread)

// Sum of a and maximum of b over the block, in every thread.  `sm` holds two
// sets of 32 pairs; consecutive calls alternate `set`, so that one barrier a
// call is enough.
__device__ __forceinline__ float2 block_sum_max(float a, float b, float2 (*sm)[32], int set) {
  a = warp_sum(a);
  b = warp_max_nan(b);
  const int n_warps = blockDim.x >> 5;
  if (n_warps == 1) return make_float2(a, b);
  const int lane = threadIdx.x & 31;
  if (lane == 0) sm[set][threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < n_warps ? sm[set][lane] : make_float2(0.0f, 0.0f);
  return make_float2(warp_sum(v.x), warp_max_nan(v.y));
}

template <int kN>
__device__ __forceinline__ void load_weights(const ss_dense &w, int64_t c, float (&f)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i)
    f[i] = w.type == SS_VALUES_F32    ? static_cast<const float *>(w.data)[c + i]
           : w.type == SS_VALUES_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(w.data)[c + i])
                                      : __half2float(static_cast<const __half *>(w.data)[c + i]);
}

// The factor that brings a row's s w to e4m3's range: q = (s w pre) mul.  Rows
// below 1e-30 are scaled up first, as 448 / max would overflow.
__device__ __forceinline__ float2 f8_factors(float most) {
  const float pre = most < 1e-30f ? 0x1p100f : 1.0f;
  return make_float2(pre, most > 0.0f ? kF8Max / (most * pre) : (most == 0.0f ? 0.0f : most));
}

// kN values a vector (16 bytes of them, or 1), kPer vectors a thread: columns
// (p * blockDim.x + tid) * kN + i.
template <typename T, bool kF8, int kN, int kPer>
__global__ void __launch_bounds__(kMostThreads) k_rms_norm(const rms_args a) {
  __shared__ float2 sm[2][32];
  const int64_t D = a.x.n_cols, R = a.x.n_rows;
  const T *x = static_cast<const T *>(a.x.data), *r = static_cast<const T *>(a.residual.data);
  T *total = static_cast<T *>(a.total.data);
  float w[kPer][kN];
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * kN;
    if (c < D) load_weights<kN>(a.weight, c, w[p]);
  }
  Pack<T, kN> xv[kPer], rv[kPer];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * kN;
      if (c < D) {
        xv[p] = load_pack<T, kN>(x + row * a.x.ld + c);
        if (r) rv[p] = load_pack<T, kN>(r + row * a.residual.ld + c);
      }
    }
  };
  int set = 0;
  if (blockIdx.x < R) fetch(blockIdx.x);
  for (int64_t row = blockIdx.x; row < R; row += gridDim.x, set ^= 1) {
    float s[kPer][kN], sq = 0.0f, most = 0.0f;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * kN;
      if (c < D) {
        widen(xv[p], s[p]);
        if (r) {
          float f[kN];
          widen(rv[p], f);
#pragma unroll
          for (int i = 0; i < kN; ++i) s[p][i] += f[i];
          if (total) store_pack(total + row * a.total.ld + c, narrow<T, kN>(s[p]));
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          sq = fmaf(s[p][i], s[p][i], sq);
          if (kF8) most = max_nan(most, fabsf(s[p][i] * w[p][i]));
        }
      }
    }
    if (row + gridDim.x < R) fetch(row + gridDim.x);
    const float2 red = block_sum_max(sq, most, sm, set);
    const float rstd = 1.0f / sqrtf(red.x / (float)D + a.eps);
    if (threadIdx.x == 0) {
      if (a.rstd) a.rstd[row] = rstd;
      if (kF8) a.scale[row] = red.y * rstd / kF8Max;
    }
    const float2 to8 = f8_factors(red.y);
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * kN;
      if (c < D) {
        float y[kN];
        if (kF8) {
#pragma unroll
          for (int i = 0; i < kN; ++i) y[i] = s[p][i] * w[p][i] * to8.x * to8.y;
          store_f8<kN>(static_cast<uint8_t *>(a.y.data) + row * a.y.ld + c, y);
        } else {
#pragma unroll
          for (int i = 0; i < kN; ++i) y[i] = s[p][i] * rstd * w[p][i];
          store_pack(static_cast<T *>(a.y.data) + row * a.y.ld + c, narrow<T, kN>(y));
        }
      }
    }
  }
}

// Rows too wide for registers: the row is read twice, the second time from
// L2.
template <typename T, bool kF8, int kN>
__global__ void __launch_bounds__(kWideThreads) k_rms_norm_wide(const rms_args a) {
  __shared__ float2 sm[2][32];
  const int64_t D = a.x.n_cols, R = a.x.n_rows;
  const T *x = static_cast<const T *>(a.x.data), *r = static_cast<const T *>(a.residual.data);
  T *total = static_cast<T *>(a.total.data);
  int set = 0;
  for (int64_t row = blockIdx.x; row < R; row += gridDim.x, set ^= 1) {
    auto values = [&](int64_t c, float (&s)[kN]) {
      widen(load_pack<T, kN>(x + row * a.x.ld + c), s);
      if (r) {
        float f[kN];
        widen(load_pack<T, kN>(r + row * a.residual.ld + c), f);
#pragma unroll
        for (int i = 0; i < kN; ++i) s[i] += f[i];
      }
    };
    float sq = 0.0f, most = 0.0f;
    for (int64_t c = (int64_t)threadIdx.x * kN; c < D; c += (int64_t)blockDim.x * kN) {
      float s[kN], w[kN];
      values(c, s);
      if (kF8) load_weights<kN>(a.weight, c, w);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        sq = fmaf(s[i], s[i], sq);
        if (kF8) most = max_nan(most, fabsf(s[i] * w[i]));
      }
    }
    const float2 red = block_sum_max(sq, most, sm, set);
    const float rstd = 1.0f / sqrtf(red.x / (float)D + a.eps);
    if (threadIdx.x == 0) {
      if (a.rstd) a.rstd[row] = rstd;
      if (kF8) a.scale[row] = red.y * rstd / kF8Max;
    }
    const float2 to8 = f8_factors(red.y);
    for (int64_t c = (int64_t)threadIdx.x * kN; c < D; c += (int64_t)blockDim.x * kN) {
      float s[kN], w[kN], y[kN];
      values(c, s);
      load_weights<kN>(a.weight, c, w);
#pragma unroll
      for (int i = 0; i < kN; ++i) y[i] = kF8 ? s[i] * w[i] * to8.x * to8.y : s[i] * rstd * w[i];
      if (kF8)
        store_f8<kN>(static_cast<uint8_t *>(a.y.data) + row * a.y.ld + c, y);
      else
        store_pack(static_cast<T *>(a.y.data) + row * a.y.ld + c, narrow<T, kN>(y));
      // in the second pass, by the thread that has read x and r there: total may be either
      if (r && total) store_pack(total + row * a.total.ld + c, narrow<T, kN>(s));
    }
  }
}

// grad_x of the block's rows, and the block's part of grad_w into
// scratch[blockIdx.x][D].
template <typename T, int kN, int kPer>
__global__ void __launch_bounds__(kMostThreads) k_rms_grad(const rms_grad_args a) {
  __shared__ float2 sm[2][32];
  const int64_t D = a.total.n_cols, R = a.total.n_rows;
  const T *gy = static_cast<const T *>(a.grad_y.data), *x = static_cast<const T *>(a.total.data);
  const T *gt = static_cast<const T *>(a.grad_total.data);
  float w[kPer][kN], gw[kPer][kN];
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * kN;
    if (c < D) load_weights<kN>(a.weight, c, w[p]);
#pragma unroll
    for (int i = 0; i < kN; ++i) gw[p][i] = 0.0f;
  }
  Pack<T, kN> gv[kPer], xv[kPer], tv[kPer];
  float rstd_next = 0.0f;
  auto fetch = [&](int64_t row) {
    rstd_next = a.rstd[row];
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * kN;
      if (c < D) {
        gv[p] = load_pack<T, kN>(gy + row * a.grad_y.ld + c);
        xv[p] = load_pack<T, kN>(x + row * a.total.ld + c);
        if (gt) tv[p] = load_pack<T, kN>(gt + row * a.grad_total.ld + c);
      }
    }
  };
  int set = 0;
  if (blockIdx.x < R) fetch(blockIdx.x);
  for (int64_t row = blockIdx.x; row < R; row += gridDim.x, set ^= 1) {
    float g[kPer][kN], xh[kPer][kN], t[kPer][kN], dot = 0.0f;
    const float rstd = rstd_next;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * kN;
      if (c < D) {
        widen(gv[p], g[p]);
        widen(xv[p], xh[p]);
        if (gt) widen(tv[p], t[p]);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          xh[p][i] *= rstd;
          gw[p][i] = fmaf(g[p][i], xh[p][i], gw[p][i]);
          g[p][i] *= w[p][i];
          dot = fmaf(g[p][i], xh[p][i], dot);
        }
      }
    }
    if (row + gridDim.x < R) fetch(row + gridDim.x);
    const float mean = block_sum_max(dot, 0.0f, sm, set).x / (float)D;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * kN;
      if (c < D) {
        float y[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          y[i] = rstd * (g[p][i] - xh[p][i] * mean);
          if (gt) y[i] += t[p][i];
        }
        store_pack(static_cast<T *>(a.grad_x.data) + row * a.grad_x.ld + c, narrow<T, kN>(y));
      }
    }
  }
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int64_t c = ((int64_t)p * blockDim.x + threadIdx.x) * kN;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (c < D) a.scratch[(int64_t)blockIdx.x * D + c + i] = gw[p][i];
  }
}

// The same for rows too wide for registers: grad_x alone, the row read twice.
template <typename T, int kN>
__global__ void __launch_bounds__(kWideThreads) k_rms_grad_wide(const rms_grad_args a) {
  __shared__ float2 sm[2][32];
  const int64_t D = a.total.n_cols, R = a.total.n_rows;
  const T *gy = static_cast<const T *>(a.grad_y.data), *x = static_cast<const T *>(a.total.data);
  const T *gt = static_cast<const T *>(a.grad_total.data);
  int set = 0;
  for (int64_t row = blockIdx.x; row < R; row += gridDim.x, set ^= 1) {
    const float rstd = a.rstd[row];
    auto values = [&](int64_t c, float (&g)[kN], float (&xh)[kN]) {
      float w[kN];
      load_weights<kN>(a.weight, c, w);
      widen(load_pack<T, kN>(gy + row * a.grad_y.ld + c), g);
      widen(load_pack<T, kN>(x + row * a.total.ld + c), xh);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        g[i] *= w[i];
        xh[i] *= rstd;
      }
    };
    float dot = 0.0f, g[kN], xh[kN];
    for (int64_t c = (int64_t)threadIdx.x * kN; c < D; c += (int64_t)blockDim.x * kN) {
      values(c, g, xh);
#pragma unroll
      for (int i = 0; i < kN; ++i) dot = fmaf(g[i], xh[i], dot);
    }
    const float mean = block_sum_max(dot, 0.0f, sm, set).x / (float)D;
    for (int64_t c = (int64_t)threadIdx.x * kN; c < D; c += (int64_t)blockDim.x * kN) {
      float y[kN], t[kN];
      values(c, g, xh);
      if (gt) widen(load_pack<T, kN>(gt + row * a.grad_total.ld + c), t);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        y[i] = rstd * (g[i] - xh[i] * mean);
        if (gt) y[i] += t[i];
      }
      store_pack(static_cast<T *>(a.grad_x.data) + row * a.grad_x.ld + c, narrow<T, kN>(y));
    }
  }
}

// Wide rows' grad_w: a block sums 32 columns over its share of the rows into
// scratch[blockIdx.y][D].
template <typename T>
__global__ void __launch_bounds__(256) k_rms_grad_cols(const rms_grad_args a) {
  __shared__ float sm[8][33];
  const int64_t D = a.total.n_cols, R = a.total.n_rows;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const T *gy = static_cast<const T *>(a.grad_y.data), *x = static_cast<const T *>(a.total.data);
  float sum = 0.0f;
  if (c < D)
    for (int64_t row = (int64_t)blockIdx.y * 8 + warp; row < R; row += (int64_t)gridDim.y * 8)
      sum = fmaf(Type<T>::up(gy[row * a.grad_y.ld + c]), Type<T>::up(x[row * a.total.ld + c]) * a.rstd[row], sum);
  sm[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && c < D) {
    for (int k = 1; k < 8; ++k) sum += sm[k][lane];
    a.scratch[(int64_t)blockIdx.y * D + c] = sum;
  }
}

// grad_w[c] = sum over the n rows of part, in a fixed order: eight warps take
// every eighth row of 32 columns each.
__global__ void __launch_bounds__(256) k_sum_rows(const float *part, int64_t n, int64_t D, void *out, int32_t type) {
  __shared__ float sm[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float sum = 0.0f;
  if (c < D)
    for (int64_t k = warp; k < n; k += 8) sum += part[k * D + c];
  sm[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && c < D) {
    for (int k = 1; k < 8; ++k) sum += sm[k][lane];
    if (type == SS_VALUES_F32)
      static_cast<float *>(out)[c] = sum;
    else if (type == SS_VALUES_BF16)
      static_cast<__nv_bfloat16 *>(out)[c] = __float2bfloat16_rn(sum);
    else
      static_cast<__half *>(out)[c] = __float2half_rn(sum);
  }
}

// Threads and vectors a thread for D columns in vectors of n values: one
// vector a thread where kMostThreads threads allow it (a row is then one load
// a thread), else 4, else most_per; 0 vectors: too wide for registers.
struct Shape {
  int threads, per;
};
Shape shape_for(int64_t D, int n, int most_per) {
  const int64_t vecs = (D + n - 1) / n;
  for (int per = 1; per <= most_per; per *= 4) {
    if (vecs <= (int64_t)per * kMostThreads) {
      const int64_t t = (vecs + per - 1) / per;
      return {(int)((t + 31) / 32 * 32), per};
    }
  }
  return {kWideThreads, 0};
}

// Blocks that fill the GPU at `threads` a block, at most `rows`.
int64_t fill(const ss_handle *h, int threads, int64_t rows) {
  return std::min<int64_t>(rows, (int64_t)std::max(1, h->sm_count) * std::min(32, 2048 / threads));
}

template <typename T, bool kF8>
cudaError_t rms_norm_typed(ss_handle *h, const rms_args &a, cudaStream_t s) {
  constexpr int kV = Type<T>::kVec;
  const int64_t R = a.x.n_rows, D = a.x.n_cols;
  auto aligned = [&](const ss_dense &m, int64_t unit) { return !m.data || rows_aligned(m, unit); };
  const bool vec = D % kV == 0 && aligned(a.x, 16) && aligned(a.residual, 16) && aligned(a.total, 16) &&
                   aligned(a.y, kF8 ? kV : 16);
  const Shape sh = shape_for(D, vec ? kV : 1, vec ? 4 : 16);
  auto run = [&](auto kernel) {
    kernel<<<(unsigned)fill(h, sh.threads, R), sh.threads, 0, s>>>(a);
  };
  if (sh.per == 0)
    vec ? run(k_rms_norm_wide<T, kF8, kV>) : run(k_rms_norm_wide<T, kF8, 1>);
  else if (vec)
    sh.per == 1 ? run(k_rms_norm<T, kF8, kV, 1>) : run(k_rms_norm<T, kF8, kV, 4>);
  else
    sh.per == 1   ? run(k_rms_norm<T, kF8, 1, 1>)
    : sh.per == 4 ? run(k_rms_norm<T, kF8, 1, 4>)
                  : run(k_rms_norm<T, kF8, 1, 16>);
  return cudaGetLastError();
}

// Most blocks of a gradient launch: enough to fill the GPU, while the rows of
// partial sums stay a few megabytes.
int64_t most_parts(const ss_handle *h, int64_t R, int64_t D) {
  return std::min<int64_t>(R, std::max<int64_t>(std::max(1, h->sm_count), (int64_t)(5 << 18) / D));
}

template <typename T>
cudaError_t rms_grad_typed(ss_handle *h, const rms_grad_args &a, cudaStream_t s, int *queued) {
  constexpr int kV = Type<T>::kVec;
  const int64_t R = a.total.n_rows, D = a.total.n_cols;
  if (R == 0)  // the sum over no rows
    return cudaMemsetAsync(a.grad_weight.data, 0, (size_t)(D * size_of(a.grad_weight.type)), s);
  auto aligned = [&](const ss_dense &m) { return !m.data || rows_aligned(m, 16); };
  const bool vec = D % kV == 0 && aligned(a.grad_y) && aligned(a.total) && aligned(a.grad_total) && aligned(a.grad_x);
  const Shape sh = shape_for(D, vec ? kV : 1, vec ? 4 : 16);
  int64_t n = most_parts(h, R, D);
  auto run = [&](auto kernel, int64_t blocks) {
    blocks = std::min(blocks, fill(h, sh.threads, R));
    kernel<<<(unsigned)blocks, sh.threads, 0, s>>>(a);
    return blocks;
  };
  if (sh.per == 0) {
    vec ? run(k_rms_grad_wide<T, kV>, R) : run(k_rms_grad_wide<T, 1>, R);
    n = std::min<int64_t>(n, 32);
    k_rms_grad_cols<T><<<dim3((unsigned)((D + 31) / 32), (unsigned)n), 256, 0, s>>>(a);
    *queued += 1;
  } else if (vec) {
    n = sh.per == 1 ? run(k_rms_grad<T, kV, 1>, n) : run(k_rms_grad<T, kV, 4>, n);
  } else {
    n = sh.per == 1   ? run(k_rms_grad<T, 1, 1>, n)
        : sh.per == 4 ? run(k_rms_grad<T, 1, 4>, n)
                      : run(k_rms_grad<T, 1, 16>, n);
  }
  k_sum_rows<<<(unsigned)((D + 31) / 32), 256, 0, s>>>(a.scratch, n, D, a.grad_weight.data, a.grad_weight.type);
  *queued += 2;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rms_norm(ss_handle *h, const rms_args &a, cudaStream_t s, int *queued) {
  const bool f8 = a.y.type == SS_VALUES_F8;
  *queued = 1;
  switch (a.x.type) {
    case SS_VALUES_F32:
      return f8 ? rms_norm_typed<float, true>(h, a, s) : rms_norm_typed<float, false>(h, a, s);
    case SS_VALUES_BF16:
      return f8 ? rms_norm_typed<__nv_bfloat16, true>(h, a, s) : rms_norm_typed<__nv_bfloat16, false>(h, a, s);
    default:
      return f8 ? rms_norm_typed<__half, true>(h, a, s) : rms_norm_typed<__half, false>(h, a, s);
  }
}

int64_t rms_grad_scratch(const ss_handle *h, int64_t R, int64_t D) {
  return R > 0 ? most_parts(h, R, D) * D * (int64_t)sizeof(float) : 0;
}

cudaError_t launch_rms_norm_grad(ss_handle *h, const rms_grad_args &a, cudaStream_t s, int *queued) {
  *queued = 0;
  switch (a.total.type) {
    case SS_VALUES_F32:
      return rms_grad_typed<float>(h, a, s, queued);
    case SS_VALUES_BF16:
      return rms_grad_typed<__nv_bfloat16>(h, a, s, queued);
    default:
      return rms_grad_typed<__half>(h, a, s, queued);
  }
}
