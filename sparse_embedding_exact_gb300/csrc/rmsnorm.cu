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
// Both are bound by memory: every value is read from it once and written
// once.  A group of threads takes a row at a time, each thread the same
// columns of every row, so the weights (and the gradient's sums over rows)
// stay in registers; values are worked on in pairs, one instruction for two.
// Rows arrive by bulk copies in a ring of shared-memory slots, the next rows
// while one is worked on: with plain loads into registers too few bytes were
// in flight (16,384 rows of 4096 bf16 with residual to 8 bits: 113 us).  A bulk
// copy moves whole 16-byte units, those that a row shares with its neighbours
// included; where all matrices' rows start alike within a unit, threads work
// on units and drop what is not the row's.  The sums over a block's rows go to
// scratch, one row of it a block, and a second kernel adds them in a fixed
// order: no atomics, the same bits every time.
//
// Measured: 16,384 x 4096 bf16 with residual to 8 bits 86 us (5.4 TB/s: memory);
// the gradient of 16,384 x 2048 bf16 59 us, of which the kernel 50 and the sums 6
// to 7 (4.6 TB/s: waiting, at 1.8 of 4 instructions issued a clock by 16 warps an
// SM, which its registers allow); of 5000 x 1001 float32 27 us (22 and 5, the
// same at 23 warps).
#include <algorithm>
#include <initializer_list>

#include "kept.cuh"
#include "product.cuh"

namespace {

using namespace dense;

constexpr int kWideThreads = 1024;
constexpr int64_t kRingBytes = 200 << 10;  // of an SM's shared memory, for the rings of its blocks
constexpr int kMostThreads = 512;  // of a block that holds its rows in registers, up to 128 a thread

// Threads of a block of the gradient: 16 values a thread leave room for three
// blocks of 256.
constexpr int grad_threads(int n, int per) { return n * per == 16 ? 256 : kMostThreads; }

// Threads of a block that work on one row: `index` of them in the block's
// order, each of `threads` threads.
struct Group {
  int index, threads, lane;  // lane: this thread within its group
  __device__ explicit Group(int t) : index(threadIdx.x / t), threads(t), lane(threadIdx.x % t) {}
  __device__ void sync() const {
    if (threads == 32)
      __syncwarp();
    else
      tc::named_sync(1 + index, threads);
  }
};

// Sum of a (and, with kMax, maximum of b) over the group, in every thread.  `sm`
// holds two sets of 32 pairs, a group's at its first warp's number;
// consecutive calls alternate `set`, so that one barrier a call is enough.
template <bool kMax>
__device__ __forceinline__ float2 group_reduce(const Group &gr, float a, float b, float2 (*sm)[32], int set) {
  a = warp_sum(a);
  if (kMax) b = warp_max_nan(b);
  const int n_warps = gr.threads >> 5;
  if (n_warps == 1) {
    __syncwarp();
    return make_float2(a, b);
  }
  const int lane = threadIdx.x & 31, first = gr.index * n_warps;
  if (lane == 0) sm[set][threadIdx.x >> 5] = make_float2(a, b);
  gr.sync();
  if (n_warps == 2 || n_warps == 4) {  // the usual widths: no shuffles
    const float2 v0 = sm[set][first], v1 = sm[set][first + 1];
    float2 r = make_float2(v0.x + v1.x, kMax ? max_nan(v0.y, v1.y) : 0.0f);
    if (n_warps == 4) {
      const float2 v2 = sm[set][first + 2], v3 = sm[set][first + 3];
      r.x += v2.x + v3.x;
      if (kMax) r.y = max_nan(r.y, max_nan(v2.y, v3.y));
    }
    return r;
  }
  const float2 v = lane < n_warps ? sm[set][first + lane] : make_float2(0.0f, 0.0f);
  return make_float2(warp_sum(v.x), kMax ? warp_max_nan(v.y) : 0.0f);
}

// Weights c .. c + kN - 1, 0 where the row has none.
template <int kN>
__device__ __forceinline__ void load_weights(const ss_dense &w, int64_t c, float (&f)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i)
    f[i] = c + i < 0 || c + i >= w.n_cols ? 0.0f
           : w.type == SS_VALUES_F32    ? static_cast<const float *>(w.data)[c + i]
           : w.type == SS_VALUES_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(w.data)[c + i])
                                      : __half2float(static_cast<const __half *>(w.data)[c + i]);
}

// The factor that brings a row's s w to e4m3's range: q = (s w pre) mul.  Rows
// below 1e-30 are scaled up first, as 448 / max would overflow.
__device__ __forceinline__ float2 f8_factors(float most) {
  const float pre = most < 1e-30f ? 0x1p100f : 1.0f;
  return make_float2(pre, most > 0.0f ? kF8Max / (most * pre) : (most == 0.0f ? 0.0f : most));
}

// A row's scale, max|y| / 448; 0 for a row of zeros, also where eps = 0 makes
// its rstd infinite.
__device__ __forceinline__ float scale_of(float most, float rstd) { return most * (most == 0.0f ? 0.0f : rstd) / kF8Max; }

// A group's ring of rows in shared memory: slot s holds the current row of kRows
// matrices.  Value c of a row lies at the same place within 16 bytes as in
// global memory.
template <typename T, int kRows>
struct Ring {
  uint32_t base, pitch;  // bytes of a row's place
  uint32_t n;            // matrices present (the absent ones come last)
  uint32_t bars;
  int64_t R, D;

  static __host__ __device__ uint32_t pitch_for(int64_t D) { return (uint32_t)((D * (int64_t)sizeof(T) + 15) / 16 * 16 + 16); }
  // What a bulk copy of row `row` at p takes: whole 16-byte units, those that
  // the row shares with the rows before and after it included where these are
  // there (and a unit long).
  __device__ __forceinline__ void span(const T *p, int64_t row, uintptr_t &b, uintptr_t &e) const {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p), end = at + D * sizeof(T);
    const bool lengthy = D * (int64_t)sizeof(T) >= 16;
    b = lengthy && row > 0 ? at & ~(uintptr_t)15 : (at + 15) & ~(uintptr_t)15;
    e = lengthy && row < R - 1 ? (end + 15) & ~(uintptr_t)15 : end & ~(uintptr_t)15;
    if (e < b) e = b;
  }
  // By one thread: copies row `row` of each matrix (null: none) into a slot.
  // The few values outside whole units, of the first and the last row or of
  // rows shorter than a unit, it copies itself.
  __device__ void fetch(int slot, const T *const (&p)[kRows], const int64_t (&ld)[kRows], int64_t row) const {
    uint32_t bytes = 0;
    const uint32_t bar = bars + 8u * slot;
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (p[k]) {
        const T *q = p[k] + row * ld[k];
        uintptr_t b, e;
        span(q, row, b, e);
        bytes += (uint32_t)(e - b);
        const uintptr_t at = reinterpret_cast<uintptr_t>(q), end = at + D * sizeof(T);
        const uint32_t to = place(slot, k, q);
        if (b > at || e < end)
          for (uintptr_t v = at; v < end; v += sizeof(T)) {
            if (v >= b && v < e) v = e;
            if (v < end) tc::write_shared(to + (uint32_t)(v - at), *reinterpret_cast<const T *>(v));
          }
      }
    tc::bar_expect(bar, bytes);
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (p[k]) {
        const T *q = p[k] + row * ld[k];
        uintptr_t b, e;
        span(q, row, b, e);
        if (e > b)
          tc::load_bulk(place(slot, k, q) + (uint32_t)(int32_t)(int64_t)(b - reinterpret_cast<uintptr_t>(q)),
                        reinterpret_cast<const void *>(b), (uint32_t)(e - b), bar);
      }
  }
  // Where value 0 of the row at p lies in `slot`.
  __device__ __forceinline__ uint32_t place(int slot, int k, const T *p) const {
    return base + ((uint32_t)slot * n + k) * pitch + (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
  }
  // Values c .. c + kN - 1 of the row of matrix k in `slot`, 0 where the row
  // has none; `at`: their place from the row's (for kN > 1 a 16-byte unit's,
  // the same for every row).
  template <int kN, bool kEdges>
  __device__ __forceinline__ Pack<T, kN> read(int slot, int k, uint32_t at, int c) const {
    Pack<T, kN> v = tc::read_shared<Pack<T, kN>>(base + ((uint32_t)slot * n + k) * pitch + at);
    if (kEdges && (c < 0 || c + kN > (int)D)) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (c + i < 0 || c + i >= (int)D) clear_item(v, i);
    }
    return v;
  }
  // That place: units count from the 16 bytes that the row starts in.
  template <int kN>
  __device__ __forceinline__ uint32_t at_of(const T *p, int unit) const {
    return kN > 1 ? 16u * unit : (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15) + (uint32_t)(unit * sizeof(T));
  }
};

// Values c .. c + kN - 1 of a row at p, those that it has.
template <typename T, int kN, bool kEdges>
__device__ __forceinline__ void write(T *p, int c, int D, const float (&f)[kN]) {
  const Pack<T, kN> v = narrow<T, kN>(f);
  if (!kEdges || (c >= 0 && c + kN <= D)) {
    store_pack(p + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (c + i >= 0 && c + i < D) p[c + i] = item(v, i);
  }
}
template <int kN, bool kEdges>
__device__ __forceinline__ void write_f8(uint8_t *p, int c, int D, const float (&f)[kN]) {
  if (!kEdges || (c >= 0 && c + kN <= D)) {
    store_f8<kN>(p + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float one[1] = {f[i]};
      if (c + i >= 0 && c + i < D) store_f8<1>(p + c + i, one);
    }
  }
}

// kN values worked on in pairs, or one alone.
template <typename T, int kN>
struct Work {
  using V = Two;
  static constexpr int kM = kN / 2;
  static __device__ __forceinline__ V get(const Pack<T, kN> &p, int i) { return pair_of(p, i); }
  static __device__ __forceinline__ V all(float x) { return two(x, x); }
  static __device__ __forceinline__ V of(const float (&f)[kN], int i) { return two(f[2 * i], f[2 * i + 1]); }
  static __device__ __forceinline__ void put(float (&f)[kN], int i, V v) {
    const float2 q = both(v);
    f[2 * i] = q.x;
    f[2 * i + 1] = q.y;
  }
  static __device__ __forceinline__ float sum(V v) {
    const float2 q = both(v);
    return q.x + q.y;
  }
  static __device__ __forceinline__ float most(float m, V v) {
    const float2 q = both(v);
    return max_nan(m, max_nan(fabsf(q.x), fabsf(q.y)));
  }
  template <typename F>
  static __device__ __forceinline__ V each(V v, F f) {
    const float2 q = both(v);
    return two(f(q.x), f(q.y));
  }
};
__device__ __forceinline__ float fma_of(float a, float b, float c) { return fmaf(a, b, c); }
using dense::fma_of;
template <typename T>
struct Work<T, 1> {
  using V = float;
  static constexpr int kM = 1;
  static __device__ __forceinline__ V get(const Pack<T, 1> &p, int) { return Type<T>::up(p.v[0]); }
  static __device__ __forceinline__ V all(float x) { return x; }
  static __device__ __forceinline__ V of(const float (&f)[1], int) { return f[0]; }
  static __device__ __forceinline__ void put(float (&f)[1], int, V v) { f[0] = v; }
  static __device__ __forceinline__ float sum(V v) { return v; }
  static __device__ __forceinline__ float most(float m, V v) { return max_nan(m, fabsf(v)); }
  template <typename F>
  static __device__ __forceinline__ V each(V v, F f) { return f(v); }
};

// Barriers and place of this group's ring in dynamic shared memory (the
// barriers of 16 groups of 4 slots come first); the first rows' copies are
// under way on return.  Row `first` and every `step`-th after it are the
// group's.
constexpr int kBarBytes = 16 * 4 * 8;
template <typename T, int kRows>
__device__ __forceinline__ Ring<T, kRows> open_ring(unsigned char *raw, const Group &gr, int slots, const T *const (&p)[kRows],
                                                    const int64_t (&ld)[kRows], int64_t first, int64_t step, int64_t R,
                                                    int64_t D) {
  Ring<T, kRows> ring;
  ring.R = R;
  ring.D = D;
  ring.pitch = Ring<T, kRows>::pitch_for(D);
  ring.bars = tc::smem_u32(raw) + 32u * gr.index;
  ring.n = 0;
  for (int k = 0; k < kRows; ++k) ring.n += p[k] != nullptr;
  ring.base = tc::smem_u32(raw) + kBarBytes + (uint32_t)(gr.index * slots) * ring.n * ring.pitch;
  if (gr.lane == 0) {
    for (int k = 0; k < slots; ++k) tc::bar_init(ring.bars + 8u * k, 1);
    tc::bar_init_fence();
    for (int k = 0; k < slots; ++k)
      if (first + k * step < R) ring.fetch(k, p, ld, first + k * step);
  }
  __syncthreads();
  return ring;
}

// Values by which the rows of a group start past a 16-byte boundary: the same
// for all of them, as `step` is a multiple of the values in 16 bytes where
// that is not the same for all rows.
template <typename T, int kN>
__device__ __forceinline__ int shift_of(const T *p, int64_t ld, int64_t row) {
  return kN == 1 ? 0 : (int)(reinterpret_cast<uintptr_t>(p + row * ld) / sizeof(T) % kN);
}

// kN values a vector (a 16-byte unit of them, or 1), kPer vectors a thread:
// columns (p * threads + lane) * kN - shift + i of the group's row, those that
// it has.  kEdges: units of several values, some of which have values before
// or after the row's.
template <typename T, bool kF8, int kN, int kPer, bool kEdges>
__global__ void __launch_bounds__(kMostThreads, 1) k_rms_norm(const rms_args a, int threads, int slots, int32_t *status) {
  using W = Work<T, kN>;
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ float2 sm[2][32];
  __shared__ int stalled;
  if (threadIdx.x == 0) stalled = 0;
  const Group gr(threads);
  const int64_t D = a.x.n_cols, R = a.x.n_rows;
  const T *const src[2] = {static_cast<const T *>(a.x.data), static_cast<const T *>(a.residual.data)};
  const int64_t ld[2] = {a.x.ld, a.residual.ld};
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / threads);
  const int64_t first = (int64_t)gr.index * gridDim.x + blockIdx.x;
  const Ring<T, 2> ring = open_ring<T, 2>(raw, gr, slots, src, ld, first, step, R, D);
  const int shift = kEdges ? shift_of<T, kN>(src[0], ld[0], first) : 0;
  const float inv_d = 1.0f / (float)D;
  T *total = static_cast<T *>(a.total.data);
  typename W::V w[kPer][W::kM];
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int unit = p * threads + gr.lane, c = unit * kN - shift;
    if (c < (int)D) {
      float f[kN];
      load_weights<kN>(a.weight, c, f);
#pragma unroll
      for (int i = 0; i < W::kM; ++i) w[p][i] = W::of(f, i);
    }
  }
  int set = 0, slot = 0;
  uint32_t phase = 0;
  for (int64_t row = first; row < R; row += step, set ^= 1) {
    tc::bar_wait_on(ring.bars + 8u * slot, phase, status, &stalled);
    typename W::V s[kPer][W::kM], sq = W::all(0.0f);
    float most = 0.0f;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int unit = p * threads + gr.lane, c = unit * kN - shift;
      if (c < (int)D) {
        const Pack<T, kN> x = ring.template read<kN, kEdges>(slot, 0, ring.template at_of<kN>(src[0] + row * ld[0], unit), c);
#pragma unroll
        for (int i = 0; i < W::kM; ++i) s[p][i] = W::get(x, i);
        if (src[1]) {
          const Pack<T, kN> r = ring.template read<kN, kEdges>(slot, 1, ring.template at_of<kN>(src[1] + row * ld[1], unit), c);
#pragma unroll
          for (int i = 0; i < W::kM; ++i) s[p][i] = s[p][i] + W::get(r, i);
        }
#pragma unroll
        for (int i = 0; i < W::kM; ++i) {
          sq = fma_of(s[p][i], s[p][i], sq);
          if (kF8) most = W::most(most, s[p][i] * w[p][i]);
        }
      }
    }
    const float2 red = group_reduce<kF8>(gr, W::sum(sq), most, sm, set);
    // every thread has read the slot: the row that comes `slots` turns later
    const int64_t later = row + slots * step;
    if (gr.lane == 0 && later < R) ring.fetch(slot, src, ld, later);
    if (++slot == slots) {
      slot = 0;
      phase ^= 1;
    }
    const float rstd = 1.0f / sqrtf(red.x * inv_d + a.eps);
    if (gr.lane == 0) {
      if (a.rstd) a.rstd[row] = rstd;
      if (kF8) a.scale[row] = scale_of(red.y, rstd);
    }
    const float2 to8 = kF8 ? f8_factors(red.y) : make_float2(0.0f, 0.0f);
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int unit = p * threads + gr.lane, c = unit * kN - shift;
      if (c < (int)D) {
        float f[kN];
        if (total && src[1]) {
#pragma unroll
          for (int i = 0; i < W::kM; ++i) W::put(f, i, s[p][i]);
          write<T, kN, kEdges>(total + row * a.total.ld, c, (int)D, f);
        }
#pragma unroll
        for (int i = 0; i < W::kM; ++i)
          W::put(f, i, kF8 ? s[p][i] * w[p][i] * W::all(to8.x) * W::all(to8.y) : s[p][i] * W::all(rstd) * w[p][i]);
        if (kF8)
          write_f8<kN, kEdges>(static_cast<uint8_t *>(a.y.data) + row * a.y.ld, c, (int)D, f);
        else
          write<T, kN, kEdges>(static_cast<T *>(a.y.data) + row * a.y.ld, c, (int)D, f);
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
  const Group gr(blockDim.x);
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
    const float2 red = group_reduce<kF8>(gr, sq, most, sm, set);
    const float rstd = 1.0f / sqrtf(red.x / (float)D + a.eps);
    if (threadIdx.x == 0) {
      if (a.rstd) a.rstd[row] = rstd;
      if (kF8) a.scale[row] = scale_of(red.y, rstd);
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
template <typename T, int kN, int kPer, bool kEdges>
__global__ void __launch_bounds__(grad_threads(kN, kPer), kN * kPer == 16 ? 3 : 1) k_rms_grad(const rms_grad_args a, int threads, int slots, int32_t *status) {
  using W = Work<T, kN>;
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ float2 sm[2][32];
  __shared__ int stalled;
  if (threadIdx.x == 0) stalled = 0;
  const Group gr(threads);
  const int64_t D = a.total.n_cols, R = a.total.n_rows;
  const T *const src[3] = {static_cast<const T *>(a.grad_y.data), static_cast<const T *>(a.total.data),
                           static_cast<const T *>(a.grad_total.data)};
  const int64_t ld[3] = {a.grad_y.ld, a.total.ld, a.grad_total.ld};
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / threads);
  const int64_t first = (int64_t)gr.index * gridDim.x + blockIdx.x;
  const Ring<T, 3> ring = open_ring<T, 3>(raw, gr, slots, src, ld, first, step, R, D);
  const int shift = kEdges ? shift_of<T, kN>(src[0], ld[0], first) : 0;
  const float inv_d = 1.0f / (float)D;
  typename W::V w[kPer][W::kM], gw[kPer][W::kM];
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int unit = p * threads + gr.lane, c = unit * kN - shift;
    float f[kN];
    if (c < (int)D) load_weights<kN>(a.weight, c, f);
#pragma unroll
    for (int i = 0; i < W::kM; ++i) {
      if (c < (int)D) w[p][i] = W::of(f, i);
      gw[p][i] = W::all(0.0f);
    }
  }
  int set = 0, slot = 0;
  uint32_t phase = 0;
  float rstd_next = first < R ? a.rstd[first] : 0.0f;
  for (int64_t row = first; row < R; row += step, set ^= 1) {
    const float rstd = rstd_next;
    if (row + step < R) rstd_next = a.rstd[row + step];
    tc::bar_wait_on(ring.bars + 8u * slot, phase, status, &stalled);
    typename W::V dot = W::all(0.0f);
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int unit = p * threads + gr.lane, c = unit * kN - shift;
      if (c < (int)D) {
        const Pack<T, kN> gv = ring.template read<kN, kEdges>(slot, 0, ring.template at_of<kN>(src[0] + row * ld[0], unit), c);
        const Pack<T, kN> xv = ring.template read<kN, kEdges>(slot, 1, ring.template at_of<kN>(src[1] + row * ld[1], unit), c);
#pragma unroll
        for (int i = 0; i < W::kM; ++i) {
          const typename W::V g = W::get(gv, i), xh = W::get(xv, i) * W::all(rstd);
          gw[p][i] = fma_of(g, xh, gw[p][i]);
          dot = fma_of(g * w[p][i], xh, dot);
        }
      }
    }
    const float mean = group_reduce<false>(gr, W::sum(dot), 0.0f, sm, set).x * inv_d;
    // Every thread is through with the row before: its slot's next row.  (The
    // row itself is read again below, rather than kept: half the registers,
    // half again as many blocks on an SM.)
    if (gr.lane == 0 && slots > 1 && row != first && row + (slots - 1) * step < R)
      ring.fetch(slot == 0 ? slots - 1 : slot - 1, src, ld, row + (slots - 1) * step);
    // rstd (g w - xh mean) + t = g w rstd + (x (-rstd^2 mean) + t)
    const typename W::V fx = W::all(-rstd * rstd * mean), fg = W::all(rstd);
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const int unit = p * threads + gr.lane, c = unit * kN - shift;
      if (c < (int)D) {
        const Pack<T, kN> gv = ring.template read<kN, kEdges>(slot, 0, ring.template at_of<kN>(src[0] + row * ld[0], unit), c);
        const Pack<T, kN> xv = ring.template read<kN, kEdges>(slot, 1, ring.template at_of<kN>(src[1] + row * ld[1], unit), c);
        Pack<T, kN> tv;
        if (src[2]) tv = ring.template read<kN, kEdges>(slot, 2, ring.template at_of<kN>(src[2] + row * ld[2], unit), c);
        float y[kN];
#pragma unroll
        for (int i = 0; i < W::kM; ++i) {
          const typename W::V t = src[2] ? W::get(tv, i) : W::all(0.0f);
          W::put(y, i, fma_of(W::get(gv, i) * w[p][i], fg, fma_of(W::get(xv, i), fx, t)));
        }
        write<T, kN, kEdges>(static_cast<T *>(a.grad_x.data) + row * a.grad_x.ld, c, (int)D, y);
      }
    }
    if (slots == 1) {
      gr.sync();
      if (gr.lane == 0 && row + step < R) ring.fetch(0, src, ld, row + step);
    }
    if (++slot == slots) {
      slot = 0;
      phase ^= 1;
    }
  }
  // The groups' sums in their order, through the rings (whose copies have all
  // been read).
  const int groups = blockDim.x / threads;
  float *mine = a.scratch + (int64_t)blockIdx.x * D;
  float *place = reinterpret_cast<float *>(raw + kBarBytes);
  if (groups > 1) {
    __syncthreads();
    mine = place + gr.index * D;
  }
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int c = (p * threads + gr.lane) * kN - shift;
    float f[kN];
#pragma unroll
    for (int i = 0; i < W::kM; ++i) W::put(f, i, gw[p][i]);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (c + i >= 0 && c + i < D) mine[c + i] = f[i];
  }
  if (groups > 1) {
    __syncthreads();
    for (int64_t c = threadIdx.x; c < D; c += blockDim.x) {
      float v = place[c];
      for (int g = 1; g < groups; ++g) v += place[g * D + c];
      a.scratch[(int64_t)blockIdx.x * D + c] = v;
    }
  }
}

// The same from a total kept in 8 bits: 5 bytes a value of 16 bits in place of 6,
// and no copy of it widened.  A thread has kPer units of kN columns of every row.
// Where rows start on 16-byte boundaries it copies its units of the next rows
// into shared memory, which it alone reads, a slot a row: no barrier, and no
// registers for what is under way.  (Loads one row ahead into registers left
// room for half the warps.)  Other rows are loaded value by value.  16,384 x 2048
// bf16 47 us (5.0 TB/s, 7 of it the sums; by way of a widened copy 94), 4096 x
// 4096 31 (from 16 bits 38); 5000 x 1001 float32 25.
template <typename T, int kN, int kPer>
struct KeptRow {
  Pack<T, kN> g[kPer], t[kPer];
  Codes<kN> c[kPer];
};
// A thread's small change of a row, asked for two rows ahead.
template <int kPer>
struct KeptScales {
  float rstd;
  uint8_t byte[kPer];
};

// The sum of a over the group, in every thread: a warp's by shuffles, the warps'
// read back by all (eight of them in two loads).  sm as in group_reduce.
__device__ __forceinline__ float group_sum(const Group &gr, float a, float *sm) {
  a = warp_sum(a);
  const int n_warps = gr.threads >> 5;
  if (n_warps == 1) {
    __syncwarp();
    return a;
  }
  const int lane = threadIdx.x & 31, first = gr.index * n_warps;
  if (lane == 0) sm[threadIdx.x >> 5] = a;
  gr.sync();
  if (n_warps == 8) {
    const float4 p = reinterpret_cast<const float4 *>(sm + first)[0], q = reinterpret_cast<const float4 *>(sm + first)[1];
    return ((p.x + p.y) + (p.z + p.w)) + ((q.x + q.y) + (q.z + q.w));
  }
  return warp_sum(lane < n_warps ? sm[first + lane] : 0.0f);
}

constexpr int kKeptThreads = 256;  // of a block, or a row's own where it has more
// Rows under way: four, three where 512 threads' units would not fit 227 KB.
constexpr int kept_slots(int n, int per) { return kMostThreads * per * (32 + n) * 4 <= 220 * 1024 ? 4 : 3; }
static_assert(kMostThreads * 4 * (32 + 4) * kept_slots(4, 4) <= 220 * 1024 && kMostThreads * 2 * (32 + 8) * kept_slots(8, 2) <= 220 * 1024, "too large");
template <typename T, int kN, int kPer, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == kKeptThreads ? 3 : 1) k_rms_grad_kept(const rms_grad_args a, int threads) {
  using W = Work<T, kN>;
  constexpr bool kAsync = kN > 1;
  constexpr int kSlots = kept_slots(kN, kPer);
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ __align__(16) float sm[2][32];
  tc::let_next();
  const Group gr(threads);
  const int D = (int)a.total.n_cols, R = (int)a.total.n_rows, step = (int)gridDim.x * ((int)blockDim.x / threads);
  const float inv_d = 1.0f / (float)D;
  const bool past = a.grad_total.data != nullptr;
  // A thread past the row's end works on the last unit again, without branches,
  // and keeps it to itself.
  int at[kPer];
  bool in[kPer];
  typename W::V w[kPer][W::kM], gw[kPer][W::kM];
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    const int c = (p * threads + gr.lane) * kN;
    in[p] = c < D;
    at[p] = min(c, D - kN);
    float f[kN];
    load_weights<kN>(a.weight, at[p], f);
#pragma unroll
    for (int i = 0; i < W::kM; ++i) {
      w[p][i] = W::of(f, i);
      gw[p][i] = W::all(0.0f);
    }
  }
  const int first = gr.index * (int)gridDim.x + (int)blockIdx.x;
  // What is read next, and written: a step of rows further every turn
  const T *gy = static_cast<const T *>(a.grad_y.data) + first * a.grad_y.ld;
  const T *gt = static_cast<const T *>(a.grad_total.data) + (past ? first * a.grad_total.ld : 0);
  const uint8_t *codes = static_cast<const uint8_t *>(a.total_kept.codes) + first * a.total_kept.ld;
  const uint8_t *scale = a.total_kept.scale + first * a.total_kept.ld_scale;
  T *gx = static_cast<T *>(a.grad_x.data) + first * a.grad_x.ld;
  const int64_t step_g = step * a.grad_y.ld, step_t = step * a.grad_total.ld, step_c = step * a.total_kept.ld;
  const int64_t step_s = step * a.total_kept.ld_scale, step_x = step * a.grad_x.ld;
  // A slot: 16 bytes of g and of t and kN of codes for every unit of the block
  const uint32_t units = kPer * blockDim.x, slot_bytes = units * (32 + kN), base = tc::smem_u32(raw), base_end = base + kSlots * slot_bytes;
  auto fetch = [&](uint32_t slot, int row) {
    if (row < R) {
#pragma unroll
      for (int p = 0; p < kPer; ++p) {
        const uint32_t u = p * blockDim.x + threadIdx.x;
        tc::copy_async<16>(slot + 16 * u, gy + at[p]);
        if (past) tc::copy_async<16>(slot + 16 * units + 16 * u, gt + at[p]);
        tc::copy_async<kN == 1 ? 4 : kN>(slot + 32 * units + kN * u, codes + at[p]);
      }
      gy += step_g;
      gt += step_t;
      codes += step_c;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto scales = [&](int row) {
    KeptScales<kPer> s = {};
    if (row < R) {
      s.rstd = a.rstd[row];
#pragma unroll
      for (int p = 0; p < kPer; ++p) s.byte[p] = scale[at[p] / kGroup];
      scale += step_s;
    }
    return s;
  };
  int set = 0;
  uint32_t now = base, fill = base + (kSlots - 1) * slot_bytes;  // the slots of this row, and of the next to be fetched
  KeptScales<kPer> s0 = scales(first), s1 = scales(first + step), s2;
  if (kAsync)
    for (int i = 0; i < kSlots - 1; ++i) fetch(base + i * slot_bytes, first + i * step);
  for (int row = first; row < R; row += step, set ^= 1) {
    KeptRow<T, kN, kPer> v;
    if constexpr (kAsync) {
      fetch(fill, row + (kSlots - 1) * step);  // into the slot of the row before
      fill = now;
      asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
#pragma unroll
      for (int p = 0; p < kPer; ++p) {
        const uint32_t u = p * blockDim.x + threadIdx.x;
        v.g[p] = tc::read_shared<Pack<T, kN>>(now + 16 * u);
        if (past) v.t[p] = tc::read_shared<Pack<T, kN>>(now + 16 * units + 16 * u);
        v.c[p].load_shared(now + 32 * units + kN * u);
      }
      now += slot_bytes;
      if (now == base_end) now = base;
    } else {
#pragma unroll
      for (int p = 0; p < kPer; ++p) {
        v.g[p] = load_pack<T, kN>(gy + at[p]);
        if (past) v.t[p] = load_pack<T, kN>(gt + at[p]);
        v.c[p].load(codes + at[p]);
      }
      gy += step_g;
      gt += step_t;
      codes += step_c;
    }
    s2 = scales(row + 2 * step);
    auto code = [&](int p, int i) {
      if constexpr (kN == 1) {
        return v.c[p].one();
      } else {
        const float2 f = v.c[p].pair(i);
        return two(f.x, f.y);
      }
    };
    float dot = 0.0f;
    typename W::V weighed[kPer][W::kM], scaled[kPer][W::kM];  // g w and x, for both passes
    bool exact = true;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const typename W::V s = W::all(scale_of_byte(s0.byte[p]));
      exact = exact && exact_byte<T>(s0.byte[p]);
#pragma unroll
      for (int i = 0; i < W::kM; ++i) scaled[p][i] = code(p, i) * s;
    }
    // one branch for all units (4096 x 8192 float32 110 us, one each 116; 5000 x 1001
    // bf16 21 and 23; 2000 x 4095 bf16 37 and 35)
    if (!exact) {
#pragma unroll
      for (int p = 0; p < kPer; ++p)
#pragma unroll
        for (int i = 0; i < W::kM; ++i) scaled[p][i] = W::each(scaled[p][i], [](float x) { return as_type<T>(x); });
    }
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const typename W::V r = W::all(s0.rstd);
      typename W::V sum = W::all(0.0f);
#pragma unroll
      for (int i = 0; i < W::kM; ++i) {
        const typename W::V g = W::get(v.g[p], i);
        weighed[p][i] = g * w[p][i];
        const typename W::V xh = scaled[p][i] * r;
        gw[p][i] = fma_of(g, xh, gw[p][i]);
        sum = fma_of(weighed[p][i], xh, sum);
      }
      dot += in[p] ? W::sum(sum) : 0.0f;
    }
    const float mean = group_sum(gr, dot, sm[set]) * inv_d;
    const typename W::V fx = W::all(-s0.rstd * s0.rstd * mean), fg = W::all(s0.rstd);
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      float y[kN];
#pragma unroll
      for (int i = 0; i < W::kM; ++i) {
        const typename W::V t = past ? W::get(v.t[p], i) : W::all(0.0f);
        W::put(y, i, fma_of(weighed[p][i], fg, fma_of(scaled[p][i], fx, t)));
      }
      if (in[p]) store_pack(gx + at[p], narrow<T, kN>(y));
    }
    gx += step_x;
    s0 = s1;
    s1 = s2;
  }
  if (kAsync) asm volatile("cp.async.wait_all;" ::: "memory");
  // The groups' sums in their order, through shared memory where there are several.
  const int groups = blockDim.x / threads;
  float *place = reinterpret_cast<float *>(raw), *mine = groups > 1 ? place + gr.index * D : a.scratch + (int64_t)blockIdx.x * D;
  if (groups > 1) __syncthreads();  // the slots have all been read
#pragma unroll
  for (int p = 0; p < kPer; ++p) {
    float f[kN];
#pragma unroll
    for (int i = 0; i < W::kM; ++i) W::put(f, i, gw[p][i]);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (in[p]) mine[at[p] + i] = f[i];
  }
  if (groups > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      float v = place[c];
      for (int g = 1; g < groups; ++g) v += place[g * D + c];
      a.scratch[(int64_t)blockIdx.x * D + c] = v;
    }
  }
}

// The same for rows too wide for registers: grad_x alone, the row read twice.
template <typename T, int kN>
__global__ void __launch_bounds__(kWideThreads) k_rms_grad_wide(const rms_grad_args a) {
  __shared__ float2 sm[2][32];
  const int64_t D = a.total.n_cols, R = a.total.n_rows;
  const T *gy = static_cast<const T *>(a.grad_y.data), *x = static_cast<const T *>(a.total.data);
  const T *gt = static_cast<const T *>(a.grad_total.data);
  const Group gr(blockDim.x);
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
    const float mean = group_reduce<false>(gr, dot, 0.0f, sm, set).x / (float)D;
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

// out[c] = sum over the n rows of part, in a fixed order: a block takes kCols
// columns, each of its threads every (1024 / kCols)-th row of one, four at a
// time.  8 columns where 32 would leave more than half of the SMs idle (456
// rows of 1001: 5 us with 32, 3 with 8), else 32, a line a warp.
template <int kCols>
__global__ void __launch_bounds__(1024) k_sum_rows(const float *part, int64_t n, int64_t D, void *out, int32_t type) {
  tc::wait_before();
  constexpr int kLanes = 1024 / kCols;
  __shared__ float sm[kLanes][kCols + 1];
  const int col = threadIdx.x % kCols, lane = threadIdx.x / kCols;
  const int64_t c = (int64_t)blockIdx.x * kCols + col;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < D)
    for (int64_t k = lane; k < n; k += 4 * kLanes) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k + kLanes * u < n) sum[u] += part[(k + kLanes * u) * D + c];
    }
  sm[lane][col] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  __syncthreads();
  const int warp = threadIdx.x >> 5, t = threadIdx.x & 31;
  if (warp >= kCols) return;
  float v = 0.0f;
#pragma unroll
  for (int u = 0; u < kLanes; u += 32) v += sm[t + u][warp];
  v = warp_sum(v);
  const int64_t at = (int64_t)blockIdx.x * kCols + warp;
  if (t == 0 && at < D) {
    if (type == SS_VALUES_F32)
      static_cast<float *>(out)[at] = v;
    else if (type == SS_VALUES_BF16)
      static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
    else
      static_cast<__half *>(out)[at] = __float2half_rn(v);
  }
}

// How rows of D columns in vectors of n values are worked on: `per` vectors a
// thread of `threads` a row, `groups` rows a block, `slots` rows of the ring a
// group, `blocks` an SM.  per = 0: too wide for registers.
//
// Many rows: 4 vectors a thread, 16 or 32 values of it.  What a thread spends on
// a row besides its values (the reduction's shuffles and barrier, the root) is
// as much as 8 values cost: with 8 values a thread the norm of 16,384 x 4096
// bf16 rows to 8 bits took 94 us against 72, and with 16 the gradient of
// 16,384 x 2048 rows 63 against 59.  Rows for every SM or fewer: one vector a
// thread, for the time of one row.
constexpr int kVecPers[3] = {1, 4, 4}, kF32Pers[3] = {1, 4, 8}, kOnePers[3] = {1, 4, 16};
struct Shape {
  int per, threads, groups, slots, blocks, smem;
};
Shape shape_for(const ss_handle *h, int64_t R, int64_t D, int n, const int (&pers)[3], bool grad, int64_t row_bytes) {
  const int64_t vecs = (D + n - 1) / n;
  Shape sh = {0, kWideThreads, 1, 0, 2, 0};
  for (const int per : pers) {
    const int64_t t = ((vecs + per - 1) / per + 31) / 32 * 32;
    if (t > (grad ? grad_threads(n, per) : kMostThreads) || row_bytes > kRingBytes) continue;
    if (sh.per && (vecs < 32 * per || R <= h->sm_count)) break;
    if (sh.per && per > 4) break;  // where 4 do not reach
    sh.per = per;
    sh.threads = (int)t;
  }
  if (!sh.per) return sh;
  const bool many = R > h->sm_count;
  const int values = sh.per * n;
  sh.groups = many ? std::max(1, 256 / sh.threads) : 1;
  sh.blocks = std::max(1, (values <= 8 ? 1024 : grad && values == 16 ? 768 : 512) / (sh.groups * sh.threads));
  // up to four slots a group within the SM's ring bytes
  while (sh.blocks > 1 && sh.blocks * sh.groups * row_bytes > kRingBytes) --sh.blocks;
  while (sh.groups > 1 && sh.groups * row_bytes > kRingBytes) sh.groups /= 2;
  sh.slots = (int)std::min<int64_t>(4, kRingBytes / (sh.blocks * sh.groups * row_bytes));
  sh.smem = (int)(kBarBytes + sh.groups * sh.slots * row_bytes);
  return sh;
}

// Whether rows of these matrices (those present) can be worked on in 16-byte
// units of n values of the first: each row starts as many values past such a
// unit in all of them.  *shifting: not the same number in every row.
bool in_units(std::initializer_list<ss_dense> ms, int n, int64_t D, bool *shifting) {
  int64_t start = -1, ld = -1;
  for (const ss_dense &m : ms) {
    if (!m.data) continue;
    const int64_t s = (int64_t)(reinterpret_cast<uintptr_t>(m.data) / (uintptr_t)size_of(m.type) % (uintptr_t)n);
    const int64_t l = m.n_rows > 1 ? m.ld % n : 0;
    if (start >= 0 && (s != start || l != ld)) return false;
    start = s;
    ld = l;
  }
  *shifting = ld != 0;
  return D >= n || (start == 0 && ld == 0 && D % n == 0);
}
// A grid of `blocks` at most whose groups' step keeps a row's shift: a multiple
// of n rows.
int64_t keep_shift(int64_t blocks, int groups, int64_t R, int n, bool shifting) {
  if (!shifting || blocks * groups >= R) return blocks;
  while (blocks > 1 && blocks * groups % n != 0) --blocks;
  return blocks;
}

template <typename T, bool kF8>
cudaError_t rms_norm_typed(ss_handle *h, const rms_args &a, cudaStream_t s) {
  constexpr int kV = Type<T>::kVec;
  const int64_t R = a.x.n_rows, D = a.x.n_cols, sms = std::max(1, h->sm_count);
  bool shifting = false;
  const bool vec = in_units({a.x, a.residual, a.total, a.y}, kV, D, &shifting);
  const bool aligned = vec && !shifting && reinterpret_cast<uintptr_t>(a.x.data) % 16 == 0 && D % kV == 0;
  const Shape sh = shape_for(h, R, vec && !aligned ? D + kV - 1 : D, vec ? kV : 1, vec ? (kV == 4 ? kF32Pers : kVecPers) : kOnePers, false,
                             (a.residual.data ? 2 : 1) * (int64_t)Ring<T, 2>::pitch_for(D));
  if (sh.per == 0) {
    const unsigned grid = (unsigned)std::min<int64_t>(R, sms * sh.blocks);
    if (aligned)
      k_rms_norm_wide<T, kF8, kV><<<grid, sh.threads, 0, s>>>(a);
    else
      k_rms_norm_wide<T, kF8, 1><<<grid, sh.threads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const int64_t grid = keep_shift(std::min<int64_t>((R + sh.groups - 1) / sh.groups, sms * sh.blocks), sh.groups, R, kV, shifting && vec);
  auto run = [&](auto kernel) -> cudaError_t {
    const cudaError_t e = ensure_dyn_smem(kernel, sh.smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)grid, sh.groups * sh.threads, sh.smem, s>>>(a, sh.threads, sh.slots, h->d_status);
    return cudaGetLastError();
  };
  constexpr int kMore = kV == 4 ? 8 : 4;
  if (aligned)
    return sh.per == 1   ? run(k_rms_norm<T, kF8, kV, 1, false>)
           : sh.per == 4 ? run(k_rms_norm<T, kF8, kV, 4, false>)
                         : run(k_rms_norm<T, kF8, kV, kMore, false>);
  if (vec)
    return sh.per == 1   ? run(k_rms_norm<T, kF8, kV, 1, true>)
           : sh.per == 4 ? run(k_rms_norm<T, kF8, kV, 4, true>)
                         : run(k_rms_norm<T, kF8, kV, kMore, true>);
  return sh.per == 1   ? run(k_rms_norm<T, kF8, 1, 1, false>)
         : sh.per == 4 ? run(k_rms_norm<T, kF8, 1, 4, false>)
                       : run(k_rms_norm<T, kF8, 1, 16, false>);
}

// Most rows of partial sums of a gradient: its blocks, at most four an SM.
constexpr int kGradBlocks = 4;
int64_t most_parts(const ss_handle *h, int64_t R) {
  return std::min<int64_t>(R, (int64_t)kGradBlocks * std::max(1, h->sm_count));
}

// Rows of more values than this are widened into scratch and take the other
// kernels: a thread's sums over the rows would not stay in registers.
constexpr int64_t kKeptMost = 16 * kMostThreads;

template <typename T>
cudaError_t rms_grad_kept_typed(ss_handle *h, const rms_grad_args &a, cudaStream_t s, int *queued) {
  constexpr int kV = Type<T>::kVec;
  const int64_t R = a.total.n_rows, D = a.total.n_cols;
  if (R == 0) return cudaMemsetAsync(a.grad_weight.data, 0, (size_t)(D * size_of(a.grad_weight.type)), s);
  bool vec = D % kV == 0 && kept_aligned(a.total_kept, kV);
  for (const ss_dense *m : {&a.grad_y, &a.grad_total, &a.grad_x}) vec = vec && (!m->data || rows_aligned(*m, 16));
  // units a thread: two, one for short rows, more where a row's threads would be
  // more than a block has (one unit, 16,384 x 2048 bf16: 51 us; float32 by the same
  // rule 76, 86% of the memory's rate); values one by one four, up to sixteen, of
  // which 600 bytes are spilled (2000 x 4095 bf16 37 us, 2000 x 7001 164)
  const int64_t units = vec ? D / kV : D;
  int64_t per = vec ? (units > 128 ? 2 : 1) : 4;
  while ((units + per - 1) / per > (per == 1 ? kKeptThreads : kMostThreads)) per *= 2;
  const int threads = (int)(((units + per - 1) / per + 31) / 32 * 32), groups = std::max(1, kKeptThreads / threads);
  const size_t slots = vec ? (size_t)kept_slots(kV, (int)per) * per * (threads * groups) * (32 + kV) : 0;
  const size_t smem = std::max(slots, groups > 1 ? (size_t)groups * D * sizeof(float) : 0);
  auto run = [&](auto kernel, int an_sm) -> cudaError_t {
    cudaError_t e = ensure_dyn_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    const int64_t n = std::min<int64_t>((R + groups - 1) / groups, (int64_t)std::max(1, h->sm_count) * an_sm);
    kernel<<<(unsigned)n, groups * threads, smem, s>>>(a, threads);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    *queued += 2;
    return launch_sum_rows(h, a.scratch, n, D, a.grad_weight.data, a.grad_weight.type, s, true);
  };
  const bool small = threads * groups <= kKeptThreads;
  if (vec) {
    if (per == 1) return run(k_rms_grad_kept<T, kV, 1, kKeptThreads>, 3);
    // two units want more registers than three blocks an SM leave (4096 x 4096
    // bf16 with them 65 us)
    if (per == 2) return run(k_rms_grad_kept<T, kV, 2, kMostThreads>, small ? 2 : 1);
    if constexpr (kV == 4) return run(k_rms_grad_kept<T, kV, 4, kMostThreads>, 1);
  }
  if (per == 4) return small ? run(k_rms_grad_kept<T, 1, 4, kKeptThreads>, 3) : run(k_rms_grad_kept<T, 1, 4, kMostThreads>, 1);
  return per == 8 ? run(k_rms_grad_kept<T, 1, 8, kMostThreads>, 1) : run(k_rms_grad_kept<T, 1, 16, kMostThreads>, 1);
}

template <typename T>
cudaError_t rms_grad_typed(ss_handle *h, const rms_grad_args &a, cudaStream_t s, int *queued) {
  constexpr int kV = Type<T>::kVec;
  const int64_t R = a.total.n_rows, D = a.total.n_cols;
  if (R == 0)  // the sum over no rows
    return cudaMemsetAsync(a.grad_weight.data, 0, (size_t)(D * size_of(a.grad_weight.type)), s);
  bool shifting = false;
  const bool vec = in_units({a.grad_y, a.total, a.grad_total, a.grad_x}, kV, D, &shifting);
  const bool aligned = vec && !shifting && reinterpret_cast<uintptr_t>(a.total.data) % 16 == 0 && D % kV == 0;
  const Shape sh = shape_for(h, R, vec && !aligned ? D + kV - 1 : D, vec ? kV : 1, vec ? (kV == 4 ? kF32Pers : kVecPers) : kOnePers, true,
                             (a.grad_total.data ? 3 : 2) * (int64_t)Ring<T, 3>::pitch_for(D));
  int64_t n = std::min<int64_t>(most_parts(h, (R + sh.groups - 1) / sh.groups), (int64_t)std::max(1, h->sm_count) * sh.blocks);
  if (sh.per) n = keep_shift(n, sh.groups, R, kV, shifting && vec);
  auto run = [&](auto kernel) -> cudaError_t {
    const cudaError_t e = ensure_dyn_smem(kernel, sh.smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)n, sh.groups * sh.threads, sh.smem, s>>>(a, sh.threads, sh.slots, h->d_status);
    return cudaGetLastError();
  };
  cudaError_t e = cudaSuccess;
  if (sh.per == 0) {
    const unsigned grid = (unsigned)std::min<int64_t>(R, (int64_t)std::max(1, h->sm_count) * sh.blocks);
    if (aligned)
      k_rms_grad_wide<T, kV><<<grid, sh.threads, 0, s>>>(a);
    else
      k_rms_grad_wide<T, 1><<<grid, sh.threads, 0, s>>>(a);
    n = std::min<int64_t>(n, 32);
    k_rms_grad_cols<T><<<dim3((unsigned)((D + 31) / 32), (unsigned)n), 256, 0, s>>>(a);
    *queued += 1;
    e = cudaGetLastError();
  } else if (vec) {
    constexpr int kMore = kV == 4 ? 8 : 4;
    if (aligned)
      e = sh.per == 1   ? run(k_rms_grad<T, kV, 1, false>)
          : sh.per == 4 ? run(k_rms_grad<T, kV, 4, false>)
                        : run(k_rms_grad<T, kV, kMore, false>);
    else
      e = sh.per == 1   ? run(k_rms_grad<T, kV, 1, true>)
          : sh.per == 4 ? run(k_rms_grad<T, kV, 4, true>)
                        : run(k_rms_grad<T, kV, kMore, true>);
  } else {
    e = sh.per == 1   ? run(k_rms_grad<T, 1, 1, false>)
        : sh.per == 4 ? run(k_rms_grad<T, 1, 4, false>)
                      : run(k_rms_grad<T, 1, 16, false>);
  }
  if (e != cudaSuccess) return e;
  *queued += 2;
  return launch_sum_rows(h, a.scratch, n, D, a.grad_weight.data, a.grad_weight.type, s);
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

cudaError_t launch_sum_rows(const ss_handle *h, const float *part, int64_t n, int64_t cols, void *out, int32_t type, cudaStream_t s,
                            bool beside) {
  if (cols / 32 >= h->sm_count / 2) return launch_beside(k_sum_rows<32>, (unsigned)((cols + 31) / 32), 1024, 0, s, beside, part, n, cols, out, type);
  return launch_beside(k_sum_rows<8>, (unsigned)((cols + 7) / 8), 1024, 0, s, beside, part, n, cols, out, type);
}

int64_t rms_grad_scratch(const ss_handle *h, int64_t R, int64_t D) {
  return R > 0 ? most_parts(h, R) * D * (int64_t)sizeof(float) : 0;
}

static int64_t kept_total_at(const ss_handle *h, int64_t R, int64_t D) {
  return (rms_grad_scratch(h, R, D) + SS_SCRATCH_ALIGN - 1) / SS_SCRATCH_ALIGN * SS_SCRATCH_ALIGN;
}
int64_t rms_kept_grad_scratch(const ss_handle *h, int64_t R, int64_t D, int32_t type) {
  return D <= kKeptMost ? rms_grad_scratch(h, R, D) : kept_total_at(h, R, D) + R * ((D + 15) / 16 * 16) * size_of(type);
}

cudaError_t launch_rms_norm_grad(ss_handle *h, const rms_grad_args &given, cudaStream_t s, int *queued) {
  *queued = 0;
  rms_grad_args a = given;
  if (a.total_kept.codes && a.total.n_cols <= kKeptMost) {
    switch (a.total.type) {
      case SS_VALUES_F32:
        return rms_grad_kept_typed<float>(h, a, s, queued);
      case SS_VALUES_BF16:
        return rms_grad_kept_typed<__nv_bfloat16>(h, a, s, queued);
      default:
        return rms_grad_kept_typed<__half>(h, a, s, queued);
    }
  }
  if (a.total_kept.codes) {
    const int64_t R = a.total.n_rows, D = a.total.n_cols;
    a.total.data = reinterpret_cast<unsigned char *>(a.scratch) + kept_total_at(h, R, D);
    a.total.ld = (D + 15) / 16 * 16;
    const cudaError_t e = launch_expand(a.total_kept, a.total, s, queued);
    if (e != cudaSuccess) return e;
  }
  switch (a.total.type) {
    case SS_VALUES_F32:
      return rms_grad_typed<float>(h, a, s, queued);
    case SS_VALUES_BF16:
      return rms_grad_typed<__nv_bfloat16>(h, a, s, queued);
    default:
      return rms_grad_typed<__half>(h, a, s, queued);
  }
}
