// Linear layers: y = act((x w^T) sx sw^T + b) + r, and their gradients.
//
//   z = (x w^T) sx[m] sw[n] + b[n],   y = act(z) + r,   pre = z if kept
//   gz = grad_y act'(pre),  grad_x = gz w,  grad_w = gz^T x,  grad_b = sum gz
//
// x [M, K] and w [N, K] hold bf16, fp16 or e4m3 values (one scale a row then);
// products are exact and summed in float32, the epilogue is float32, and each
// output is rounded once.  gz is rounded to the inputs' type, as the tensor
// cores take it.
//
// Many rows (k_product_pair): bound by the tensor cores.  D = A B^T by tiles
// of 256 x 256, a pair of blocks a tile: each holds half of A's rows and half
// of B's in shared memory and its rows' sums in tensor memory, twice, so that
// one tile's epilogue runs beside the next one's products.  Operands arrive by
// tensor copies in the 128-byte swizzle through a ring of stages; one warp
// copies, one thread issues the products, sixteen warps run the epilogue and
// store by tensor copies.  Measured, 8192 x 4096 x 4096 bf16, ten calls after a
// pause: 151 us alone (1,820 TFLOP/s; cuBLAS on the same card 144), 173 us with
// bias, gelu, residual and kept pre-activation (the last tiles' epilogue and the
// 200 MB of it); 5000 x 10000 x 2048 e4m3: 84 us.  8192 x 4096 x 1024 with bias
// and gelu 56 us, 63 with the pre-activation kept in 16 bits and 71 in 8.
//
// Fewer tiles than that fills (k_product): blocks on their own with tiles of
// 128 x kBN, the summed dimension split over a cluster of up to 8 of them
// where there are few, which add their tiles through each other's shared
// memory in a fixed order.  With few rows the sides are swapped, A = w and B =
// x, so that 128 features fill the tile's rows and few columns are spent on
// rows that do not exist; then reading w is the bound.  16 x 4096 x 4096 e4m3:
// 9.4 us a call, most of it latency (set-up, first copies, exchange).
// cut_of chooses by estimated time.
//
// The three products of a layer differ in which operand runs along the summed
// dimension: x w^T has both rows contiguous in it (K-major), gz w has w
// contiguous across it, and gz^T x both (MN-major); the copies and descriptors
// take either, so nothing is transposed in memory.  A gradient's two products go
// into one launch (gradients.cu) where that is estimated to end sooner: 8192 x
// 4096 x 1024 bf16 95 us, where one after the other they took 56 and 52.
//
// One row, two of 16 bits (k_rows): a warp takes whole rows of w with 16-byte loads and
// ordinary multiply-adds, no tile to fill.  One row, 65,536 features of 1024
// bf16: 25.7 us (5.2 TB/s).
//
// Rows that do not start on 16-byte boundaries, which tensor copies cannot
// take, are first copied into scratch with padded rows.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>
#include <mutex>
#include <type_traits>

#include "kept.cuh"
#include "product.cuh"

namespace {

using namespace dense;

constexpr int kEpiFew = 8;        // epilogue warps of a block on its own, two for each 32 tensor-memory lanes
constexpr int kThreads = 64 + 32 * kEpiFew;  // copy warp, product warp, epilogue

// ---------------------------------------------------------------- activations
// The normal distribution function Phi and e = exp(-z^2 / 2).  For x = |z| / sqrt 2,
// erfc(x) exp(x^2) / t with t = 1 / (1 + 0.43 x) is smooth over t in (0, 1] and
// near a polynomial: the one below (its minimax fit in relative error, of degree
// 7, over x up to 9.4, past which e is 0; with the 1/2 of Phi in it) is within
// 8.4e-8 of it.  So Phi of a negative z is accurate relative to itself, within
// (1.25 z^2 + 24) 2^-24, most of it the rounding of z^2.  One exponential serves
// the gelu's slope as well: with erff and expf the gradient's pass over 8192 x
// 4096 values took 72 us where one exponential took 45.
__device__ __forceinline__ float normal_cdf(float z, float &e) {
  float t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.304055929f, fabsf(z), 1.0f)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * z * -0.72134752044448170f));
  float poly = fmaf(t, 0.0368539476f, -0.155186636f);
  poly = fmaf(t, poly, 0.191852769f);
  poly = fmaf(t, poly, -0.0428628107f);
  poly = fmaf(t, poly, 0.12342219f);
  poly = fmaf(t, poly, 0.102475558f);
  poly = fmaf(t, poly, 0.12218772f);
  poly = fmaf(t, poly, 0.121257304f);
  const float tail = t * poly * e;
  return z > 0.0f ? 1.0f - tail : tail;
}

// The same for two values, one instruction for both where there is one: the same
// operations in the same order, so the same bits.
__device__ __forceinline__ Two normal_cdf2(Two z, Two &e) {
  const float2 f = both(z);
  float2 t, x;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(fmaf(0.304055929f, fabsf(f.x), 1.0f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(fmaf(0.304055929f, fabsf(f.y), 1.0f)));
  const float2 q = both(z * z * two(-0.72134752044448170f, -0.72134752044448170f));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x.x) : "f"(q.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x.y) : "f"(q.y));
  e = two(x.x, x.y);
  const Two u = two(t.x, t.y);
  auto same = [](float c) { return two(c, c); };
  Two poly = fma_of(u, same(0.0368539476f), same(-0.155186636f));
  poly = fma_of(u, poly, same(0.191852769f));
  poly = fma_of(u, poly, same(-0.0428628107f));
  poly = fma_of(u, poly, same(0.12342219f));
  poly = fma_of(u, poly, same(0.102475558f));
  poly = fma_of(u, poly, same(0.12218772f));
  poly = fma_of(u, poly, same(0.121257304f));
  const Two tail = u * poly * e;
  const float2 low = both(tail), high = both(fma_of(tail, same(-1.0f), same(1.0f)));
  return two(f.x > 0.0f ? high.x : low.x, f.y > 0.0f ? high.y : low.y);
}

// (1 + tanh u) / 2 with u = sqrt(2 / pi) (z + 0.044715 z^3), as 1 / (1 + exp(-2 u)):
// 1 + tanh u itself is the difference of two values near 1 where z is negative.
__device__ __forceinline__ float tanh_share(float z) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-z * fmaf(z * z, 0.10294324f, 2.30220818f)));  // 2 log2(e) sqrt(2 / pi) = 2.3022
  return __fdividef(1.0f, 1.0f + e);
}

template <int kAct>
__device__ __forceinline__ float act_of(float z) {
  if (kAct == SS_ACT_RELU) return z > 0.0f ? z : (z == z ? 0.0f : z);
  if (kAct == SS_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  if (kAct == SS_ACT_GELU_TANH) return z * tanh_share(z);
  if (kAct == SS_ACT_SILU) return __fdividef(z, 1.0f + __expf(-z));  // an IEEE quotient's slow path orders the values: 128 cycles each
  if (kAct == SS_ACT_LOG1P_RELU) return z > 0.0f ? log1pf(z) : (z == z ? 0.0f : z);
  return z;
}
__device__ __forceinline__ float act_any(int32_t act, float z) {
  switch (act) {
    case SS_ACT_RELU: return act_of<SS_ACT_RELU>(z);
    case SS_ACT_GELU: return act_of<SS_ACT_GELU>(z);
    case SS_ACT_GELU_TANH: return act_of<SS_ACT_GELU_TANH>(z);
    case SS_ACT_SILU: return act_of<SS_ACT_SILU>(z);
    case SS_ACT_LOG1P_RELU: return act_of<SS_ACT_LOG1P_RELU>(z);
    default: return z;
  }
}
// act'(z); 0 at the kink of the rectified ones.
template <int kAct>
__device__ __forceinline__ float act_slope(float z) {
  if (kAct == SS_ACT_RELU) return z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
  if (kAct == SS_ACT_GELU) {
    float e;
    const float cdf = normal_cdf(z, e);
    return fmaf(z * 0.39894228040143268f, e, cdf);
  }
  if (kAct == SS_ACT_GELU_TANH) {
    if (fabsf(z) > 1e4f) return z > 0.0f ? 1.0f : 0.0f;  // where z^2 could overflow
    const float s = tanh_share(z);
    return s + z * s * (1.0f - s) * 1.5957691216057308f * (1.0f + 0.134145f * z * z);
  }
  if (kAct == SS_ACT_SILU) {
    const float s = 1.0f / (1.0f + __expf(-z));  // __fdividef gives 0 where the sum is past 2^126
    return s * (1.0f + z * (1.0f - s));
  }
  if (kAct == SS_ACT_LOG1P_RELU) return z > 0.0f ? 1.0f / (1.0f + z) : (z == z ? 0.0f : z);
  return 1.0f;
}

// ---------------------------------------------------------------- epilogue
// What follows the product, for output rows m and features n.
struct Epilogue {
  ss_dense y, pre, residual;
  const float *row_scale, *col_scale, *bias;
  int32_t act;
  int32_t vec;  // y, pre and residual rows start on 16-byte boundaries
  ss_kept keep;   // in pre's place, or null codes; by kernels of their own (their code cost the others registers)
};
__device__ __forceinline__ float read_any(const ss_dense &m, int64_t i) {
  return m.type == SS_VALUES_F32    ? static_cast<const float *>(m.data)[i]
         : m.type == SS_VALUES_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(m.data)[i])
                                    : __half2float(static_cast<const __half *>(m.data)[i]);
}
__device__ __forceinline__ void write_any(const ss_dense &m, int64_t i, float v) {
  if (m.type == SS_VALUES_F32)
    static_cast<float *>(m.data)[i] = v;
  else if (m.type == SS_VALUES_BF16)
    static_cast<__nv_bfloat16 *>(m.data)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half *>(m.data)[i] = __float2half_rn(v);
}
__device__ __forceinline__ void finish_one(const Epilogue &ep, int64_t m, int64_t n, float v) {
  if (ep.row_scale) v = v * ep.row_scale[m] * ep.col_scale[n];  // one after the other: their product may leave float32's range
  if (ep.bias) v += ep.bias[n];
  if (ep.pre.data) write_any(ep.pre, m * ep.pre.ld + n, v);
  v = act_any(ep.act, v);
  if (ep.residual.data) v += read_any(ep.residual, m * ep.residual.ld + n);
  write_any(ep.y, m * ep.y.ld + n, v);
}
template <typename T>
__device__ __forceinline__ void write16(T *p, const float (&v)[16]) {
  constexpr int kV = Type<T>::kVec;
#pragma unroll
  for (int q = 0; q < 16 / kV; ++q) {
    float f[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) f[i] = v[q * kV + i];
    store_pack(p + q * kV, narrow<T, kV>(f));
  }
}
__device__ __forceinline__ void write16_any(const ss_dense &m, int64_t i, const float (&v)[16]) {
  if (m.type == SS_VALUES_F32)
    write16(static_cast<float *>(m.data) + i, v);
  else if (m.type == SS_VALUES_BF16)
    write16(static_cast<__nv_bfloat16 *>(m.data) + i, v);
  else
    write16(static_cast<__half *>(m.data) + i, v);
}
// 16 features n .. n + 15 of row m.
__device__ __forceinline__ void finish16(const Epilogue &ep, int64_t m, int64_t n, float (&v)[16]) {
  if (m >= ep.y.n_rows || n >= ep.y.n_cols) return;
  if (!ep.vec || n + 16 > ep.y.n_cols) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (n + i < ep.y.n_cols) finish_one(ep, m, n + i, v[i]);
    return;
  }
  if (ep.row_scale) {
    const float s = ep.row_scale[m];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = v[i] * s * ep.col_scale[n + i];
  }
  if (ep.bias) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += ep.bias[n + i];
  }
  if (ep.pre.data) write16_any(ep.pre, m * ep.pre.ld + n, v);
  if (ep.act != SS_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = act_any(ep.act, v[i]);
  }
  if (ep.residual.data) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += read_any(ep.residual, m * ep.residual.ld + n + i);
  }
  write16_any(ep.y, m * ep.y.ld + n, v);
}

// A box of 16-bit values, rows m0 .. m0 + 31 and columns n0 .. n0 + 31 of m, by
// loads of 16 bytes, four lanes along a row, or of one value, a row at a time,
// for rows that start anywhere or end in the box, into shared memory (box), by
// asynchronous copies where they are of 16 bytes: held in registers until it is
// added, it left too few for the rest (8192 x 4096 x 1024 bf16, gelu, residual and
// kept pre-activation: 87 us, so 70).  (A row a lane reads 16 bytes of each of 32
// lines at a time: a residual then cost 13 us of 170 at 8192 x 4096 x 4096.)
__device__ __forceinline__ void fetch_box(const ss_dense &m, bool whole, uint32_t box, int64_t m0, int64_t n0, int lane) {
  const uint16_t *p = static_cast<const uint16_t *>(m.data) + n0;
  if (whole) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = min(m0 + 8 * j + lane / 4, m.n_rows - 1);  // rows past the end are not used
      tc::copy_async<16>(unit_at(box, 8 * j + lane / 4, lane % 4), p + row * m.ld + lane % 4 * 8);
    }
  } else {
    uint16_t w[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) w[r] = n0 + lane < m.n_cols && m0 + r < m.n_rows ? p[(m0 + r) * m.ld + lane] : (uint16_t)0;
#pragma unroll
    for (int r = 0; r < 32; ++r) tc::write_shared(unit_at(box, r, lane / 8) + (uint32_t)(lane % 8 * 2), w[r]);
  }
}
// Adds the box's row `lane` to v.
template <typename T>
__device__ __forceinline__ void add_box(uint32_t box, int lane, float (&v)[32]) {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float f[8];
    widen(tc::read_shared<Pack<T, 8>>(unit_at(box, lane, j)), f);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * j + i] += f[i];
  }
  __syncwarp();
}
// A group of 32 values of each lane's row to codes and a scale, as compress has
// them of the float32 values.
__device__ __forceinline__ void keep32(const Epilogue &ep, int64_t m, int64_t n0, const float (&v)[32]) {
  const ss_kept &k = ep.keep;
  if (m >= k.n_rows) return;
  const bool whole = n0 + 32 <= k.n_cols;
  float top = 0.0f;  // NaN is left out by fmaxf, an infinity after it
  if (whole) {
#pragma unroll
    for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(v[i]));
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (n0 + i < k.n_cols) top = fmaxf(top, fabsf(v[i]));
  }
  const bool odd = top == INFINITY;
  uint32_t most = __float_as_uint(top);
  if (odd) {
    most = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (n0 + i < k.n_cols) most = max(most, finite_bits(v[i]));
  }
  const int e = exponent_of(most, least_exponent(ep.y.type));
  const float down = power_of(-e);
  uint8_t *to = static_cast<uint8_t *>(k.codes) + m * k.ld + n0;
  const bool wide = whole && (reinterpret_cast<uintptr_t>(to) & 15) == 0;
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float *f = v + 16 * part + 4 * j;
      w[j] = codes2(f[0] * down, f[1] * down) | codes2(f[2] * down, f[3] * down) << 16;
    }
    if (odd) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float *f = v + 16 * part + 4 * j;
        w[j] = codes2(scaled_down(f[0], down), scaled_down(f[1], down)) | codes2(scaled_down(f[2], down), scaled_down(f[3], down)) << 16;
      }
    }
    if (wide) {
      reinterpret_cast<uint4 *>(to)[part] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (n0 + 16 * part + i < k.n_cols) to[16 * part + i] = (uint8_t)(w[i / 4] >> i % 4 * 8);
    }
  }
  k.scale[m * k.ld_scale + n0 / kGroup] = (uint8_t)(e + 127);
}

template <int kAct>
__device__ __forceinline__ void act32(float (&v)[32]) {
  if constexpr (kAct == SS_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const Two z = two(v[i], v[i + 1]);
      Two e;
      const float2 y = both(z * normal_cdf2(z, e));
      v[i] = y.x;
      v[i + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = act_of<kAct>(v[i]);
  }
}

// 32 columns n0 .. of rows m0 + lane: everything that follows the product,
// from the accumulators at `acc`; `done` is called once they are read.  The
// warp's boxes: one for what goes out, one for the residual.  kFull: there may be
// a residual or a pre-activation to write; a kernel of its own for neither has
// the registers (8192 x 4096 x 1024 bf16, gelu: 57 us, in one for all 62).
template <bool kKeep, bool kFull, typename F>
__device__ __forceinline__ void finish32(const Epilogue &ep, const CUtensorMap *map_y, const CUtensorMap *map_pre, uint32_t boxes,
                                         int lane, int64_t m0, int64_t n0, uint32_t acc, F done) {
  const int64_t m = m0 + lane, M = ep.y.n_rows, N = ep.y.n_cols;
  const bool there = m0 < M && n0 < N, whole = ep.vec && n0 + 32 <= N;
  const bool by_box = kFull && there && ep.residual.data && ep.residual.type != SS_VALUES_F32;
  float v[32];
  {
    uint32_t r[32];
    tc::load_acc32(acc, r);
    if (by_box) fetch_box(ep.residual, whole, boxes + kStaging, m0, n0, lane);  // the rest hides the wait
    tc::load_acc_wait();
    done();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
  }
  if (!there) return;

  if (ep.row_scale) {
    const float s = m < M ? ep.row_scale[m] : 0.0f;
    along32(ep.col_scale + n0, N - n0, [&](int i, float f) { v[i] = v[i] * s * f; });
  }
  if (ep.bias) along32(ep.bias + n0, N - n0, [&](int i, float f) { v[i] += f; });
  if (kKeep)
    keep32(ep, m, n0, v);
  else if (kFull && ep.pre.data)
    put32<!kFull>(ep.pre, map_pre, ep.vec, boxes, lane, m0, n0, v);
  switch (ep.act) {
    case SS_ACT_RELU: act32<SS_ACT_RELU>(v); break;
    case SS_ACT_GELU: act32<SS_ACT_GELU>(v); break;
    case SS_ACT_GELU_TANH: act32<SS_ACT_GELU_TANH>(v); break;
    case SS_ACT_SILU: act32<SS_ACT_SILU>(v); break;
    case SS_ACT_LOG1P_RELU: act32<SS_ACT_LOG1P_RELU>(v); break;
    default: break;
  }
  if (by_box) {
    if (ep.residual.type == SS_VALUES_BF16)
      add_box<__nv_bfloat16>(boxes + kStaging, lane, v);
    else
      add_box<__half>(boxes + kStaging, lane, v);
  } else if (kFull && ep.residual.data && m < M) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (n0 + i < N) v[i] += read_any(ep.residual, m * ep.residual.ld + n0 + i);
  }
  put32<!kFull>(ep.y, map_y, ep.vec, boxes, lane, m0, n0, v);
}

// ---------------------------------------------------------------- products
struct Product {
  CUtensorMap a, b, y, pre;
  Epilogue ep;
  int64_t rows_a, rows_b;
  int32_t blocks_k;   // stages of the summed dimension
  int32_t tiles_a, tiles_b;
  int32_t swapped;    // A holds the features, B the rows
  uint32_t idesc;
  int32_t *status;
};

template <int kBN>
struct Ring {
  static constexpr int kBytesA = kTileM * kRowBytes, kBytesB = kBN * kRowBytes;
  static constexpr int kStage = kBytesA + kBytesB;
  // narrow tiles: short rings, so that two or three blocks an SM hide each
  // other's set-up and epilogue
  static constexpr int kStages = kBN == 16 ? 4 : kBN <= 64 ? 3 : (kSmemMost - 2048) / kStage;
  static constexpr int kSmem = kStages * kStage + 1024;  // + alignment to 1024
  static_assert((kBN + 1) * kTileM * 4 <= kStages * kStage, "a tile to exchange fits the ring");
  static_assert(2 * kEpiFew * kStaging <= kStages * kStage, "and so do the epilogue's boxes");
};

// One tile a cluster; its blocks take equal shares of the summed dimension.
template <int kBN, int kMajA, int kMajB, bool kF8, bool kKeep>
__global__ void __launch_bounds__(kThreads) k_product(const __grid_constant__ Product a) {
  using R = Ring<kBN>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t bars[2 * R::kStages + 1];
  __shared__ uint32_t tmem_slot;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = (tc::smem_u32(raw) + 1023u) & ~1023u;
  auto full = [&](int s) { return tc::smem_u32(&bars[s]); };
  auto empty = [&](int s) { return tc::smem_u32(&bars[R::kStages + s]); };
  const uint32_t done = tc::smem_u32(&bars[2 * R::kStages]);
  constexpr uint32_t kCols = kBN < 32 ? 32 : kBN;
  if (tid == 0) {
    for (int i = 0; i < 2 * R::kStages + 1; ++i) tc::bar_init(tc::smem_u32(&bars[i]), 1);
    tc::bar_init_fence();
    tc::prefetch_map(&a.a);
    tc::prefetch_map(&a.b);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(&tmem_slot)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;

  uint32_t split;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(split));
  const uint32_t rank = split > 1 ? tc::cluster_rank() : 0;
  const int64_t tile = blockIdx.x / split;
  // Tiles go down groups of 8 tile rows of A, so that the blocks of a wave
  // share both operands in L2.
  const int64_t group = 8ll * a.tiles_b, g0 = tile / group * 8, gh = min((int64_t)8, (int64_t)a.tiles_a - g0);
  const int64_t ta = g0 + (tile % group) % gh, tb = (tile % group) / gh;
  const int32_t row_a = (int32_t)(ta * kTileM), row_b = (int32_t)(tb * kBN);
  const int k0 = (int)((int64_t)a.blocks_k * rank / split), k1 = (int)((int64_t)a.blocks_k * (rank + 1) / split);
  const int n = k1 - k0;
  constexpr int kUnit = kF8 ? kRowBytes : kRowBytes / 2;  // values of the summed dimension a stage

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      for (; issued < n; ++issued) {
        const int s = issued % R::kStages, turn = issued / R::kStages;
        if (turn > 0 && !tc::bar_wait(empty(s), (uint32_t)((turn - 1) & 1), a.status)) break;
        tc::bar_expect(full(s), R::kStage);
        const int32_t k = (k0 + issued) * kUnit;
        const uint32_t sa = ring + (uint32_t)(s * R::kStage), sb = sa + R::kBytesA;
        if (kMajA == kMajorK) {
          tc::load_2d(sa, &a.a, k, row_a, full(s));
        } else {
#pragma unroll
          for (int i = 0; i < kTileM / 64; ++i) tc::load_2d(sa + i * 8192, &a.a, row_a + 64 * i, k, full(s));
        }
        if (kMajB == kMajorK) {
          tc::load_2d(sb, &a.b, k, row_b, full(s));
        } else {
#pragma unroll
          for (int i = 0; i < kBN / 64; ++i) tc::load_2d(sb + i * 8192, &a.b, row_b + 64 * i, k, full(s));
        }
      }
      // Every copy issued lands before the block goes on, also after a wait
      // that gave up: a stage's next copy is issued only once its previous
      // one was read, so at most the last copy of each stage is in flight.
      for (int s = 0; s < R::kStages; ++s) {
        const int m = (issued + R::kStages - 1 - s) / R::kStages;
        if (m > 0) tc::bar_wait(full(s), (uint32_t)((m - 1) & 1), a.status);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      for (int i = 0; i < n; ++i) {
        const int s = i % R::kStages;
        if (!tc::bar_wait(full(s), (uint32_t)((i / R::kStages) & 1), a.status)) break;
        tc::fence_after();
        const uint32_t sa = ring + (uint32_t)(s * R::kStage), sb = sa + R::kBytesA;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t da = kMajA == kMajorK ? tc::desc_128b(sa + 32 * j, 16, 1024) : tc::desc_128b(sa + 2048 * j, 8192, 1024);
          const uint64_t db = kMajB == kMajorK ? tc::desc_128b(sb + 32 * j, 16, 1024) : tc::desc_128b(sb + 2048 * j, 8192, 1024);
          tc::mma<kF8>(tmem, da, db, a.idesc, (i > 0 || j > 0) ? 1u : 0u);
        }
        tc::commit(empty(s));
      }
      tc::commit(done);
    }
  }
  __syncwarp();
  // All warps wait: shared memory is free for the exchange once the products
  // are done (they read every copy that landed).
  const bool ok = tc::bar_wait(done, 0, a.status);
  __syncthreads();
  tc::fence_after();

  const int q = warp & 3, r = q * 32 + lane;  // epilogue: tensor-memory lane, row of A in the tile
  const int half = (warp - 2) >> 2;           // which columns of it
  const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
  constexpr int kSlice = kBN / 2 < 16 ? 16 : kBN / 2;
  const int slice0 = half * kSlice, slice1 = min(kBN, slice0 + kSlice);  // none for the second of 16 columns
  if (split == 1) {
    if (warp >= 2 && ok) {
      if (a.swapped) {  // the lanes along the features
        for (int c = slice0; c < slice1; c += 16) {
          float v[16];
          tc::load_acc16(lanes + (uint32_t)c, v);
          if ((int64_t)row_a + r < a.rows_a) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if ((int64_t)row_b + c + i < a.rows_b) finish_one(a.ep, (int64_t)row_b + c + i, row_a + r, v[i]);
          }
        }
      } else if constexpr (kBN < 64) {
        for (int c = slice0; c < slice1; c += 16) {
          float v[16];
          tc::load_acc16(lanes + (uint32_t)c, v);
          finish16(a.ep, row_a + r, (int64_t)row_b + c, v);
        }
      } else {
        const uint32_t boxes = ring + (uint32_t)((warp - 2) * 2 * kStaging);
#pragma unroll 1
        for (int c = slice0; c < slice1; c += 32)
          finish32<kKeep, true>(a.ep, &a.y, &a.pre, boxes, lane, (int64_t)row_a + q * 32, (int64_t)row_b + c, lanes + (uint32_t)c, [] {});
        if (lane == 0) tc::store_wait_all();
      }
    }
  } else {
    // This block's share of the sum to shared memory, [column][row of A]
    // where the features are the rows of A, else [row of A][column + 1 pad]:
    // either way the features lie along the lanes below.
    constexpr int kPitch = kBN + 1;
    if (warp >= 2) {
      for (int c = slice0; c < slice1; c += 16) {
        float v[16];
        tc::load_acc16(lanes + (uint32_t)c, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int at = a.swapped ? (c + i) * kTileM + r : r * kPitch + c + i;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(ring + (uint32_t)at * 4), "f"(n > 0 ? v[i] : 0.0f) : "memory");
        }
      }
    }
    tc::cluster_sync();
    if (warp >= 2 && ok) {
      if (a.swapped) {
        const int c0 = (int)(kBN * rank / split), c1 = (int)(kBN * (rank + 1) / split);
        for (int c = c0 + half; c < c1; c += 2) {
          const int64_t ra = (int64_t)row_a + r, rb = (int64_t)row_b + c;
          if (rb >= a.rows_b) break;
          float v = 0.0f;
          for (uint32_t p = 0; p < split; ++p) v += tc::load_remote(ring + (uint32_t)(c * kTileM + r) * 4, p);
          if (ra < a.rows_a) finish_one(a.ep, rb, ra, v);
        }
      } else {
        const int rows = kTileM / (int)split;
        for (int i = warp - 2; i < rows; i += kEpiFew) {
          const int row = rows * (int)rank + i;
          if ((int64_t)row_a + row >= a.rows_a) break;
          for (int c = lane; c < kBN && (int64_t)row_b + c < a.rows_b; c += 32) {
            float v = 0.0f;
            for (uint32_t p = 0; p < split; ++p) v += tc::load_remote(ring + (uint32_t)(row * kPitch + c) * 4, p);
            finish_one(a.ep, (int64_t)row_a + row, (int64_t)row_b + c, v);
          }
        }
      }
    }
    tc::cluster_sync();  // no block leaves while another reads its tile
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
  }
}

// ---------------------------------------------------------------- products by pairs of blocks
struct PairProduct {
  CUtensorMap a, b, y, pre;
  Epilogue ep;
  int32_t blocks_k, tiles_a, tiles_b;
  uint32_t idesc;
  int32_t *status;
};

// Persistent: each pair of blocks takes every n-th tile of 256 x kBN.
template <int kBN, int kMajA, int kMajB, bool kF8, bool kKeep, bool kFull>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_product_pair(const __grid_constant__ PairProduct a) {
  const int lane = threadIdx.x & 31;
  const int64_t rank_rows = (int64_t)tc::cluster_rank() * kTileM;
  pair_products<kBN, kMajA, kMajB, kF8, 2>(
      &a.a, &a.b, &a.idesc, a.status, TileWalk<PairProduct>{a, (int32_t)(blockIdx.x / 2)},
      [&](const TileWalk<PairProduct> &, const Tile &t, int q, int quarter, uint32_t acc, uint32_t boxes, auto release) {
        const int64_t m0 = (int64_t)t.ta * 2 * kTileM + rank_rows + q * 32;
#pragma unroll 1
        for (int c = quarter * (kBN / 4); c < (quarter + 1) * (kBN / 4); c += 32) {
          const bool last = c + 32 == (quarter + 1) * (kBN / 4);
          finish32<kKeep, kFull>(a.ep, &a.y, &a.pre, boxes, lane, m0, (int64_t)t.tb * kBN + c, acc + (uint32_t)c, [&] {
            if (last) release();
          });
        }
      });
}

// ---------------------------------------------------------------- few rows
template <typename T, int kN>
__device__ __forceinline__ void read_vec(const T *p, float (&f)[kN]) {
  if constexpr (sizeof(T) == 1) {
    const Pack<uint8_t, kN> q = *reinterpret_cast<const Pack<uint8_t, kN> *>(p);
    if constexpr (kN == 1) {
      f[0] = __half2float(__half(__nv_cvt_fp8_to_halfraw(q.v[0], __NV_E4M3)));
    } else {
      Pack<uint16_t, kN / 2> two;
      memcpy(&two, &q, sizeof(two));
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two.v[i], __NV_E4M3)));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    }
  } else {
    widen(load_pack<T, kN>(p), f);
  }
}

constexpr int kRowWarps = 2;
// A warp takes kW features and, in turns, kM rows of x; kN values a load.  Small
// blocks, so that a finished warp's place is filled soon, and for one row 32
// warps an SM (65,536 features of 1024 bf16: 25.7 us; blocks of eight warps
// with the registers they like, 24 warps an SM, 28.5 us).
template <typename T, int kM, int kW, int kN>
__global__ void __launch_bounds__(32 * kRowWarps, kM == 1 ? 16 : 1) k_rows(const ss_dense x, const ss_dense w, const Epilogue ep) {
  const int lane = threadIdx.x & 31;
  const int64_t n0 = ((int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5)) * kW;
  const int64_t N = w.n_rows, M = x.n_rows, K = x.n_cols;
  if (n0 >= N) return;
  const T *xp = static_cast<const T *>(x.data), *wp = static_cast<const T *>(w.data);
  for (int64_t m0 = (int64_t)blockIdx.y * kM; m0 < M; m0 += (int64_t)gridDim.y * kM) {
    float sum[kW][kM];
#pragma unroll
    for (int j = 0; j < kW; ++j)
#pragma unroll
      for (int m = 0; m < kM; ++m) sum[j][m] = 0.0f;
#pragma unroll(kW == 1 ? 8 : 2)
    for (int64_t k = (int64_t)lane * kN; k < K; k += 32 * kN) {
      float xv[kM][kN], wv[kW][kN];
#pragma unroll
      for (int j = 0; j < kW; ++j) read_vec<T, kN>(wp + min(n0 + j, N - 1) * w.ld + k, wv[j]);
#pragma unroll
      for (int m = 0; m < kM; ++m) read_vec<T, kN>(xp + min(m0 + m, M - 1) * x.ld + k, xv[m]);
#pragma unroll
      for (int j = 0; j < kW; ++j)
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int i = 0; i < kN; ++i) sum[j][m] = fmaf(wv[j][i], xv[m][i], sum[j][m]);
    }
    float mine = 0.0f;
#pragma unroll
    for (int j = 0; j < kW; ++j)
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const float v = warp_sum(sum[j][m]);
        if (lane == j * kM + m) mine = v;
      }
    if (lane < kW * kM) {
      const int64_t n = n0 + lane / kM, m = m0 + lane % kM;
      if (n < N && m < M) finish_one(ep, m, n, mine);
    }
  }
}

// ---------------------------------------------------------------- gradients
// gz = grad_y act'(pre) into gz[M][ld] (or nowhere), and the sums of its
// columns over the block's rows into part[blockIdx.y][N] (or nowhere).  A warp
// takes every eighth row of the block's share, two of them at a time.  Bound
// by memory and, with a gelu, by instructions: 8192 x 4096 bf16 36 us (5.5 TB/s),
// from codes 40, at four blocks an SM: some activations spill 4 to 36 bytes of a
// thread's then, which costs less than three blocks do (the whole gradient of 8192
// x 4096 x 1024 fp16 with gelu_tanh or log1p_relu 140 us, at three 145 and 147).
// kAny: rows that start anywhere, or end within a unit of kN values.
template <typename T, int kAct, bool kKept, bool kAny>
__global__ void __launch_bounds__(256, kAny ? 1 : 4) k_act_grad(const ss_dense grad_y, const ss_dense pre, const ss_kept kept, T *gz, int64_t ld, float *part) {
  constexpr int kN = 8;
  tc::let_next();
  __shared__ float sm[8][32 * kN + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t M = grad_y.n_rows, N = grad_y.n_cols, c = ((int64_t)blockIdx.x * 32 + lane) * kN;
  const int64_t step = (int64_t)gridDim.y * 8, first = (int64_t)blockIdx.y * 8 + warp;
  const T *gp = static_cast<const T *>(grad_y.data) + first * grad_y.ld + c;
  const T *zp = static_cast<const T *>(pre.data) + (kAct != SS_ACT_NONE && !kKept ? first * pre.ld + c : 0);
  const uint8_t *codes = static_cast<const uint8_t *>(kept.codes) + (kKept ? first * kept.ld + c : 0);
  const uint8_t *scale = kept.scale + (kKept ? first * kept.ld_scale + c / kGroup : 0);
  const void *end_g = end_of(grad_y.data, M, N, grad_y.ld, sizeof(T)), *end_z = end_of(pre.data, M, N, pre.ld, sizeof(T));
  const void *end_c = end_of(kept.codes, M, N, kept.ld, 1);
  const int left = (int)min((int64_t)kN, N - c);
  T *to = gz ? gz + first * ld + c : nullptr;
  const int64_t step_g = step * grad_y.ld, step_z = step * pre.ld, step_c = step * kept.ld, step_s = step * kept.ld_scale, step_to = step * ld;
  float sum[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) sum[i] = 0.0f;
  if (c < N)
    for (int64_t m = first; m < M; m += 2 * step) {
      Pack<T, kN> gv[2], zv[2];
      Codes<kN> cv[2];
      uint32_t byte[2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (m + u * step < M) {
          if (kAny)
            load_anywhere<16, 2>(gp + u * step_g, grad_y.data, end_g, gv[u].w);
          else
            gv[u] = load_pack<T, kN>(gp + u * step_g);
          if (kKept) {
            if (kAny)
              load_anywhere<8, 1>(codes + u * step_c, kept.codes, end_c, cv[u].w);
            else
              cv[u].load(codes + u * step_c);
            byte[u] = scale[u * step_s];
          } else if (kAct != SS_ACT_NONE) {
            if (kAny)
              load_anywhere<16, 2>(zp + u * step_z, pre.data, end_z, zv[u].w);
            else
              zv[u] = load_pack<T, kN>(zp + u * step_z);
          }
        }
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (m + u * step < M) {
          float g[kN], z[kN];
          widen(gv[u], g);
          if (kKept) {
            const float s = scale_of_byte(byte[u]);
#pragma unroll
            for (int i = 0; i < kN; i += 2) {
              const float2 f = cv[u].pair(i / 2), q = both(two(f.x, f.y) * two(s, s));
              z[i] = q.x;
              z[i + 1] = q.y;
            }
            if (!exact_byte<T>(byte[u])) {
#pragma unroll
              for (int i = 0; i < kN; ++i) z[i] = as_type<T>(z[i]);
            }
          } else if (kAct != SS_ACT_NONE) {
            widen(zv[u], z);
          }
          if (kAny && left < kN) {  // what lies past the row's end
#pragma unroll
            for (int i = 0; i < kN; ++i)
              if (i >= left) g[i] = z[i] = 0.0f;
          }
          if constexpr (kAct == SS_ACT_GELU) {
#pragma unroll
            for (int i = 0; i < kN; i += 2) {
              const Two zz = two(z[i], z[i + 1]);
              Two ex;
              const Two cdf = normal_cdf2(zz, ex);
              const Two slope = fma_of(zz * two(0.39894228040143268f, 0.39894228040143268f), ex, cdf);
              const float2 q = both(two(g[i], g[i + 1]) * slope);
              g[i] = q.x;
              g[i + 1] = q.y;
            }
          } else if constexpr (kAct != SS_ACT_NONE) {
#pragma unroll
            for (int i = 0; i < kN; ++i) g[i] *= act_slope<kAct>(z[i]);
          }
          if (to) store_pack(to + u * step_to, narrow<T, kN>(g));
#pragma unroll
          for (int i = 0; i < kN; ++i) sum[i] += g[i];
        }
      gp += 2 * step_g;
      zp += 2 * step_z;
      codes += 2 * step_c;
      scale += 2 * step_s;
      if (to) to += 2 * step_to;
    }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < kN; ++i) sm[warp][i * 32 + lane] = sum[i];
  __syncthreads();
  for (int t = threadIdx.x; t < 32 * kN; t += 256) {
    float v = 0.0f;
    for (int k = 0; k < 8; ++k) v += sm[k][t];
    const int64_t col = ((int64_t)blockIdx.x * 32 + t % 32) * kN + t / 32;
    if (col < N) part[(int64_t)blockIdx.y * N + col] = v;
  }
}

// Copies of matrices into rows of ld values that start on 16-byte boundaries,
// one of them each blockIdx.y.
struct Copies {
  ss_dense src[2];
  void *dst[2];
  int64_t ld[2];
};
template <typename T>
__global__ void __launch_bounds__(256, 6) k_copy_rows(const Copies a) {
  tc::let_next();
  const bool second = blockIdx.y == 1;
  const ss_dense src = second ? a.src[1] : a.src[0];
  const int64_t ld = (second ? a.ld[1] : a.ld[0]) * (int64_t)sizeof(T), bytes = src.n_cols * (int64_t)sizeof(T);
  unsigned char *dst = static_cast<unsigned char *>(second ? a.dst[1] : a.dst[0]);
  const unsigned char *from = static_cast<const unsigned char *>(src.data);
  const void *end = end_of(from, src.n_rows, src.n_cols, src.ld, sizeof(T));
  auto read = [&](int64_t r, int64_t c) {
    uint32_t v[4];
    load_anywhere<16, (int)sizeof(T)>(from + r * src.ld * (int64_t)sizeof(T) + c, from, end, v);
    return make_uint4(v[0], v[1], v[2], v[3]);
  };
  // What lies past a row's end within its last 16 bytes goes along: no one reads
  // it there.  blockDim.x threads along a row, blockDim.y rows
  for (int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; r < src.n_rows; r += (int64_t)gridDim.x * blockDim.y)
    for (int64_t c = (int64_t)threadIdx.x * 16; c < bytes; c += 2 * 16 * (int64_t)blockDim.x) {  // two loads under way at a time
      const int64_t c1 = c + 16 * (int64_t)blockDim.x;
      const uint4 v0 = read(r, c);
      uint4 v1;
      if (c1 < bytes) v1 = read(r, c1);
      *reinterpret_cast<uint4 *>(dst + r * ld + c) = v0;
      if (c1 < bytes) *reinterpret_cast<uint4 *>(dst + r * ld + c1) = v1;
    }
  tc::wait_before();  // what follows waits for this kernel, and so for the one before it
}

// ---------------------------------------------------------------- host side
// Each matrix itself, or its copy with padded rows at *scratch (advanced past
// it); one launch, beside the end of the one before where `beside`.
cudaError_t aligned_rows(ss_handle *h, std::initializer_list<ss_dense *> ms, unsigned char **scratch, cudaStream_t s, int *queued,
                         bool beside = false) {
  Copies a = {};
  int n = 0;
  int64_t rows = 0, units = 1;
  bool bytes = false;
  for (ss_dense *m : ms) {
    if (rows_aligned(*m, 16)) continue;
    a.src[n] = *m;
    a.dst[n] = *scratch;
    a.ld[n] = padded_ld(*m);
    bytes = size_of(m->type) == 1;
    rows = std::max(rows, m->n_rows);
    units = std::max(units, (m->n_cols * size_of(m->type) + 15) / 16);
    m->data = *scratch;
    m->ld = a.ld[n++];
    *scratch += align_up(m->n_rows * m->ld * size_of(m->type));
  }
  if (n == 0) return cudaSuccess;
  unsigned x = 8;
  while (x < 256 && 2 * (int64_t)x < units) x *= 2;
  const unsigned y = 256 / x;
  cudaLaunchConfig_t cfg = {};
  // as many blocks as run at once: with 16 an SM the copy took half as long again
  cfg.gridDim = dim3((unsigned)std::min<int64_t>((rows + y - 1) / y, 6 * (int64_t)std::max(1, h->sm_count)), (unsigned)n);
  cfg.blockDim = dim3(x, y);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = beside ? 1 : 0;
  *queued += 1;
  return bytes ? cudaLaunchKernelEx(&cfg, k_copy_rows<uint8_t>, a) : cudaLaunchKernelEx(&cfg, k_copy_rows<uint16_t>, a);
}

template <int kBN, int kMajA, int kMajB, bool kF8>
cudaError_t run_product(Product &p, int split, cudaStream_t s) {
  auto kernel = k_product<kBN, kMajA, kMajB, kF8, false>;
  if constexpr (kBN >= 64 && kMajA == kMajorK && kMajB == kMajorK)
    if (p.ep.keep.codes) kernel = k_product<kBN, kMajA, kMajB, kF8, true>;
  cudaError_t e = ensure_dyn_smem(kernel, Ring<kBN>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.tiles_a * p.tiles_b * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Ring<kBN>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int kBN, int kMajA, int kMajB, bool kF8>
cudaError_t run_pair(ss_handle *h, PairProduct &p, cudaStream_t s) {
  auto kernel = k_product_pair<kBN, kMajA, kMajB, kF8, false, false>;
  if constexpr (kMajA == kMajorK && kMajB == kMajorK) {
    if (p.ep.keep.codes)
      kernel = k_product_pair<kBN, kMajA, kMajB, kF8, true, true>;
    else if (p.ep.pre.data || p.ep.residual.data)
      kernel = k_product_pair<kBN, kMajA, kMajB, kF8, false, true>;
  }
  cudaError_t e = ensure_dyn_smem(kernel, PairRing<kBN, 2>::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)p.tiles_a * p.tiles_b;
  const int64_t pairs = std::min<int64_t>(tiles, std::max(1, h->sm_count / 2));
  kernel<<<(unsigned)(2 * pairs), kPairThreads, PairRing<kBN, 2>::kSmem, s>>>(p);
  return cudaGetLastError();
}

template <int kBN>
cudaError_t product_pair(ss_handle *h, const ss_dense &A, int majA, const ss_dense &B, int majB, const Epilogue &ep,
                         int64_t rows_a, int64_t rows_b, int64_t K, cudaStream_t s) {
  const bool f8 = A.type == SS_VALUES_F8;
  const int unit = f8 ? kRowBytes : kRowBytes / 2;
  PairProduct p = {};
  p.ep = ep;
  p.status = h->d_status;
  p.blocks_k = (int32_t)((K + unit - 1) / unit);
  p.tiles_a = (int32_t)((rows_a + 2 * kTileM - 1) / (2 * kTileM));
  p.tiles_b = (int32_t)((rows_b + kBN - 1) / kBN);
  p.idesc = idesc_of(A, majA, majB, 2 * kTileM, kBN);
  cudaError_t e = majA == kMajorK ? encode(&p.a, A, unit, kTileM) : encode(&p.a, A, 64, unit);
  if (e == cudaSuccess) e = majB == kMajorK ? encode(&p.b, B, unit, kBN / 2) : encode(&p.b, B, 64, unit);
  if (e == cudaSuccess && ep.vec) e = encode_out(&p.y, ep.y);
  if (e == cudaSuccess && ep.vec && ep.pre.data) e = encode_out(&p.pre, ep.pre);
  if (e != cudaSuccess) return e;
  if (f8) return run_pair<kBN, kMajorK, kMajorK, true>(h, p, s);
  if (majA == kMajorK && majB == kMajorK) return run_pair<kBN, kMajorK, kMajorK, false>(h, p, s);
  if (majA == kMajorK) return run_pair<kBN, kMajorK, kMajorMN, false>(h, p, s);
  return run_pair<kBN, kMajorMN, kMajorMN, false>(h, p, s);
}

// How a product is cut: a tile's columns, the blocks that share its sum, and
// whether pairs of blocks take tiles of 256 x 256.
struct Cut {
  int bn, split;
  bool pair;
  double clocks;
};
// The cut of the least estimated time.  A stage of the summed dimension takes
// a pair 600 clocks (512 are the tensor cores' own), measured over 8192 x 4096
// x 4096, and a tile as long as its epilogue, 7,000, at least, as the next
// one's products run beside it; a block on its own takes its bytes at 85 a
// clock (128 x 256: 520 measured with rows along the sum, 610 across it), one
// after the other with its set-up, its epilogue and, for a split sum, the
// exchange.  It is an estimate: a tile of 5000 x 10000 x 2048 e4m3 takes 14,000
// clocks where it counts 9,600.
Cut cut_of(const ss_handle *h, int64_t rows_a, int64_t rows_b, int64_t blocks_k, int least, bool pairs, int most_split = 8) {
  const int64_t sms = std::max(1, h->sm_count);
  auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  Cut best = {256, 1, false, 0.0};
  best.pair = pairs;
  best.clocks = pairs ? 18e3 + (double)up(up(rows_a, 256) * up(rows_b, 256), std::max<int64_t>(1, sms / 2)) * std::max(600.0 * (double)blocks_k, 7e3) : 1e30;
  for (int bn = 256; bn >= least; bn /= 2) {
    if (bn < 256 && bn < 64 && rows_b > bn) break;  // narrow tiles: where they hold all of B's rows
    for (int split = 1; split <= (bn <= 128 ? most_split : 1) && (split == 1 || blocks_k / split >= 2); split *= 2) {
      // Blocks at a time: clusters stay within a group of SMs, and of 152 SMs 36
      // of 4 blocks and 15 of 8 run at once (of 456 places 110 and 51).
      const int64_t an_sm = bn <= 32 ? 3 : bn == 64 ? 2 : 1, places = sms * an_sm;
      const int64_t at_once = std::max<int64_t>(1, split == 8 ? places * (an_sm > 1 ? 17 : 15) / 19 : split == 4 ? places * 18 / 19 : places);
      const int64_t blocks = up(rows_a, kTileM) * up(rows_b, bn) * split;
      const double sharing = (double)std::min(an_sm, up(blocks, sms));
      // a matrix that one row of tiles reads once comes from memory, not L2
      const double rate = up(rows_a, kTileM) == 1 || up(rows_b, bn) == 1 ? 40.0 : 85.0;
      const double turns = (double)up(blocks, at_once);
      const double each = 5e3 + (split > 1 ? 5e3 + 80.0 * bn : 0.0) + 30.0 * bn / split + (double)up(blocks_k, split) * (kTileM + bn) * kRowBytes * sharing / rate;
      const double clocks = 4e3 + turns * each;
      if (clocks < best.clocks) best = {bn, split, false, clocks};
    }
  }
  return best;
}

// ep.y = the product of A and B over their summed dimension; A and B are
// [rows][summed] (kMajorK) or [summed][rows] (kMajorMN), rows aligned.
cudaError_t product(ss_handle *h, const ss_dense &A, int majA, const ss_dense &B, int majB, bool swapped, const Cut &cut,
                    const Epilogue &ep, cudaStream_t s, int *queued) {
  const bool f8 = A.type == SS_VALUES_F8;
  Product p = {};
  p.rows_a = majA == kMajorK ? A.n_rows : A.n_cols;
  p.rows_b = majB == kMajorK ? B.n_rows : B.n_cols;
  const int64_t K = majA == kMajorK ? A.n_cols : A.n_rows;
  p.ep = ep;
  p.swapped = swapped ? 1 : 0;
  p.status = h->d_status;
  const int unit = f8 ? kRowBytes : kRowBytes / 2;
  p.blocks_k = (int32_t)((K + unit - 1) / unit);
  if (cut.pair) {
    *queued += 1;
    return product_pair<256>(h, A, majA, B, majB, ep, p.rows_a, p.rows_b, K, s);
  }
  const int bn = cut.bn, split = cut.split;
  p.tiles_a = (int32_t)((p.rows_a + kTileM - 1) / kTileM);
  p.tiles_b = (int32_t)((p.rows_b + bn - 1) / bn);
  if ((int64_t)p.tiles_a * p.tiles_b * split > INT32_MAX) return cudaErrorInvalidConfiguration;
  p.idesc = idesc_of(A, majA, majB, kTileM, bn);
  cudaError_t e;
  e = majA == kMajorK ? encode(&p.a, A, unit, kTileM) : encode(&p.a, A, 64, unit);
  if (e != cudaSuccess) return e;
  e = majB == kMajorK ? encode(&p.b, B, unit, bn) : encode(&p.b, B, 64, unit);
  if (!swapped && split == 1 && bn >= 64 && ep.vec) {  // the epilogue that stores by tensor copies
    if (e == cudaSuccess) e = encode_out(&p.y, ep.y);
    if (e == cudaSuccess && ep.pre.data) e = encode_out(&p.pre, ep.pre);
  }
  if (e != cudaSuccess) return e;
  *queued += 1;
  if (f8) {
    switch (bn) {
      case 16: return run_product<16, kMajorK, kMajorK, true>(p, split, s);
      case 32: return run_product<32, kMajorK, kMajorK, true>(p, split, s);
      case 64: return run_product<64, kMajorK, kMajorK, true>(p, split, s);
      case 128: return run_product<128, kMajorK, kMajorK, true>(p, split, s);
      default: return run_product<256, kMajorK, kMajorK, true>(p, split, s);
    }
  }
  if (majA == kMajorK && majB == kMajorK) {
    switch (bn) {
      case 16: return run_product<16, kMajorK, kMajorK, false>(p, split, s);
      case 32: return run_product<32, kMajorK, kMajorK, false>(p, split, s);
      case 64: return run_product<64, kMajorK, kMajorK, false>(p, split, s);
      case 128: return run_product<128, kMajorK, kMajorK, false>(p, split, s);
      default: return run_product<256, kMajorK, kMajorK, false>(p, split, s);
    }
  }
  if (majA == kMajorK) {
    switch (bn) {
      case 64: return run_product<64, kMajorK, kMajorMN, false>(p, split, s);
      case 128: return run_product<128, kMajorK, kMajorMN, false>(p, split, s);
      default: return run_product<256, kMajorK, kMajorMN, false>(p, split, s);
    }
  }
  switch (bn) {
    case 64: return run_product<64, kMajorMN, kMajorMN, false>(p, split, s);
    case 128: return run_product<128, kMajorMN, kMajorMN, false>(p, split, s);
    default: return run_product<256, kMajorMN, kMajorMN, false>(p, split, s);
  }
}

// k_rows up to this many rows: two of 1024 bf16 against 65,536 take it 32 us and
// tiles 41, three 43 and 41; two of e4m3 26 and 20.  Other lengths and rows that
// start off 16 bytes go by the same rule, unmeasured.
int64_t few_rows_of(const ss_dense &x) { return x.type == SS_VALUES_F8 ? 1 : 2; }
constexpr int64_t kSwapRows = 256;  // features as A is looked at up to this many rows

template <typename T, int kN>
cudaError_t rows_typed(const ss_dense &x, const ss_dense &w, const Epilogue &ep, int sms, cudaStream_t s) {
  const int64_t M = x.n_rows, N = w.n_rows;
  auto run = [&](auto kernel, int m, int wide) {
    kernel<<<dim3((unsigned)((N + kRowWarps * wide - 1) / (kRowWarps * wide)), (unsigned)std::min<int64_t>(65535, (M + m - 1) / m)), 32 * kRowWarps, 0,
             s>>>(x, w, ep);
  };
  // one feature a warp where four leave less than 16 warps an SM
  if (M == 1 && N >= 64 * (int64_t)std::max(1, sms))
    run(k_rows<T, 1, 4, kN>, 1, 4);
  else if (M == 1)
    run(k_rows<T, 1, 1, kN>, 1, 1);
  else
    run(k_rows<T, 2, 2, kN>, 2, 2);
  return cudaGetLastError();
}

// Stages of a summed dimension of K values of m's type.
int64_t stages_of(const ss_dense &m, int64_t K) {
  const int unit = m.type == SS_VALUES_F8 ? kRowBytes : kRowBytes / 2;
  return (K + unit - 1) / unit;
}

bool few_rows(const ss_dense &x) { return x.n_rows <= few_rows_of(x) || x.n_cols == 0; }

int64_t grad_parts(const ss_handle *h, int64_t M, int64_t N) {
  const int64_t slabs = std::max<int64_t>(1, (N + 255) / 256);
  return std::max<int64_t>(1, std::min<int64_t>((M + 31) / 32, 8 * (int64_t)std::max(1, h->sm_count) / slabs));
}

// Whether a gradient's products take less time as one launch (gradients.cu) than
// as two, by their estimates, and that launch's scratch.  A tenth less is asked
// for, as large products at the power cap take longer together than estimated:
// 12,000 x 4096 x 4096 bf16 (estimates 0.915 to 1) 576 us and 526 apart, 6000 x 8192
// x 8192 (0.967) 1106 and 1036, where 8192 x 4096 x 1024 (0.87) takes 95 and 108.
bool together(const ss_handle *h, int64_t M, int64_t N, int64_t K, int64_t *parts) {
  int64_t clocks;
  *parts = grad_product_parts(h, M, N, K, &clocks);
  const double apart = cut_of(h, M, K, (N + 63) / 64, 64, true).clocks + cut_of(h, N, K, (M + 63) / 64, 64, true).clocks;
  return K > 0 && (double)clocks < 0.9 * apart;
}
int64_t together_bytes(const ss_handle *h, int64_t M, int64_t N, int64_t K) {
  int64_t parts;
  return together(h, M, N, K, &parts) && parts > 1 ? parts * grad_part_bytes(M, K) : 0;
}

}  // namespace

cudaError_t launch_aligned_rows(ss_handle *h, ss_dense *m, ss_dense *other, unsigned char **scratch, cudaStream_t s, int *queued) {
  int n = 0;
  cudaError_t e;
  if (other)
    e = aligned_rows(h, {m, other}, scratch, s, &n);
  else
    e = aligned_rows(h, {m}, scratch, s, &n);
  *queued += n;
  return e;
}

int64_t linear_scratch(const ss_handle *, const ss_dense &x, const ss_dense &w, bool keep) {
  return few_rows(x) && !keep ? 0 : copy_bytes(x) + copy_bytes(w);
}

int64_t linear_grad_scratch(const ss_handle *h, const ss_dense &grad_y, const ss_dense &x, const ss_dense &w,
                            int32_t act, bool x_kept) {
  const int64_t M = grad_y.n_rows, N = grad_y.n_cols;
  if (M == 0 || N == 0) return 0;  // the gradients are zeroed
  const bool own = act != SS_ACT_NONE || !rows_aligned(grad_y, 16);
  return (x_kept ? align_up(x.n_rows * padded_ld(x) * 2) : copy_bytes(x)) + copy_bytes(w) + together_bytes(h, M, N, x.n_cols) + (own ? align_up(M * padded_ld(grad_y) * size_of(grad_y.type)) : 0) +
         align_up(grad_parts(h, M, N) * N * (int64_t)sizeof(float));
}

cudaError_t launch_linear(ss_handle *h, const linear_args &a, cudaStream_t s, int *queued) {
  *queued = 0;
  if (a.y.n_rows == 0 || a.y.n_cols == 0) return cudaSuccess;
  Epilogue ep = {a.y, a.pre, a.residual, a.x_scale, a.w_scale, a.bias, a.activation, 0};
  auto aligned = [](const ss_dense &m) { return !m.data || rows_aligned(m, 16); };
  ep.vec = aligned(a.y) && aligned(a.pre) && aligned(a.residual);
  if (a.keep.codes) ep.keep = a.keep;
  if (few_rows(a.x) && !a.keep.codes) {
    *queued = 1;
    const int v = a.x.type == SS_VALUES_F8 ? 16 : 8;
    const bool vec = a.x.n_cols % v == 0 && rows_aligned(a.x, 16) && rows_aligned(a.w, 16);
    switch (a.x.type) {
      case SS_VALUES_F8:
        return vec ? rows_typed<uint8_t, 16>(a.x, a.w, ep, h->sm_count, s) : rows_typed<uint8_t, 1>(a.x, a.w, ep, h->sm_count, s);
      case SS_VALUES_BF16:
        return vec ? rows_typed<__nv_bfloat16, 8>(a.x, a.w, ep, h->sm_count, s) : rows_typed<__nv_bfloat16, 1>(a.x, a.w, ep, h->sm_count, s);
      default:
        return vec ? rows_typed<__half, 8>(a.x, a.w, ep, h->sm_count, s) : rows_typed<__half, 1>(a.x, a.w, ep, h->sm_count, s);
    }
  }
  ss_dense x = a.x, w = a.w;
  unsigned char *scratch = a.scratch;
  cudaError_t e;
  if ((e = aligned_rows(h, {&x, &w}, &scratch, s, queued)) != cudaSuccess) return e;
  const int64_t M = x.n_rows, N = w.n_rows, kb = stages_of(x, x.n_cols);
  if (a.keep.codes)  // whole groups of a row in a thread: tiles of 64 columns at least, their sums not split
    return product(h, x, kMajorK, w, kMajorK, false, cut_of(h, M, N, kb, 64, true, 1), ep, s, queued);
  const Cut cut = cut_of(h, M, N, kb, 16, true);
  if (M <= kSwapRows) {
    const Cut other = cut_of(h, N, M, kb, 16, false);
    if (other.clocks <= cut.clocks) return product(h, w, kMajorK, x, kMajorK, true, other, ep, s, queued);
  }
  return product(h, x, kMajorK, w, kMajorK, false, cut, ep, s, queued);
}

namespace {
template <typename T>
cudaError_t grad_typed(ss_handle *h, const linear_grad_args &a, cudaStream_t s, int *queued) {
  const int64_t M = a.grad_y.n_rows, N = a.grad_y.n_cols;
  cudaError_t e;
  unsigned char *scratch = a.scratch;
  ss_dense gz = a.grad_y, x = a.x, w = a.w;
  const bool own = a.activation != SS_ACT_NONE || !rows_aligned(a.grad_y, 16);
  if (own) {
    gz.ld = padded_ld(a.grad_y);
    gz.data = scratch;
    scratch += align_up(M * gz.ld * (int64_t)sizeof(T));
  }
  int64_t parts_x;
  // also where one of the two is left out: the other's bits are the same then
  const bool joint = together(h, M, N, x.n_cols, &parts_x);
  float *part = reinterpret_cast<float *>(scratch);
  const int64_t parts = grad_parts(h, M, N);
  scratch += align_up(parts * N * (int64_t)sizeof(float));
  if (own || a.grad_bias) {
    T *to = own ? static_cast<T *>(gz.data) : nullptr;
    float *sums = a.grad_bias ? part : nullptr;
    const bool kept = a.pre_kept.codes != nullptr;
    const bool vec = N % 8 == 0 && rows_aligned(a.grad_y, 16) && (!a.pre.data || rows_aligned(a.pre, 16)) && (!kept || kept_aligned(a.pre_kept, 8));
    auto run_of = [&](auto act, auto is_kept) {
      constexpr int kAct = decltype(act)::value;
      constexpr bool kKept = decltype(is_kept)::value;
      const dim3 grid((unsigned)((N + 255) / 256), (unsigned)parts);
      if (vec)
        k_act_grad<T, kAct, kKept, false><<<grid, 256, 0, s>>>(a.grad_y, a.pre, a.pre_kept, to, gz.ld, sums);
      else
        k_act_grad<T, kAct, kKept, true><<<grid, 256, 0, s>>>(a.grad_y, a.pre, a.pre_kept, to, gz.ld, sums);
    };
    auto run = [&](auto act) {
      if constexpr (decltype(act)::value != SS_ACT_NONE) {
        if (kept) return run_of(act, std::true_type());
      }
      run_of(act, std::false_type());
    };
    switch (a.activation) {
      case SS_ACT_RELU: run(std::integral_constant<int, SS_ACT_RELU>()); break;
      case SS_ACT_GELU: run(std::integral_constant<int, SS_ACT_GELU>()); break;
      case SS_ACT_GELU_TANH: run(std::integral_constant<int, SS_ACT_GELU_TANH>()); break;
      case SS_ACT_SILU: run(std::integral_constant<int, SS_ACT_SILU>()); break;
      case SS_ACT_LOG1P_RELU: run(std::integral_constant<int, SS_ACT_LOG1P_RELU>()); break;
      default: run(std::integral_constant<int, SS_ACT_NONE>()); break;
    }
    *queued += 1;
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (sums && !joint) {
      if ((e = launch_sum_rows(h, part, parts, N, a.grad_bias, SS_VALUES_F32, s)) != cudaSuccess) return e;
      *queued += 1;
    }
  }
  auto out = [](const ss_dense &m) {
    Epilogue ep = {};
    ep.y = m;
    ep.vec = rows_aligned(m, 16);
    return ep;
  };
  if (a.grad_x.data && (e = aligned_rows(h, {&w}, &scratch, s, queued, joint && *queued > 0)) != cudaSuccess) return e;
  if (a.grad_w.data) {
    if (a.x_kept.codes) {
      x.ld = padded_ld(x);
      x.data = scratch;
      scratch += align_up(x.n_rows * x.ld * (int64_t)sizeof(T));
      int n = 0;
      if ((e = launch_expand(a.x_kept, x, s, &n, joint && *queued > 0)) != cudaSuccess) return e;
      *queued += n;
    } else if ((e = aligned_rows(h, {&x}, &scratch, s, queued, joint && *queued > 0)) != cudaSuccess) {
      return e;
    }
  }
  if (joint) {
    grad_products g = {gz, w, x, a.grad_x, a.grad_w, reinterpret_cast<float *>(scratch), nullptr, (int32_t)parts_x, false, true, *queued > 0};
    if (a.grad_bias) {
      g.sums = part;
      g.sum_rows = parts;
      g.sum_cols = N;
      g.sum_to = a.grad_bias;
    }
    return launch_grad_products(h, g, s, queued);
  }
  if (a.grad_x.data &&
      (e = product(h, gz, kMajorK, w, kMajorMN, false, cut_of(h, M, x.n_cols, stages_of(gz, N), 64, true), out(a.grad_x), s, queued)) != cudaSuccess)
    return e;
  if (a.grad_w.data &&
      (e = product(h, gz, kMajorMN, x, kMajorMN, false, cut_of(h, N, x.n_cols, stages_of(gz, M), 64, true), out(a.grad_w), s, queued)) != cudaSuccess)
    return e;
  return cudaSuccess;
}

// Zeroes the rows of m (a sum over nothing).
cudaError_t zero(const ss_dense &m, cudaStream_t s) {
  if (!m.data || m.n_rows == 0 || m.n_cols == 0) return cudaSuccess;
  const size_t size = (size_t)size_of(m.type);
  return cudaMemset2DAsync(m.data, (size_t)m.ld * size, 0, (size_t)m.n_cols * size, (size_t)m.n_rows, s);
}
}  // namespace

cudaError_t launch_linear_grad(ss_handle *h, const linear_grad_args &a, cudaStream_t s, int *queued) {
  *queued = 0;
  const int64_t M = a.grad_y.n_rows, N = a.grad_y.n_cols, K = a.x.n_cols;
  if (M == 0 || N == 0) {
    cudaError_t e = zero(a.grad_x, s);
    if (e == cudaSuccess) e = zero(a.grad_w, s);
    if (e == cudaSuccess && a.grad_bias && N > 0) e = cudaMemsetAsync(a.grad_bias, 0, sizeof(float) * (size_t)N, s);
    return e;
  }
  linear_grad_args b = a;
  if (K == 0) b.grad_x.data = b.grad_w.data = nullptr;
  return a.x.type == SS_VALUES_BF16 ? grad_typed<__nv_bfloat16>(h, b, s, queued) : grad_typed<__half>(h, b, s, queued);
}
