// Softmax cross entropy over every item without the logits, and its gradients.
//
//   z = (x w^T + bias) / T,  lse_r = log sum_v exp(z_rv)
//   loss_r = weight_r (lse_r - z_r[target_r])
//   gz_rv = weight_r grad_loss_r / T (exp(z_rv - lse_r) - [v = target_r])
//   grad_x = gz w,  grad_w = gz^T x,  grad_bias = sum_r gz_r
//
// x [M, K] rows, w [V, K] items, 16 bits; sums, statistics and the epilogue
// float32.  A row without a target, with one that the bias masks (its logit is
// -inf) or of weight 0 is absent: loss 0 and gradient 0, whatever x holds.
//
// The loss (k_logits<false>): tiles of 256 x 256 logits by pairs of blocks
// (product.cuh) that stay in tensor memory.  A thread of the epilogue owns a row
// of the block's and 64 of the tile's columns; it keeps their running maximum
// and sum of exponentials in registers over a unit of consecutive tiles of one
// row of tiles, and writes one pair a unit.  k_join adds the pairs up in a fixed
// order.  Bound by the tensor cores where rows are many and by reading w where
// they are few.
//
// The gradients, in pieces of the items: k_logits<true> computes a piece's
// logits again and writes gz, rounded to x's type, as the two products that
// follow take it: grad_w's rows of the piece at once, grad_x added up over the
// pieces in float32.  Nothing of the size of the logits is ever held; the
// price are the logits' flops once more (8 M V K in place of 6).
//
// gz of binary16 is held times a power of two that brings the largest |weight
// grad_loss / T| below 2^15, as a softmax over many items lies below binary16's
// smallest values; the products' epilogues take it out again.  bfloat16 has
// float32's exponents and needs none.
#include <math.h>

#include <algorithm>

#include "product.cuh"

namespace {

using namespace dense;

constexpr int kBN = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The exponent of a logit is fma(z, c, -base_of(largest z)), c = log2(e) / T:
// the same rounded base everywhere, so that it cancels.
__device__ __forceinline__ float base_of(float most, float c) { return most == -INFINITY ? 0.0f : most * c; }

// Units of consecutive tiles of one row of tiles; units that share their items
// follow one another, so that the tiles in flight share w's rows in L2.
struct UnitWalk {
  int64_t unit, step, tiles_a, tiles_b, units;  // units of a row of tiles
  int32_t kb;
  int64_t tb = 0, end = 0, ta = 0;
  int64_t number = 0;
  bool first = false;
  __device__ __forceinline__ bool next(Tile &t) {
    first = tb == end;
    if (first) {
      if (unit >= tiles_a * units) return false;
      number = unit / tiles_a;
      ta = unit % tiles_a;
      tb = tiles_b * number / units;
      end = tiles_b * (number + 1) / units;
      unit += step;
    }
    t = {ta, tb++, 0, kb, 0};
    return true;
  }
  __device__ __forceinline__ bool last() const { return tb == end; }
};

struct Logits {
  CUtensorMap a, b, gz;
  int32_t blocks_k, tiles_a, tiles_b, units;
  uint32_t idesc;
  int32_t *status;
  int64_t M, V;          // rows, and items of the piece
  int64_t first;         // the piece's first item
  const float *bias;     // of the piece, or null
  const int64_t *targets;
  float c;               // log2(e) / T
  // statistics
  float2 *part;          // [units * 4][M]
  float *here;           // [M]: the target's logit
  // gradient
  const float2 *stats;
  const float *weight, *grad_loss, *factor;
  float inv_t;
  ss_dense out;
  float *sums;           // [tiles_a * 8][V] or null: columns' sums over 32 rows
};

// The sum over the lanes of v[j], in lane j.
__device__ __forceinline__ float column_sums(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
    }
  }
  return v[0];
}

template <bool kGrad>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1) k_logits(const __grid_constant__ Logits a) {
  const int lane = threadIdx.x & 31;
  const int64_t rank_rows = (int64_t)tc::cluster_rank() * kTileM;
  float most = -INFINITY, sum = 0.0f;
  UnitWalk walk = {};
  walk.unit = blockIdx.x / 2;
  walk.step = gridDim.x / 2;
  walk.tiles_a = a.tiles_a;
  walk.tiles_b = a.tiles_b;
  walk.units = a.units;
  walk.kb = a.blocks_k;
  pair_products<kBN, kMajorK, kMajorK, false, kGrad ? 1 : 0>(
      &a.a, &a.b, &a.idesc, a.status, walk,
      [&](const UnitWalk &w, const Tile &t, int q, int quarter, uint32_t acc, uint32_t boxes, auto release) {
        const int64_t m0 = t.ta * 2 * kTileM + rank_rows + q * 32, m = m0 + lane;
        const bool rows = m0 < a.M;
        float base = 0.0f, scale = 0.0f, share = 0.0f;
        bool absent = true;
        int64_t target = -1;
        if (m < a.M) {
          target = a.targets[m] - a.first;
          if (kGrad) {
            const float2 st = a.stats[m];
            const float weight = a.weight ? a.weight[m] : 1.0f;
            absent = st.y == INFINITY || weight == 0.0f;
            scale = weight * (a.grad_loss ? a.grad_loss[m] : 1.0f) * a.inv_t;
            if (a.factor) scale *= a.factor[0];
            share = scale / st.y;
            base = base_of(st.x, a.c);
          }
        }
        if (!kGrad && w.first) {
          most = -INFINITY;
          sum = 0.0f;
        }
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int col = quarter * (kBN / 4) + half * 32;
          const int64_t n0 = t.tb * kBN + col;
          float v[32];
          {
            uint32_t r[32];
            tc::load_acc32(acc + (uint32_t)col, r);
            tc::load_acc_wait();
            if (half == 1) release();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          }
          if (!rows || n0 >= a.V) continue;
          if (a.bias) along32(a.bias + n0, a.V - n0, [&](int i, float f) { v[i] += f; });
          const uint64_t at = (uint64_t)(target - n0);
          if (!kGrad) {
            if (n0 + 32 > a.V) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (n0 + i >= a.V) v[i] = -INFINITY;
            }
            if (at < 32) {
              // by bits: where i == at picks it, the compiler puts v into memory
              const uint32_t bit = 1u << (uint32_t)at;
              float z = 0.0f;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (bit & (1u << i)) z = v[i];
              if (n0 + (int64_t)at < a.V) a.here[m] = z;
            }
            float top = most;
#pragma unroll
            for (int i = 0; i < 32; ++i) top = fmaxf(top, v[i]);
            const float b = base_of(top, a.c);
            float s = most == -INFINITY ? 0.0f : sum * exp2_fast(base_of(most, a.c) - b), s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              s += exp2_fast(fmaf(v[i], a.c, -b));
              s2 += exp2_fast(fmaf(v[i + 1], a.c, -b));
            }
            sum = s + s2;
            most = top;
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = exp2_fast(fmaf(v[i], a.c, -base)) * share;
            if (at < 32) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] -= i == (int)at ? scale : 0.0f;
            }
            if (absent) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0.0f;
            }
            put32(a.out, &a.gz, true, boxes, lane, m0, n0, v);
            if (a.sums) {
              float total = column_sums(v, lane);
              if (a.factor) total *= a.factor[1];
              if (n0 + lane < a.V) a.sums[(m0 / 32) * a.V + n0 + lane] = total;
            }
          }
        }
        if (!kGrad && w.last() && m < a.M) a.part[(w.number * 4 + quarter) * a.M + m] = make_float2(most, sum);
      });
}

// The rows' losses and statistics from the units' pairs, in their order: a block
// takes 32 rows, eight threads a row.
struct Join {
  const float2 *part;
  const float *here, *weight;
  const int64_t *targets;
  int64_t M, V;
  int32_t parts;
  float c;
  float *loss;
  float2 *stats;
  int32_t *status;
};
__global__ void __launch_bounds__(256) k_join(const Join a) {
  __shared__ float2 sm[8][32];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t m = (int64_t)blockIdx.x * 32 + lane;
  float most = -INFINITY, sum = 0.0f;
  auto add = [&](float2 p) {
    const float top = fmaxf(most, p.x), b = base_of(top, a.c);
    sum = (most == -INFINITY ? 0.0f : sum * exp2_fast(base_of(most, a.c) - b)) +
          (p.x == -INFINITY && p.y == 0.0f ? 0.0f : p.y * exp2_fast(base_of(p.x, a.c) - b));
    most = top;
  };
  if (m < a.M)
#pragma unroll 4
    for (int p = g; p < a.parts; p += 8) add(a.part[(int64_t)p * a.M + m]);
  sm[g][lane] = make_float2(most, sum);
  __syncthreads();
  if (g != 0 || m >= a.M) return;
  for (int k = 1; k < 8; ++k) add(sm[k][lane]);
  const int64_t target = a.targets[m];
  const float weight = a.weight ? a.weight[m] : 1.0f;
  const bool past = target >= a.V;
  if (past) flag(a.status, DEV_OUT_OF_RANGE);
  bool live = target >= 0 && !past && weight != 0.0f;
  float loss = 0.0f;
  if (live) {
    const float z = a.here[m];
    live = z != -INFINITY;
    if (live) loss = weight * (kLn2 * (log2f(sum) - fmaf(z, a.c, -base_of(most, a.c))));
  }
  a.loss[m] = loss;
  a.stats[m] = make_float2(most, live ? sum : INFINITY);
}

// x with the absent rows' values 0, as 0 times an infinity or NaN there would
// reach grad_w; and for binary16 gz's power of two and its reciprocal.
struct Prepare {
  ss_dense x;
  void *to;
  int64_t ld;
  const int64_t *targets;
  const float *weight, *grad_loss;
  float inv_t;
  int64_t V;
  float *factor;  // or null
};
template <int kN>
__global__ void __launch_bounds__(256) k_prepare(const Prepare a) {
  using P = Pack<uint16_t, kN>;
  const int64_t M = a.x.n_rows, K = a.x.n_cols;
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const int64_t t = a.targets[m];
    const bool there = t >= 0 && t < a.V && (!a.weight || a.weight[m] != 0.0f);
    const uint16_t *from = static_cast<const uint16_t *>(a.x.data) + m * a.x.ld;
    uint16_t *to = static_cast<uint16_t *>(a.to) + m * a.ld;
    for (int64_t c = (int64_t)threadIdx.x * kN; c < K; c += 256 * kN) {
      P v = {};
      if (there) v = *reinterpret_cast<const P *>(from + c);
      *reinterpret_cast<P *>(to + c) = v;
    }
  }
  if (!a.factor || blockIdx.x != 0) return;
  __shared__ float sm[8];
  float most = 0.0f;
  for (int64_t m = threadIdx.x; m < M; m += 256) {
    const float g = fabsf((a.weight ? a.weight[m] : 1.0f) * (a.grad_loss ? a.grad_loss[m] : 1.0f) * a.inv_t);
    if (g < INFINITY) most = fmaxf(most, g);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < 8; ++k) most = fmaxf(most, sm[k]);
    const int e = most > 0.0f ? max(-100, min(100, 14 - ilogbf(most))) : 0;
    a.factor[0] = ldexpf(1.0f, e);
    a.factor[1] = ldexpf(1.0f, -e);
  }
}

// ---------------------------------------------------------------- host side
int64_t up(int64_t x, int64_t y) { return (x + y - 1) / y; }

// Units of a row of tiles: the fewest for which the pairs, each taking whole
// units in turn, end soonest.
int64_t units_of(const ss_handle *h, int64_t tiles_a, int64_t tiles_b) {
  const int64_t pairs = std::max(1, h->sm_count / 2), most = std::min<int64_t>(tiles_b, 256);
  int64_t best = 1, least = INT64_MAX;
  for (int64_t n = 1; n <= most; ++n) {
    const int64_t tiles = up(tiles_a * n, pairs) * up(tiles_b, n);
    if (tiles < least) {
      least = tiles;
      best = n;
    }
  }
  return best;
}

// The scratch of a call, in this order.
struct Room {
  int64_t V, K, piece, x, w, factor, part, here, stats, gz, acc, sums;
  int64_t units, parts;
  Room(const ss_handle *h, const ss_dense &x_, const ss_dense &w_, int32_t mode) {
    const int64_t M = x_.n_rows, tiles_a = up(M, 2 * kTileM);
    V = w_.n_rows;
    K = x_.n_cols;
    const bool loss = mode != XENT_BACKWARD, grad = mode != XENT_LOSS;
    units = units_of(h, tiles_a, up(V, kBN));
    // pieces of at most 2^27 values of gz, of whole tiles and equal sizes
    const int64_t most = std::max<int64_t>(2048, ((int64_t)1 << 27) / std::max<int64_t>(1, M)), pieces = up(V, most);
    piece = up(up(V, pieces), kBN) * kBN;
    x = grad ? align_up(M * padded_ld(x_) * 2) : copy_bytes(x_);
    w = copy_bytes(w_);
    factor = grad ? SS_SCRATCH_ALIGN : 0;
    part = loss ? align_up(units * 4 * M * (int64_t)sizeof(float2)) : 0;
    here = loss ? align_up(M * 4) : 0;
    stats = mode == XENT_STEP ? align_up(M * 8) : 0;
    gz = grad ? align_up(M * piece * 2) : 0;
    parts = grad ? grad_product_parts(h, M, piece, K) : 1;
    acc = grad && (piece < V || parts > 1) ? parts * grad_part_bytes(M, K) : 0;
    sums = grad ? align_up(tiles_a * 8 * piece * 4) : 0;
  }
  int64_t bytes() const { return x + w + factor + part + here + stats + gz + acc + sums; }
};

ss_dense rows_from(const ss_dense &m, int64_t first, int64_t n) {
  ss_dense r = m;
  r.data = static_cast<unsigned char *>(m.data) + first * m.ld * size_of(m.type);
  r.n_rows = n;
  return r;
}

template <bool kGrad>
cudaError_t run_logits(ss_handle *h, Logits &p, const ss_dense &x, const ss_dense &w, cudaStream_t s, int *queued) {
  p.blocks_k = (int32_t)up(x.n_cols, kRowBytes / 2);
  p.tiles_a = (int32_t)up(x.n_rows, 2 * kTileM);
  p.tiles_b = (int32_t)up(w.n_rows, kBN);
  p.idesc = idesc_of(x, kMajorK, kMajorK, 2 * kTileM, kBN);
  p.status = h->d_status;
  p.M = x.n_rows;
  p.V = w.n_rows;
  cudaError_t e = encode(&p.a, x, kRowBytes / 2, kTileM);
  if (e == cudaSuccess) e = encode(&p.b, w, kRowBytes / 2, kBN / 2);
  if (e == cudaSuccess && kGrad) e = encode_out(&p.gz, p.out);
  if (e == cudaSuccess) e = ensure_dyn_smem(k_logits<kGrad>, PairRing<kBN, kGrad ? 1 : 0>::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t pairs = std::min<int64_t>((int64_t)p.tiles_a * p.units, std::max(1, h->sm_count / 2));
  k_logits<kGrad><<<(unsigned)(2 * pairs), kPairThreads, PairRing<kBN, kGrad ? 1 : 0>::kSmem, s>>>(p);
  *queued += 1;
  return cudaGetLastError();
}

}  // namespace

int64_t xent_scratch(const ss_handle *h, const ss_dense &x, const ss_dense &w, int32_t mode) {
  return x.n_rows > 0 && w.n_rows > 0 ? Room(h, x, w, mode).bytes() : 0;
}

cudaError_t launch_xent(ss_handle *h, const xent_args &a, int32_t mode, cudaStream_t s, int *queued) {
  *queued = 0;
  const bool loss = mode != XENT_BACKWARD, grad = mode != XENT_LOSS;
  const int64_t M = a.x.n_rows, V = a.w.n_rows, K = a.x.n_cols;
  cudaError_t e;
  if (M == 0) {  // the gradients that are sums over rows
    if (grad && a.grad_w.data) {
      const size_t size = (size_t)size_of(a.grad_w.type);
      if ((e = cudaMemset2DAsync(a.grad_w.data, (size_t)a.grad_w.ld * size, 0, (size_t)K * size, (size_t)V, s)) != cudaSuccess) return e;
    }
    return grad && a.grad_bias ? cudaMemsetAsync(a.grad_bias, 0, sizeof(float) * (size_t)V, s) : cudaSuccess;
  }
  const Room room(h, a.x, a.w, mode);
  unsigned char *at = a.scratch;
  auto take = [&](int64_t bytes) {
    unsigned char *p = at;
    at += bytes;
    return p;
  };
  ss_dense x = a.x, w = a.w;
  float *factor = nullptr;
  if (grad) {
    Prepare p = {a.x, take(room.x), padded_ld(a.x), a.targets, a.weight, a.grad_loss, 1.0f / a.temperature, V, nullptr};
    x.data = p.to;
    x.ld = p.ld;
    if ((e = launch_aligned_rows(h, &w, nullptr, &at, s, queued)) != cudaSuccess) return e;
    float *f = reinterpret_cast<float *>(take(room.factor));
    if (a.x.type == SS_VALUES_F16) p.factor = factor = f;
    const unsigned blocks = (unsigned)std::min<int64_t>(M, 8 * (int64_t)std::max(1, h->sm_count));
    if (rows_aligned(a.x, 16) && K % 8 == 0)
      k_prepare<8><<<blocks, 256, 0, s>>>(p);
    else
      k_prepare<1><<<blocks, 256, 0, s>>>(p);
    *queued += 1;
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  } else if ((e = launch_aligned_rows(h, &x, &w, &at, s, queued)) != cudaSuccess) {
    return e;
  }
  float2 *stats = reinterpret_cast<float2 *>(a.stats);
  Logits p = {};
  p.targets = a.targets;
  p.c = kLog2e / a.temperature;
  if (loss) {
    p.part = reinterpret_cast<float2 *>(take(room.part));
    p.here = reinterpret_cast<float *>(take(room.here));
    if (mode == XENT_STEP) stats = reinterpret_cast<float2 *>(take(room.stats));
    p.bias = a.bias;
    p.units = (int32_t)room.units;
    if ((e = run_logits<false>(h, p, x, w, s, queued)) != cudaSuccess) return e;
    const Join j = {p.part, p.here, a.weight, a.targets, M, V, (int32_t)room.units * 4, p.c, a.loss, stats, h->d_status};
    k_join<<<(unsigned)up(M, 32), 256, 0, s>>>(j);
    *queued += 1;
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (!grad) return cudaSuccess;
  p.stats = stats;
  p.weight = a.weight;
  p.grad_loss = a.grad_loss;
  p.factor = factor;
  p.inv_t = 1.0f / a.temperature;
  void *gz = take(room.gz);
  grad_products g = {};
  g.x = x;
  g.grad_x = a.grad_x;
  g.acc = reinterpret_cast<float *>(take(room.acc));
  g.parts = (int32_t)room.parts;
  g.factor = factor ? factor + 1 : nullptr;
  float *sums = reinterpret_cast<float *>(take(room.sums));
  const int64_t tiles_a = up(M, 2 * kTileM);
  for (int64_t first = 0; first < V; first += room.piece) {
    const int64_t n = std::min(room.piece, V - first);
    const ss_dense wp = rows_from(w, first, n);
    p.out = {gz, M, n, room.piece, a.x.type};
    p.first = first;
    p.bias = a.bias ? a.bias + first : nullptr;
    p.sums = a.grad_bias ? sums : nullptr;
    p.units = (int32_t)units_of(h, tiles_a, up(n, kBN));
    if ((e = run_logits<true>(h, p, x, wp, s, queued)) != cudaSuccess) return e;
    if (a.grad_bias) {
      if ((e = launch_sum_rows(h, sums, up(M, 32), n, a.grad_bias + first, SS_VALUES_F32, s)) != cudaSuccess) return e;
      *queued += 1;
    }
    g.wide = wp;
    g.gz = p.out;
    g.grad_w = a.grad_w.data ? rows_from(a.grad_w, first, n) : a.grad_w;
    g.begun = first > 0;
    g.ends = first + n == V;
    if ((e = launch_grad_products(h, g, s, queued)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}
