// Softmax cross entropy over every item without the logits, and its gradients.
//
//   z = (x w^T + bias) / T,  lse_r = log sum_v exp(z_rv)
//   loss_r = weight_r (lse_r - z_r[target_r])
//   gz_rv = weight_r grad_loss_r / T (exp(z_rv - lse_r) - [v = target_r])
//   grad_x = gz w,  grad_w = gz^T x,  grad_bias = sum_r gz_r
//
// x [M, K] rows, w [V, K] items, 16 bits; sums, statistics and the epilogue
// float32.  The sums are the tensor cores': a partial sum is cut toward zero for
// every 16 products (over normal values 8e-10 K of the whole in all); sums that
// float32 holds are not.  A row without a target, with one that the bias masks or of
// weight 0 is absent: loss 0 and gradient 0, whatever x holds.
//
// The loss (k_statistics): tiles of 256 x 256 logits by pairs of blocks
// (product.cuh) that stay in tensor memory.  A thread of the epilogue owns a row
// of the block's and 64 of the tile's columns; it keeps their running maximum
// and sum of exponentials in registers over a unit of consecutive tiles of one
// row of tiles, and writes one pair a unit.  k_between adds the pairs up in a
// fixed order.  Bound by the tensor cores where rows are many: 5000 x 200,000 x
// 1024 bf16 1.26 to 1.31 ms (1,600 TFLOP/s; the card is at its power cap).  A step of
// half the rows takes 2.7 to 2.8 ms: 0.59 of it this, 0.18 and 0.29 a piece of 50,176
// items for gz and for the two products.
//
// The gradients, in pieces of the items: k_logit_gradient computes a piece's
// logits again and writes gz, rounded to x's type, as the two products that
// follow take it: grad_w's rows of the piece at once, grad_x added up over the
// pieces in float32 (gradients.cu).  Nothing of the size of the logits is ever
// held; the price are the logits' flops once more (8 M V K in place of 6).
//
// gz is held without its row's factor weight grad_loss / T, between -1 and 1:
// the target's value, p - 1, is most of a row and near -1 as a rule, where it
// rounds to next to nothing.  grad_x's rows take the factor in the epilogue,
// grad_w takes rows of x times it, rounded to x's type.  (With the factor in gz
// the target's value lost up to half a step, the whole row of grad_x with it:
// 1.6 times the final rounding's error with few rows.)  binary16's gz is held
// times 2^14, as most of a softmax over many items lies below its smallest
// values, and its rows of x times one power of two that brings the largest
// factor near 1; the epilogues take both out again.
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
// the same rounded base everywhere, so that it cancels.  A value at or below
// `low` is masked, as -infinity is: times c it may be past float32's lowest, and
// as the base of a range of items that are all masked it would give inf - inf.
// With the base 0 their exponentials are 0.
__device__ __forceinline__ float base_of(float most, float c, float low) { return most <= low ? 0.0f : most * c; }

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
    t = {(int32_t)ta, (int32_t)tb++, 0, kb, 0};
    return true;
  }
  __device__ __forceinline__ bool last() const { return tb == end; }
};

// What the gradient of a row's logits takes: gz_v = exp2(c z_v - base) share,
// less `hot` at the target, and the row's factor over `hot`.  hot, what 1 stands
// for in gz: 1, binary16 2^14.
struct alignas(16) Row {
  float base, share, scale;
  int32_t target;
};
constexpr int kHalfBits = 14;
__device__ __forceinline__ Row absent_row() { return {INFINITY, 0.0f, 0.0f, -1}; }  // exp2(-inf) 0

struct Logits {
  CUtensorMap a, b, gz;
  int32_t blocks_k, tiles_a, tiles_b, units;
  uint32_t idesc;
  int32_t *status;
  int64_t M, V;          // rows, and items of the piece
  int64_t first;         // the piece's first item
  const float *bias;     // of the piece, or null
  int32_t bias_pairs;    // it starts on an 8-byte boundary
  float c;               // log2(e) / T
  float low;             // masked from here down
  // statistics
  const int64_t *targets;
  float2 *part;          // [units * 4][M]
  float *here;           // [M]: the target's logit
  // gradient
  const Row *rows;
  float hot;
  ss_dense out;
  float *sums;           // [tiles_a * 2][ld_sums] or null: columns' sums over 128 rows
  int64_t ld_sums;
};

// A thread of the loss's epilogue: its row's largest logit so far and the sum of
// exponentials, over its columns of a unit.
struct Running {
  float most, sum;
  __device__ __forceinline__ void add32(float (&v)[32], float c, float low) {
    float top = most;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = fmaxf(top, v[i]);
    const float b = base_of(top, c, low);
    // of masked logits alone it is 0, or NaN where one among them is: fmaxf leaves
    // NaN out of `most`, the sum keeps it
    if (most > low) sum *= exp2_fast(base_of(most, c, low) - b);
    most = top;
    const Two c2 = two(c, c), b2 = two(-b, -b);
    Two s = two(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 e = both(fma_of(two(v[i], v[i + 1]), c2, b2));
      s = s + two(exp2_fast(e.x), exp2_fast(e.y));
    }
    const float2 r = both(s);
    sum += r.x + r.y;
  }
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1) k_statistics(const __grid_constant__ Logits a) {
  const int lane = threadIdx.x & 31;
  const int64_t rank_rows = (int64_t)tc::cluster_rank() * kTileM;
  Running run = {-INFINITY, 0.0f};
  UnitWalk walk = {};
  walk.unit = blockIdx.x / 2;
  walk.step = gridDim.x / 2;
  walk.tiles_a = a.tiles_a;
  walk.tiles_b = a.tiles_b;
  walk.units = a.units;
  walk.kb = a.blocks_k;
  pair_products<kBN, kMajorK, kMajorK, false, 0>(
      &a.a, &a.b, &a.idesc, a.status, walk,
      [&](const UnitWalk &w, const Tile &t, int q, int quarter, uint32_t acc, uint32_t, auto release) {
        const int64_t m0 = t.ta * 2 * kTileM + rank_rows + q * 32, m = m0 + lane;
        const int64_t target = m < a.M ? a.targets[m] : -1;
        if (w.first) run = {-INFINITY, 0.0f};
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
          if (m0 >= a.M || n0 >= a.V) continue;
          if (a.bias) along32(a.bias + n0, a.V - n0, [&](int i, float f) { v[i] += f; });
          if (n0 + 32 > a.V) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (n0 + i >= a.V) v[i] = -INFINITY;
          }
          const uint64_t at = (uint64_t)(target - n0);
          if (at < 32) {
            // by bits: where i == at picks it, the compiler puts v into memory
            const uint32_t bit = 1u << (uint32_t)at;
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (bit & (1u << i)) z = v[i];
            if (target < a.V) a.here[m] = z;
          }
          run.add32(v, a.c, a.low);
        }
        if (w.last() && m < a.M) a.part[(w.number * 4 + quarter) * a.M + m] = make_float2(run.most, run.sum);
      });
}

// The sums over the lanes t with one t % 4 of v[j]: that of j = 4 (t & 16 ? 1 : 0) +
// 2 (t & 8 ? 1 : 0) + (t & 4 ? 1 : 0) in thread t.
__device__ __forceinline__ float sum_eighth(float (&v)[8], int lane) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    const bool up = lane & (o * 4);
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o * 4);
    }
  }
  return v[0];
}

// gz of a piece.  The accumulators are read as the matrix fragments that stmatrix
// takes: a thread has 8 columns of 4 rows, so that a column's sum over 32 rows
// is 3 additions and 3 shuffles' worth in place of 5 of 32 (a row a thread,
// 31 shuffles a block of 32 x 32: 192 us for 2500 x 50,176 x 1024, where this
// takes 178; the same product without an epilogue takes 136.)
template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1) k_logit_gradient(const __grid_constant__ Logits a) {
  const int lane = threadIdx.x & 31;
  const int64_t rank_rows = (int64_t)tc::cluster_rank() * kTileM;
  UnitWalk walk = {};
  walk.unit = blockIdx.x / 2;
  walk.step = gridDim.x / 2;
  walk.tiles_a = a.tiles_a;
  walk.tiles_b = a.tiles_b;
  walk.units = a.units;
  walk.kb = a.blocks_k;
  pair_products<kBN, kMajorK, kMajorK, false, 2>(
      &a.a, &a.b, &a.idesc, a.status, walk,
      [&](const UnitWalk &, const Tile &t, int q, int quarter, uint32_t acc, uint32_t boxes, auto release) {
        const int64_t m0 = t.ta * 2 * kTileM + rank_rows + q * 32;
        Row row[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t m = m0 + lane / 4 + 8 * k;
          row[k] = m < a.M ? a.rows[m] : absent_row();
        }
        const Two c2 = two(a.c, a.c);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int col = quarter * (kBN / 4) + half * 32;
          const int64_t n0 = t.tb * kBN + col;
          uint32_t r[32];
          tc::load_acc16x32(acc + (uint32_t)col, r);
          tc::load_acc16x32(acc + (uint32_t)col + (16u << 16), r + 16);
          tc::load_acc_wait();
          if (half == 1) release();
          if (n0 >= a.V) {
            if (a.sums && half == 1) tc::named_sync(1 + quarter, 128);  // the first half's place has been read
            continue;
          }
          const int64_t left = a.V - n0;
          float sums[8];
          if (m0 < a.M) {
            Two bias[4];
            if (a.bias) {
              const float *p = a.bias + n0 + 2 * (lane % 4);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (left >= 32 && a.bias_pairs) {
                  const float2 f = __ldg(reinterpret_cast<const float2 *>(p + 8 * i));
                  bias[i] = two(f.x, f.y);
                } else {
                  const int64_t n = 8 * i + 2 * (lane % 4);
                  bias[i] = two(n < left ? __ldg(p + 8 * i) : 0.0f, n + 1 < left ? __ldg(p + 8 * i + 1) : 0.0f);
                }
              }
            }
            bool hot = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) hot = hot || (uint64_t)(row[k].target - (a.first + n0)) < 32;
            const bool any_hot = __any_sync(0xFFFFFFFFu, hot);
            if (lane == 0) tc::store_wait_read();  // the box's last copy out
            __syncwarp();
            uint32_t packed[4][4];  // of rows 8 k on, columns 8 i on
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              Two sum = two(0.0f, 0.0f);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t *f = r + 16 * (k / 2) + 4 * i + 2 * (k % 2);
                Two z = two(__uint_as_float(f[0]), __uint_as_float(f[1]));
                if (a.bias) z = z + bias[i];
                const float2 e = both(fma_of(z, c2, two(-row[k].base, -row[k].base)));
                Two g = two(exp2_fast(e.x), exp2_fast(e.y)) * two(row[k].share, row[k].share);
                if (any_hot) {
                  const int64_t at = row[k].target - (a.first + n0) - (8 * i + 2 * (lane % 4));
                  g = g + two(at == 0 ? -a.hot : 0.0f, at == 1 ? -a.hot : 0.0f);
                }
                sum = fma_of(g, two(row[k].scale, row[k].scale), sum);
                const float2 h = both(g);
                packed[k][i] = narrow2(T(), h.x, h.y);
              }
              const float2 h = both(sum);
              sums[2 * i] = h.x;
              sums[2 * i + 1] = h.y;
            }
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int i = 0; i < 4; i += 2)
                tc::store_matrices(unit_at(boxes, 16 * b + (lane / 8 & 1) * 8 + lane % 8, i + lane / 16), packed[2 * b][i], packed[2 * b + 1][i],
                                   packed[2 * b][i + 1], packed[2 * b + 1][i + 1]);
            tc::fence_async();
            __syncwarp();
            if (lane == 0) {
              tc::store_2d(&a.gz, boxes, (int)n0, (int)m0);
              tc::store_commit();
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) sums[i] = 0.0f;
          }
          if (a.sums) {
            // columns 8 i + 2 (t % 4) + j: thread t ends with i = t / 8 and j = t / 4 % 2
            float total = sum_eighth(sums, lane);
            const uint32_t mine = boxes + kStaging + (uint32_t)(half * 128);
            tc::write_shared(mine + 4 * (uint32_t)(lane / 8 * 8 + lane % 4 * 2 + (lane / 4 & 1)), total);
            // the four warps of these columns; a half's place is written again
            // only after the other half's barrier, when it has been read (the
            // second half's barrier comes in every tile)
            tc::named_sync(1 + quarter, 128);
            if (q == half) {
              const int warp = (int)(threadIdx.x >> 5) - 2;
              const uint32_t firsts = mine - (uint32_t)((warp & 3) * 2 * kStaging);
              total = 0.0f;
#pragma unroll
              for (int k = 0; k < 4; ++k) total += tc::read_shared<float>(firsts + (uint32_t)(k * 2 * kStaging) + 4 * (uint32_t)lane);
              if (lane < left) a.sums[(m0 / kTileM) * a.ld_sums + n0 + lane] = total;
            }
          }
        }
      });
}

// Between the two: the rows' losses and statistics from the units' pairs, in
// their order (unless the statistics are given), what gz takes of each row, and
// x with the absent rows' values 0, as 0 times an infinity or NaN there would
// reach grad_w, once as it is and once times the rows' factors.  A block takes
// eight rows, 32 threads a row.
struct Between {
  const float2 *part;  // or null: stats are given
  const float *here, *weight, *grad_loss, *bias;
  const int64_t *targets;
  int64_t M, V;
  int32_t parts, vec;
  float c, low, inv_t;
  float *loss;
  float2 *stats;
  int32_t *status;
  // for the gradient, or null
  Row *rows;
  ss_dense x;
  void *to;            // x's copy, or x's own data: absent rows alone are written then
  int64_t ld;
  void *scaled;         // x times the rows' factors (and the power of two)
  float hot;
  const float *factor;  // binary16's power of two, or null: 1
  int32_t type;
};
// binary16's power of two, which brings the largest |factor of a row| to 1/2 at
// least and below 1, and what takes it and gz's out of their products.  Of the
// rows that take part: a padded one's weight and gradient may be anything.
__global__ void __launch_bounds__(1024) k_factor(const int64_t *targets, const float *bias, float low, const float *weight, const float *grad_loss,
                                                 float inv_t, int64_t M, int64_t V, float *factor) {
  __shared__ float sm[32];
  tc::let_next();
  float most = 0.0f;
#pragma unroll 4
  for (int64_t k = threadIdx.x; k < M; k += 1024) {
    const int64_t target = targets[k];
    const float v = fabsf((weight ? weight[k] : 1.0f) * (grad_loss ? grad_loss[k] : 1.0f) * inv_t);
    if (target >= 0 && target < V && v < INFINITY && !(bias && bias[target] <= low)) most = fmaxf(most, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < 32; ++k) most = fmaxf(most, sm[k]);
    const int e = most > 0.0f ? max(-100, min(100, -1 - ilogbf(most))) : 0;
    factor[0] = ldexpf(1.0f, e);
    factor[1] = ldexpf(1.0f, -e - kHalfBits);
  }
  tc::wait_before();  // what follows waits for this kernel, and so for the one before it
}
// 8 values, or one, of T times f.
template <typename T>
__device__ __forceinline__ uint4 times(uint4 v, float f) {
  Pack<T, 8> p;
  memcpy(&p, &v, 16);
  float x[8];
  widen(p, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= f;
  p = narrow<T, 8>(x);
  memcpy(&v, &p, 16);
  return v;
}
constexpr int kBetweenRows = 8, kBetweenThreads = 256;
__global__ void __launch_bounds__(kBetweenThreads) k_between(const Between a) {
  __shared__ float2 sm[kBetweenThreads / 32][kBetweenRows];
  __shared__ bool there[kBetweenRows];
  __shared__ float scales[kBetweenRows];
  tc::wait_before();
  tc::let_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * kBetweenRows, m = row0 + lane % kBetweenRows;
  float most = -INFINITY, sum = 0.0f;
  auto add = [&](float2 p) {
    const float top = fmaxf(most, p.x), b = base_of(top, a.c, a.low);
    // of masked logits alone a sum is 0, or NaN
    sum = (most <= a.low ? sum : sum * exp2_fast(base_of(most, a.c, a.low) - b)) +
          (p.x <= a.low ? p.y : p.y * exp2_fast(base_of(p.x, a.c, a.low) - b));
    most = top;
  };
  if (a.part) {
    constexpr int kLanes = kBetweenThreads / kBetweenRows;  // threads of a row
    if (m < a.M)
      for (int p0 = threadIdx.x / kBetweenRows; p0 < a.parts; p0 += 8 * kLanes) {
        float2 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = p0 + k * kLanes < a.parts ? a.part[(int64_t)(p0 + k * kLanes) * a.M + m] : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (p0 + k * kLanes < a.parts) add(v[k]);
      }
#pragma unroll
    for (int o = kBetweenRows; o < 32; o *= 2) {
      const float2 other = make_float2(__shfl_down_sync(0xFFFFFFFFu, most, o), __shfl_down_sync(0xFFFFFFFFu, sum, o));
      add(other);
    }
    if (lane < kBetweenRows) sm[warp][lane] = make_float2(most, sum);
    __syncthreads();
  }
  if (threadIdx.x < kBetweenRows && m < a.M) {
    const int64_t target = a.targets[m];
    const float weight = a.weight ? a.weight[m] : 1.0f;
    const bool past = target >= a.V;
    if (past) flag(a.status, DEV_OUT_OF_RANGE);
    bool live = target >= 0 && !past && weight != 0.0f && !(a.bias && a.bias[target] <= a.low);
    there[lane] = live;
    if (a.part) {
      for (int k = 1; k < kBetweenThreads / 32; ++k) add(sm[k][lane]);
      float loss = 0.0f;
      if (live) loss = weight * (kLn2 * (log2f(sum) - fmaf(a.here[m], a.c, -base_of(most, a.c, a.low))));
      a.loss[m] = loss;
      if (a.stats) a.stats[m] = make_float2(most, live ? sum : INFINITY);
    } else {
      most = a.stats[m].x;
      sum = a.stats[m].y;
      live = live && sum != INFINITY;
    }
    if (a.rows) {
      const float scale = weight * (a.grad_loss ? a.grad_loss[m] : 1.0f) * a.inv_t;
      a.rows[m] = live ? Row{base_of(most, a.c, a.low), a.hot / sum, scale / a.hot, (int32_t)target} : absent_row();
      scales[lane] = live ? (a.factor ? scale * a.factor[0] : scale) : 0.0f;
    }
  }
  if (!a.rows) return;
  __syncthreads();
  static_assert(kBetweenThreads / 32 == kBetweenRows, "a warp a row");
  const int r = warp;
  const int64_t row = row0 + r;
  if (row < a.M) {
    uint16_t *to = static_cast<uint16_t *>(a.to) + row * a.ld, *scaled = static_cast<uint16_t *>(a.scaled) + row * a.ld;
    const uint16_t *from = static_cast<const uint16_t *>(a.x.data) + row * a.x.ld;
    const float f = scales[r];
    const bool bf16 = a.type == SS_VALUES_BF16;
    // 16 bytes at a time where rows start on such a boundary, the last values of
    // a row one by one (all of them so: 1003 x 777 19 us, like this 8)
    const int64_t K = a.x.n_cols, whole = a.vec ? K / 8 * 8 : 0;
#pragma unroll 4
    for (int64_t c = (int64_t)lane * 8; c < whole; c += 256) {
      const uint4 v = there[r] ? *reinterpret_cast<const uint4 *>(from + c) : make_uint4(0, 0, 0, 0);
      if (from != to || !there[r]) *reinterpret_cast<uint4 *>(to + c) = v;
      *reinterpret_cast<uint4 *>(scaled + c) = bf16 ? times<__nv_bfloat16>(v, f) : times<__half>(v, f);
    }
    for (int64_t c = whole + lane; c < K; c += 32) {
      const uint16_t v = there[r] ? from[c] : (uint16_t)0;
      to[c] = v;
      const uint32_t w = bf16 ? narrow2(__nv_bfloat16(), __uint_as_float((uint32_t)v << 16) * f, 0.0f)
                              : narrow2(__half(), __half2float(__ushort_as_half(v)) * f, 0.0f);
      scaled[c] = (uint16_t)w;
    }
  }
}

// ---------------------------------------------------------------- host side
int64_t up(int64_t x, int64_t y) { return (x + y - 1) / y; }

// Units of a row of tiles: the fewest for which the pairs, each taking whole
// units in turn, end soonest.
int64_t units_of(const ss_handle *h, int64_t tiles_a, int64_t tiles_b) {
  const int64_t pairs = std::max(1, h->sm_count / 2);
  const int64_t most = std::min<int64_t>({tiles_b, 256, 16 * pairs / tiles_a + 4});
  int64_t best = 1, least = INT64_MAX;
  for (int64_t turns = up(tiles_a, pairs);; ++turns) {  // the units that `turns` turns of all pairs take
    const int64_t n = std::min(most, turns * pairs / tiles_a), tiles = up(tiles_b, n);
    if (turns * tiles < least) {
      least = turns * tiles;
      best = up(tiles_b, tiles);
    }
    if (n == most) return best;
  }
}

// The scratch of a call, in this order.
struct Room {
  int64_t V, K, piece, x, scaled, w, factor, part, here, rows, gz, acc, sums;
  int64_t units, parts;
  bool whole_sums;  // the columns' sums of all pieces at once
  Room(const ss_handle *h, const ss_dense &x_, const ss_dense &w_, int32_t mode) {
    const int64_t M = x_.n_rows, tiles_a = up(M, 2 * kTileM);
    V = w_.n_rows;
    K = x_.n_cols;
    const bool loss = mode != XENT_BACKWARD, grad = mode != XENT_LOSS;
    units = units_of(h, tiles_a, up(V, kBN));
    // pieces of at most 2^27 values of gz (of 2048 items, where rows are 65,536 or
    // more), of whole tiles and equal sizes
    const int64_t most = std::max<int64_t>(2048, ((int64_t)1 << 27) / std::max<int64_t>(1, M)), pieces = up(V, most);
    piece = up(up(V, pieces), kBN) * kBN;
    x = grad ? align_up(M * padded_ld(x_) * 2) : copy_bytes(x_);
    scaled = grad ? x : 0;
    w = copy_bytes(w_);
    factor = grad ? SS_SCRATCH_ALIGN : 0;
    part = loss ? align_up(units * 4 * M * (int64_t)sizeof(float2)) : 0;
    here = loss ? align_up(M * 4) : 0;
    rows = grad ? align_up(M * (int64_t)sizeof(Row)) : 0;
    gz = grad ? align_up(M * piece * 2) : 0;
    parts = grad ? grad_product_parts(h, M, piece, K) : 1;
    acc = grad && (piece < V || parts > 1) ? parts * grad_part_bytes(M, K) : 0;
    whole_sums = tiles_a * 2 * V <= (int64_t)1 << 26;
    sums = grad ? align_up(tiles_a * 2 * (whole_sums ? V : piece) * 4) : 0;
  }
  int64_t bytes() const { return x + scaled + w + factor + part + here + rows + gz + acc + sums; }
};

ss_dense rows_from(const ss_dense &m, int64_t first, int64_t n) {
  ss_dense r = m;
  r.data = static_cast<unsigned char *>(m.data) + first * m.ld * size_of(m.type);
  r.n_rows = n;
  return r;
}

cudaError_t run_logits(ss_handle *h, Logits &p, const ss_dense &x, const ss_dense &w, bool gradient, bool beside, cudaStream_t s, int *queued) {
  p.blocks_k = (int32_t)up(x.n_cols, kRowBytes / 2);
  p.tiles_a = (int32_t)up(x.n_rows, 2 * kTileM);
  p.tiles_b = (int32_t)up(w.n_rows, kBN);
  p.idesc = idesc_of(x, kMajorK, kMajorK, 2 * kTileM, kBN);
  p.status = h->d_status;
  p.M = x.n_rows;
  p.V = w.n_rows;
  p.bias_pairs = reinterpret_cast<uintptr_t>(p.bias) % 8 == 0;
  auto kernel = !gradient ? k_statistics : x.type == SS_VALUES_BF16 ? k_logit_gradient<__nv_bfloat16> : k_logit_gradient<__half>;
  const size_t smem = gradient ? PairRing<kBN, 2>::kSmem : PairRing<kBN, 0>::kSmem;
  cudaError_t e = encode(&p.a, x, kRowBytes / 2, kTileM);
  if (e == cudaSuccess) e = encode(&p.b, w, kRowBytes / 2, kBN / 2);
  if (e == cudaSuccess && gradient) e = encode_out(&p.gz, p.out);
  if (e == cudaSuccess) e = ensure_dyn_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  const int64_t pairs = std::min<int64_t>((int64_t)p.tiles_a * p.units, std::max(1, h->sm_count / 2));
  *queued += 1;
  return launch_beside(kernel, (unsigned)(2 * pairs), kPairThreads, smem, s, beside, p);
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
  void *copy = grad ? take(room.x) : nullptr;
  void *scaled = nullptr;
  if (grad) {
    unsigned char *to = rows_aligned(x, 16) ? at : static_cast<unsigned char *>(copy);  // w's copy follows x's place
    // rows that start anywhere are copied here, the absent ones cleared later
    if ((e = launch_aligned_rows(h, &x, &w, &to, s, queued)) != cudaSuccess) return e;
    at += room.w;
    scaled = take(room.scaled);
  } else if ((e = launch_aligned_rows(h, &x, &w, &at, s, queued)) != cudaSuccess) {
    return e;
  }
  Logits p = {};
  p.c = kLog2e / a.temperature;
  p.low = -1e38f * std::min(1.0f, a.temperature);
  p.hot = a.x.type == SS_VALUES_F16 ? (float)(1 << kHalfBits) : 1.0f;
  Between b = {};
  b.weight = a.weight;
  b.grad_loss = a.grad_loss;
  b.bias = a.bias;
  b.targets = a.targets;
  b.M = M;
  b.V = V;
  b.c = p.c;
  b.low = p.low;
  b.inv_t = 1.0f / a.temperature;
  b.loss = a.loss;
  b.stats = reinterpret_cast<float2 *>(a.stats);
  b.status = h->d_status;
  float *factor = reinterpret_cast<float *>(take(room.factor));
  if (grad && a.x.type == SS_VALUES_F16) {
    if ((e = launch_beside(k_factor, 1, 1024, 0, s, *queued > 0, a.targets, a.bias, p.low, a.weight, a.grad_loss,
                           b.inv_t, M, V, factor)) != cudaSuccess) return e;
    *queued += 1;
    b.factor = factor;
  }
  if (loss) {
    p.targets = a.targets;
    p.part = reinterpret_cast<float2 *>(take(room.part));
    p.here = reinterpret_cast<float *>(take(room.here));
    p.bias = a.bias;
    p.units = (int32_t)room.units;
    if ((e = run_logits(h, p, x, w, false, *queued > 0, s, queued)) != cudaSuccess) return e;
    b.part = p.part;
    b.here = p.here;
    b.parts = (int32_t)room.units * 4;
  }
  if (grad) {
    b.rows = reinterpret_cast<Row *>(take(room.rows));
    b.x = x;
    b.to = copy;
    b.ld = padded_ld(a.x);
    b.vec = rows_aligned(x, 16);
    b.scaled = scaled;
    b.hot = p.hot;
    b.type = a.x.type;
  }
  const bool first = *queued == 0;
  *queued += 1;
  if ((e = launch_beside(k_between, (unsigned)up(M, kBetweenRows), kBetweenThreads, 0, s, !first, b)) != cudaSuccess || !grad) return e;
  x.data = copy;
  x.ld = b.ld;
  p.rows = b.rows;
  void *gz = take(room.gz);
  grad_products g = {};
  g.x = x;
  g.x.data = scaled;
  g.grad_x = a.grad_x;
  g.acc = reinterpret_cast<float *>(take(room.acc));
  g.parts = (int32_t)room.parts;
  g.beside = true;
  g.factor = b.factor ? b.factor + 1 : nullptr;
  g.row_factor = &b.rows->scale;
  g.row_step = sizeof(Row) / sizeof(float);
  float *sums = reinterpret_cast<float *>(take(room.sums));
  const int64_t tiles_a = up(M, 2 * kTileM);
  for (int64_t first = 0; first < V; first += room.piece) {
    const int64_t n = std::min(room.piece, V - first);
    const ss_dense wp = rows_from(w, first, n);
    p.out = {gz, M, n, room.piece, a.x.type};
    p.first = first;
    p.bias = a.bias ? a.bias + first : nullptr;
    p.ld_sums = room.whole_sums ? V : n;
    p.sums = a.grad_bias ? sums + (room.whole_sums ? first : 0) : nullptr;
    p.units = (int32_t)units_of(h, tiles_a, up(n, kBN));
    if ((e = run_logits(h, p, x, wp, true, true, s, queued)) != cudaSuccess) return e;
    g.wide = wp;
    g.gz = p.out;
    g.grad_w = a.grad_w.data ? rows_from(a.grad_w, first, n) : a.grad_w;
    g.begun = first > 0;
    g.ends = first + n == V;
    g.sums = nullptr;
    if (a.grad_bias && (g.ends || !room.whole_sums)) {
      g.sums = sums;
      g.sum_rows = up(M, kTileM);
      g.sum_cols = room.whole_sums ? V : n;
      g.sum_to = a.grad_bias + (room.whole_sums ? 0 : first);
    }
    if ((e = launch_grad_products(h, g, s, queued)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}
