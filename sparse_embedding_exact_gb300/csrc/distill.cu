// Distillation from a teacher's k listed scores, and its gradient.
//
// Per row, with z the student's logits over every item, T its temperature,
// and (item_j, score_j) the teacher's list:
//   p = softmax(score / U) over the listed items,   q = softmax(z / T) over all
//   loss = weight T^2 sum_j p_j (log p_j - log q[item_j])
//   dloss / dz_v = weight T (q_v - sum of p_j with item_j = v)
// An item that the student masks (z = -inf) is in neither distribution: its
// q is 0 and a list entry for it counts as absent, like one of item -1 or of
// score -inf.  A row of weight 0, or with no entry left, has loss 0 and
// gradient 0 whatever its logits hold.
//
// Bound by memory: the softmax's maximum M and sum S = sum exp((z - M) / T)
// are taken in one pass over the row (each thread rescales its sum when its
// maximum grows), then q = exp((z - M) / T) / S is written in a second one,
// and the k entries are written over by one thread each, the duplicates of an
// item summed in list order.  A row is shared by a cluster of up to 8 blocks,
// which exchange their (M, S) through each other's shared memory, so every
// call is one launch.  Loss alone and gradient alone stream the row
// (k_distill); a step keeps it on chip between its passes (k_distill_step)
// where 8 blocks can hold it, and reads it a second time where not.
//
// Measured: loss and gradient of 2,500 x 200,000 bf16 logits, top 64, 368 us
// (5.4 TB/s, 80% of the copy bandwidth; streaming it twice 457 us).
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "tc.cuh"

namespace {

using namespace dense;
namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMostK = SS_DISTILL_LIST_MAX;
constexpr int kPerLane = kMostK / 32;
constexpr int kMostCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A running maximum m and s = sum of 2^((z - m) c); m = -inf before any
// unmasked value (s is then 0, or NaN).
struct Run {
  float m, s;
};
// The value subtracted before the exponential: 0 while all is masked.
__device__ __forceinline__ float origin(float m) { return m == -INFINITY ? 0.0f : m; }

__device__ __forceinline__ void join(Run &a, float m, float s, float c) {
  const float M = fmaxf(a.m, m), o = origin(M);
  a.s = a.s * exp2_fast((a.m - o) * c) + s * exp2_fast((m - o) * c);
  a.m = M;
}
// 2^((z - o) c) of both, with `minus` = -o twice.  In pairs of values a step
// takes about 10 instructions a bf16 value, of the 21 that its share of the
// memory's time allows.
__device__ __forceinline__ Two exp_of(Two z, Two minus, Two c) {
  const float2 x = both((z + minus) * c);
  return two(exp2_fast(x.x), exp2_fast(x.y));
}

__device__ __forceinline__ float max_of(const Pack<float, 4> &p) { return fmaxf(fmaxf(p.v[0], p.v[1]), fmaxf(p.v[2], p.v[3])); }
__device__ __forceinline__ float max_of(const Pack<__nv_bfloat16, 8> &p) {
  __nv_bfloat162 q[4];
  memcpy(q, p.w, 16);
  const float2 f = __bfloat1622float2(__hmax2(__hmax2(q[0], q[1]), __hmax2(q[2], q[3])));
  return fmaxf(f.x, f.y);
}
__device__ __forceinline__ float max_of(const Pack<__half, 8> &p) {
  __half2 q[4];
  memcpy(q, p.w, 16);
  const float2 f = __half22float2(__hmax2(__hmax2(q[0], q[1]), __hmax2(q[2], q[3])));
  return fmaxf(f.x, f.y);
}

// Adds kU vectors to a run.
template <typename T, int kV, int kU>
__device__ __forceinline__ void take(Run &a, const Pack<T, kV> (&p)[kU], float c) {
  float m = max_of(p[0]);
#pragma unroll
  for (int u = 1; u < kU; ++u) m = fmaxf(m, max_of(p[u]));
  if (m > a.m) {
    a.s *= exp2_fast((a.m - m) * c);
    a.m = m;
  }
  const float o = origin(a.m);
  const Two minus = two(-o, -o), cc = two(c, c);
  Two s = two(a.s, 0.0f);
#pragma unroll
  for (int u = 0; u < kU; ++u) {
#pragma unroll
    for (int i = 0; i < kV / 2; ++i) s = s + exp_of(pair_of(p[u], i), minus, cc);
  }
  const float2 f = both(s);
  a.s = f.x + f.y;
}
// Adds one value.
__device__ __forceinline__ void take(Run &a, float z, float c) {
  if (z > a.m) {
    a.s *= exp2_fast((a.m - z) * c);
    a.m = z;
  }
  a.s += exp2_fast((z - origin(a.m)) * c);
}
// f_s 2^((z - o) c) of a vector's values, rounded.
template <typename T, int kV>
__device__ __forceinline__ Pack<T, kV> share_of(const Pack<T, kV> &p, float o, float c, float f_s) {
  float f[kV];
#pragma unroll
  for (int i = 0; i < kV / 2; ++i) {
    const float2 q = both(exp_of(pair_of(p, i), two(-o, -o), two(c, c)) * two(f_s, f_s));
    f[2 * i] = q.x;
    f[2 * i + 1] = q.y;
  }
  return narrow<T, kV>(f);
}

// A row's list in shared memory.
struct List {
  int32_t item[kMostK];  // -1: absent
  float p[kMostK];
  float z[kMostK];  // the student's logits of the present items
  float sum[kMostK];  // of p over the entries of the same item, at its first one; -1: not the first
  float plogp;      // sum p_j log p_j
  int live;         // an entry is present
};

// The teacher's distribution of row `row`, by one warp.
template <typename T>
__device__ void read_list(const distill_args &a, int64_t row, const T *z, int32_t *status, List &l) {
  const int lane = threadIdx.x & 31;
  const float inv = 1.0f / a.teacher_temperature;
  // all of a lane's loads of one kind together: three waits, whatever k is
  int64_t item[kPerLane];
  float sc[kPerLane], zj[kPerLane], most = -INFINITY;
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) {
    const int j = u * 32 + lane;
    item[u] = j < a.k ? a.items[row * a.k + j] : -1;
    sc[u] = j < a.k ? a.scores[row * a.k + j] : -INFINITY;
  }
  bool any = false, past = false;
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) {
    past |= item[u] >= a.logits.n_cols;
    if (item[u] >= a.logits.n_cols || sc[u] == -INFINITY) item[u] = -1;
    zj[u] = item[u] >= 0 ? Type<T>::up(z[item[u]]) : -INFINITY;
  }
  if (past) flag(status, DEV_OUT_OF_RANGE);
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) {
    const int j = u * 32 + lane;
    const bool here = item[u] >= 0 && !(zj[u] == -INFINITY);
    if (here) {
      any = true;
      most = max_nan(most, sc[u]);
    }
    if (j < a.k) {
      l.item[j] = here ? (int32_t)item[u] : -1;
      l.z[j] = here ? zj[u] : 0.0f;
    }
  }
  most = warp_max_nan(most);
  any = __any_sync(0xFFFFFFFFu, any);
  float sum = 0.0f;
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) {
    const int j = u * 32 + lane;
    if (j < a.k && l.item[j] >= 0) sum += expf((sc[u] - most) * inv);
  }
  sum = warp_sum(sum);
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) {
    const int j = u * 32 + lane;
    if (j < a.k) l.p[j] = l.item[j] >= 0 ? expf((sc[u] - most) * inv) / sum : 0.0f;
  }
  // sum p log p, where p = exp(t) / sum and t = (score - most) / U
  float h = 0.0f;
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) {
    const int j = u * 32 + lane;
    if (j < a.k && l.item[j] >= 0 && !(l.p[j] == 0.0f)) h += l.p[j] * ((sc[u] - most) * inv - logf(sum));
  }
  h = warp_sum(h);
  if (lane == 0) {
    l.plogp = h;
    l.live = any ? 1 : 0;
  }
  __syncwarp();
  for (int j = lane; j < a.k; j += 32) {
    const int32_t mine = l.item[j];
    float total = 0.0f;
    bool first = mine >= 0;
    for (int i = 0; i < a.k; ++i)
      if (l.item[i] == mine) {
        first = first && i >= j;
        total += l.p[i];
      }
    l.sum[j] = first ? total : -1.0f;
  }
  __syncwarp();
}

// The gradient of the listed items of columns [b, e), over what the pass wrote:
// by one thread each, an item's first entry.
template <typename T>
__device__ __forceinline__ void put_listed(const List &l, int k, T *g, int64_t b, int64_t e, float o, float c, float scale,
                                           float inv_s, int thread, int threads) {
  for (int j = thread; j < k; j += threads) {
    const int64_t item = l.item[j];
    const float sum = l.sum[j];
    if (item >= b && item < e && !(sum == -1.0f)) g[item] = Type<T>::down(scale * (exp2_fast((l.z[j] - o) * c) * inv_s - sum));
  }
}
// The row's loss, by one warp; (M, S) of the student's softmax.
__device__ __forceinline__ float loss_of(const List &l, const distill_args &a, float weight, Run total) {
  if (!l.live) return 0.0f;
  const float o = origin(total.m), log_s = logf(total.s), inv_t = 1.0f / a.temperature;
  float loss = 0.0f;
  for (int j = threadIdx.x & 31; j < a.k; j += 32)
    if (l.item[j] >= 0 && !(l.p[j] == 0.0f)) loss += l.p[j] * (log_s - (l.z[j] - o) * inv_t);
  return weight * a.temperature * a.temperature * (l.plogp + warp_sum(loss));
}

// Calls vec(first column, 1 or 4 vectors kThreads of them apart) on the
// aligned body of columns [b, e) of the row at z and one(column) on its ragged
// ends.
template <typename T, typename Vec, typename One>
__device__ __forceinline__ void walk(const T *z, int64_t b, int64_t e, Vec vec, One one) {
  constexpr int kV = Type<T>::kVec;
  const int64_t off = (int64_t)((reinterpret_cast<uintptr_t>(z + b) & 15) / sizeof(T));
  const int64_t b1 = min(e, b + (off ? kV - off : 0));
  const int64_t n = (e - b1) / kV, e1 = b1 + n * kV;
  if ((int64_t)threadIdx.x < b1 - b) one(b + threadIdx.x);
  int64_t v = threadIdx.x;
  for (; v + 3 * kThreads < n; v += 4 * kThreads) {
    Pack<T, kV> p[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) p[u] = load_pack<T, kV>(z + b1 + (v + u * kThreads) * kV);
    vec(b1 + v * kV, p);
  }
  for (; v < n; v += kThreads) {
    const Pack<T, kV> p[1] = {load_pack<T, kV>(z + b1 + v * kV)};
    vec(b1 + v * kV, p);
  }
  if ((int64_t)threadIdx.x < e - e1) one(e1 + threadIdx.x);
}

template <typename T, int kMode>
__global__ void __launch_bounds__(kThreads) k_distill(const distill_args a, int n_part, int32_t *status) {
  constexpr int kV = Type<T>::kVec;
  __shared__ List list;
  __shared__ Run warp_run[kWarps];
  __shared__ Run block_run;
  const int64_t row = blockIdx.x / n_part, V = a.logits.n_cols;
  const int part = (int)(blockIdx.x % n_part);
  // whole 16-byte units a block, so that all but the last part stay aligned
  const int64_t width = ((V + n_part - 1) / n_part + kV - 1) / kV * kV;
  const int64_t b = min(V, part * width), e = min(V, b + width);
  const T *z = static_cast<const T *>(a.logits.data) + row * a.logits.ld;
  T *g = static_cast<T *>(a.grad_logits.data) + row * a.grad_logits.ld;
  const float weight = a.weight ? a.weight[row] : 1.0f;
  const float c = kLog2e / a.temperature;
  Run total = {-INFINITY, 0.0f};
  bool live = weight != 0.0f;
  if (live) {  // the same in every block of the cluster
    if (threadIdx.x < 32) read_list<T>(a, row, z, status, list);
    if (kMode != DISTILL_BACKWARD) {
      Run r = {-INFINITY, 0.0f};
      walk(
          z, b, e,
          [&](int64_t, const auto &p) { take(r, p, c); }, [&](int64_t col) { take(r, Type<T>::up(z[col]), c); });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float m = __shfl_xor_sync(0xFFFFFFFFu, r.m, o), s = __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
        join(r, m, s, c);
      }
      if ((threadIdx.x & 31) == 0) warp_run[threadIdx.x >> 5] = r;
      __syncthreads();
      if (threadIdx.x == 0) {
        r = warp_run[0];
        for (int w = 1; w < kWarps; ++w) join(r, warp_run[w].m, warp_run[w].s, c);
        block_run = r;
      }
      if (n_part > 1) {
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        for (int q = 0; q < n_part; ++q) {
          const Run o = *cl.map_shared_rank(&block_run, q);
          join(total, o.m, o.s, c);
        }
        cl.sync();  // no block leaves or writes while another reads
      } else {
        __syncthreads();
        total = block_run;
      }
    } else {
      __syncthreads();
      total.m = a.stats[2 * row];
      total.s = a.stats[2 * row + 1];
    }
    live = list.live != 0;
  }
  if (kMode != DISTILL_BACKWARD && part == 0 && threadIdx.x < 32) {
    const float loss = live ? loss_of(list, a, weight, total) : 0.0f;
    if (threadIdx.x == 0) {
      a.loss[row] = loss;
      if (kMode == DISTILL_FORWARD) {
        a.stats[2 * row] = live ? total.m : 0.0f;
        a.stats[2 * row + 1] = live ? total.s : 0.0f;
      }
    }
  }
  if (kMode == DISTILL_FORWARD) return;

  const float scale = live ? weight * (a.grad_loss ? a.grad_loss[row] : 1.0f) * a.temperature : 0.0f;
  const bool same = ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
  const float o = origin(total.m), inv_s = 1.0f / total.s;
  if (live) {
    const float f_s = scale * inv_s;
    walk(
        z, b, e,
        [&](int64_t col, const auto &p) {
#pragma unroll
          for (int u = 0; u < (int)(sizeof(p) / sizeof(p[0])); ++u) {
            const Pack<T, kV> out = share_of(p[u], o, c, f_s);
            T *to = g + col + (int64_t)u * kThreads * kV;
            if (same) {
              store_pack(to, out);
            } else {
#pragma unroll
              for (int i = 0; i < kV; ++i) to[i] = item(out, i);
            }
          }
        },
        [&](int64_t col) { g[col] = Type<T>::down(f_s * exp2_fast((Type<T>::up(z[col]) - o) * c)); });
    __syncthreads();
    put_listed(list, a.k, g, b, e, o, c, scale, inv_s, threadIdx.x, kThreads);
  } else {
    for (int64_t col = b + threadIdx.x; col < e; col += kThreads) g[col] = Type<T>::down(0.0f);
  }
}

// ---------------------------------------------------------------- a step with its rows on chip
// A cluster takes a row, each block an equal part of it, which stays in shared
// memory from its only read to the gradient's write.  A warp of its own copies
// the next row's part chunk by chunk into the places that the gradient's pass
// leaves, another reads the lists a row ahead, so that copies, both passes and
// stores of two blocks an SM overlap.
//
// The grid has a cluster for each row; those that run take over the rows of
// those that have not started (cluster launch control) until none is left.
// With every n-th row a cluster, the blocks that an SM favours (the older of
// its two) were done after 310 us of 420.
constexpr int kChunk = 8192;                       // bytes
constexpr int kChunkUnits = kChunk / 16;
constexpr int kStepWorkers = 512, kStepWarps = kStepWorkers / 32;
constexpr int kU = 2 * kChunkUnits / kStepWorkers;  // vectors a thread of two chunks
static_assert(kU * kStepWorkers == 2 * kChunkUnits, "whole vectors");
constexpr int kAsked = 4;                          // rows known or asked for ahead
constexpr int kMostChunks = 13;                    // of a block: two blocks an SM
constexpr int kStepThreads = kStepWorkers + 64;
constexpr int kStepSmem = kMostChunks * kChunk + 128;

// The bytes of a row at `z` that block `part` of `n_part` works on, counted
// from the row's start rounded down to 16: [lo, hi), lo a multiple of 16; and
// the whole 16-byte units [in_lo, in_hi) of the row within it.
struct Part {
  int64_t lo, hi, in_lo, in_hi, off;
  int chunks;
  __device__ __forceinline__ int bytes(int j) const {
    const int64_t left = in_hi - in_lo - (int64_t)j * kChunk;
    return (int)max((int64_t)0, min((int64_t)kChunk, left));
  }
};
// Bytes and chunks of a part, the same for every row (the last chunks perhaps empty).
template <typename T>
__device__ __forceinline__ int64_t width_of(int64_t V, int n_part) {
  return ((V * (int64_t)sizeof(T) + 15) / 16 + 1 + n_part - 1) / n_part * 16;
}
template <typename T>
__device__ __forceinline__ int chunks_of(int64_t V, int n_part) {
  return (int)((width_of<T>(V, n_part) + kChunk - 1) / kChunk);
}
template <typename T>
__device__ __forceinline__ Part part_of(const T *z, int64_t V, int part, int n_part) {
  Part p;
  p.off = (int64_t)(reinterpret_cast<uintptr_t>(z) & 15);
  const int64_t end = p.off + V * (int64_t)sizeof(T);
  const int64_t width = width_of<T>(V, n_part);
  p.lo = min(end, part * width);
  p.hi = min(end, p.lo + width);
  p.in_lo = p.lo == 0 && p.off ? 16 : p.lo;
  p.in_hi = p.hi & ~(int64_t)15;
  if (p.in_hi < p.in_lo) p.in_hi = p.in_lo;
  p.chunks = chunks_of<T>(V, n_part);
  return p;
}

template <typename T>
__global__ void __launch_bounds__(kStepThreads, 2) k_distill_step(const distill_args a, int n_part, int32_t *status) {
  constexpr int kV = Type<T>::kVec;
  extern __shared__ unsigned char raw[];
  __shared__ List lists[2];
  __shared__ Run warp_run[kStepWarps];
  __shared__ float2 exchange[2][kMostCluster];
  __shared__ Run result[2];
  __shared__ int64_t row_of[2];
  __shared__ __align__(16) uint4 answers[kAsked];
  __shared__ __align__(8) uint64_t bars[2 * kMostChunks + 8 + kAsked];
  __shared__ volatile int stalled;
  __shared__ int64_t worker_row[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = (tc::smem_u32(raw) + 127u) & ~127u;
  auto full = [&](int j) { return tc::smem_u32(&bars[j]); };
  auto used = [&](int j) { return tc::smem_u32(&bars[kMostChunks + j]); };
  auto list_full = [&](int i) { return tc::smem_u32(&bars[2 * kMostChunks + i]); };
  auto list_free = [&](int i) { return tc::smem_u32(&bars[2 * kMostChunks + 2 + i]); };
  auto met = [&](int i) { return tc::smem_u32(&bars[2 * kMostChunks + 4 + i]); };  // the cluster's (M, S)
  auto row_full = [&](int i) { return tc::smem_u32(&bars[2 * kMostChunks + 6 + i]); };
  auto answered = [&](int q) { return tc::smem_u32(&bars[2 * kMostChunks + 8 + q]); };
  if (tid == 0) {
    stalled = 0;
    for (int j = 0; j < kMostChunks; ++j) {
      tc::bar_init(full(j), 1);
      tc::bar_init(used(j), kStepWarps);
    }
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(list_full(i), 1);
      tc::bar_init(list_free(i), kStepWarps + 1);
      tc::bar_init(met(i), 1);
      tc::bar_init(row_full(i), 1);
    }
    for (int q = 0; q < kAsked; ++q) tc::bar_init(answered(q), 1);
    tc::bar_init_fence();
  }
  __syncthreads();
  tc::cluster_sync();  // every block's barriers exist before one is signalled
  const int64_t V = a.logits.n_cols;
  const int part = (int)(blockIdx.x % n_part);
  const float c = kLog2e / a.temperature;
  // The long part of a wait out of line for 16-bit logits (2,500 x 200,000: 374 us,
  // 379 in line), in line for float32 (660 us, 683 out of line, where the calls
  // spill).
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return sizeof(T) == 4 ? tc::bar_wait_on(bar, parity, status, &stalled) : tc::bar_wait_far(bar, parity, status, &stalled);
  };
  // Row n of this cluster (-1: no more); its list's place, and the list's
  // barriers, are those of n & 1.
  auto row_at = [&](int64_t n) {
    const int i = (int)(n & 1);
    wait(row_full(i), (uint32_t)((n >> 1) & 1));
    return stalled ? (int64_t)-1 : row_of[i];
  };

  if (warp == kStepWarps) {
    // ---- copies: each chunk as the gradient's pass of the row before leaves it
    int64_t loaded = 0;  // rows of weight other than 0 so far
    int issued = 0;      // chunks of the last of them (lane 0)
    for (int64_t n = 0;; ++n) {
      const int64_t row = row_at(n);
      if (row < 0) break;
      if (!(a.weight && a.weight[row] == 0.0f)) {
        const T *z = static_cast<const T *>(a.logits.data) + row * a.logits.ld;
        const Part p = part_of(z, V, part, n_part);
        if (lane == 0) {
          const unsigned char *base = reinterpret_cast<const unsigned char *>(z) - p.off;
          for (issued = 0; issued < p.chunks; ++issued) {
            const int j = issued;
            const uint32_t bytes = (uint32_t)p.bytes(j);
            // (a place that may still be read is not written over)
            if (loaded > 0 && !wait(used(j), (uint32_t)((loaded - 1) & 1))) break;
            tc::bar_expect(full(j), bytes);
            if (bytes) tc::load_bulk(ring + (uint32_t)j * kChunk, base + p.in_lo + (int64_t)j * kChunk, bytes, full(j));
          }
        }
        ++loaded;
      }
      __syncwarp();
      if (lane == 0) tc::bar_arrive(list_free((int)(n & 1)));
    }
    // After a wait that ran out the copies under way may not be read by anyone:
    // the last one of each chunk lands before the block leaves.
    if (stalled && lane == 0)
      for (int j = 0; j < kMostChunks; ++j) {
        const int64_t copies = loaded - (j < issued ? 0 : 1);
        if (copies > 0 && j < chunks_of<T>(V, n_part)) wait(full(j), (uint32_t)((copies - 1) & 1));
      }
  } else if (warp == kStepWarps + 1) {
    // ---- rows and lists, a row ahead of their use (the list's three loads
    // depend on each other: with the copies they held them up by 5 us a row),
    // and losses
    float weights[2] = {0.0f, 0.0f};
    // Everyone is done with row m of this cluster: its loss (by the first
    // block), before its place is used again.  Every block of the cluster has
    // passed the exchange of row m, so has read the answer that gave it, and
    // the next one may be written over that.
    auto finish = [&](int64_t m, bool more) {
      const int i = (int)(m & 1);
      wait(list_free(i), (uint32_t)((m >> 1) & 1));
      if (part != 0) return;
      if (more && lane == 0 && !stalled) {
        tc::fence_async();
        tc::ask_for_cluster(tc::smem_u32(&answers[(m + kAsked) % kAsked]), answered((int)(m % kAsked)));
      }
      const float loss = weights[i] != 0.0f ? loss_of(lists[i], a, weights[i], result[i]) : 0.0f;
      if (lane == 0) a.loss[row_of[i]] = loss;
    };
    if (part == 0 && lane == 0)
      for (int q = 1; q < kAsked; ++q) tc::ask_for_cluster(tc::smem_u32(&answers[q]), answered(q));
    // Answer n is asked for by the first block before (n < kAsked) or when row
    // n - kAsked is finished; row 0 is the cluster's own.
    auto answer = [&](int64_t n) {
      const int q = (int)(n % kAsked);
      if (lane == 0) tc::bar_expect(answered(q), 16);
      __syncwarp();
      wait(answered(q), (uint32_t)((n / kAsked - (q == 0)) & 1));
      return tc::cluster_given(tc::smem_u32(&answers[q]));
    };
    int64_t n = 0, asked = kAsked;  // answers asked for so far, with row 0
    for (;; ++n) {
      const int i = (int)(n & 1);
      if (n >= 2) {
        finish(n - 2, true);
        ++asked;
      }
      const int64_t x = n == 0 ? (int64_t)(blockIdx.x / n_part) * n_part : answer(n);
      const int64_t row = x < 0 || stalled ? -1 : x / n_part;
      if (lane == 0) {
        row_of[i] = row;
        tc::bar_arrive(row_full(i));
      }
      __syncwarp();
      if (row < 0) break;
      weights[i] = a.weight ? a.weight[row] : 1.0f;
      if (weights[i] != 0.0f) {
        read_list<T>(a, row, static_cast<const T *>(a.logits.data) + row * a.logits.ld, status, lists[i]);
        if (lane == 0) tc::bar_arrive(list_full(i));
      }
    }
    // Answer n said that none is left: those asked for after it say the same,
    // and are waited for, as they are written to every block.
    for (int64_t k = n + 1; k < asked; ++k) answer(k);
    if (n >= 1) finish(n - 1, false);
  } else {
    int64_t loaded = 0;        // rows of weight other than 0 so far
    uint32_t lists_read = 0;   // bit i: the parity of those in place i
    for (int64_t n = 0;; ++n) {
      // One row for all of the workers, who meet at barriers, also where a wait
      // ran out.
      const int i = (int)(n & 1);
      if (warp == 0) {
        const int64_t r = row_at(n);
        if (lane == 0) worker_row[i] = r;
      }
      tc::named_sync(1, kStepWorkers);
      const int64_t row = worker_row[i];
      if (row < 0) break;
      // (M, S) of this block's part to the others, by warp 0.  As a counted
      // store: an arrival would wait for the gradient's stores of the row
      // before (5 us a row, of 15).
      auto meet = [&](Run r) {
        if (warp == 0) {
          if (lane == 0) tc::bar_expect(met(i), 8u * n_part);
          if (lane < n_part)
            tc::send_remote(tc::map_rank(tc::smem_u32(&exchange[i][part]), (uint32_t)lane), r.m, r.s,
                            tc::map_rank(met(i), (uint32_t)lane));
        }
        wait(met(i), (uint32_t)((n >> 1) & 1));
      };
      const T *z = static_cast<const T *>(a.logits.data) + row * a.logits.ld;
      T *g = static_cast<T *>(a.grad_logits.data) + row * a.grad_logits.ld;
      const Part p = part_of(z, V, part, n_part);
      const int64_t b = max((int64_t)0, p.lo - p.off) / (int64_t)sizeof(T), e = (p.hi - p.off) / (int64_t)sizeof(T);
      const float weight = a.weight ? a.weight[row] : 1.0f;
      if (weight == 0.0f) {
        for (int64_t col = b + tid; col < e; col += kStepWorkers) g[col] = Type<T>::down(0.0f);
        meet({0.0f, 0.0f});
        if (lane == 0) tc::bar_arrive(list_free(i));
        continue;
      }
      // values outside whole units: at most 7 at either end of the row
      const int64_t c0 = (p.in_lo - p.off) / (int64_t)sizeof(T), c1 = (p.in_hi - p.off) / (int64_t)sizeof(T);
      const int64_t head = p.in_hi > p.in_lo ? c0 - b : e - b, tail = p.in_hi > p.in_lo ? e - c1 : 0;
      int64_t edge = -1;
      if (tid < head)
        edge = b + tid;
      else if (tid - head < tail)
        edge = c1 + (tid - head);
      const uint32_t parity = (uint32_t)(loaded & 1);
      ++loaded;
      Run r = {-INFINITY, 0.0f};
      float at_edge = 0.0f;
      if (edge >= 0) {
        at_edge = Type<T>::up(z[edge]);
        take(r, at_edge, c);
      }
      // two chunks at a time
      const int units = (int)((p.in_hi - p.in_lo) / 16);
      for (int j = 0; j < p.chunks; j += 2) {
        wait(full(j), parity);
        if (j + 1 < p.chunks) wait(full(j + 1), parity);
        Pack<T, kV> q[kU];
        if ((j + 2) * kChunkUnits <= units) {
#pragma unroll
          for (int u = 0; u < kU; ++u) q[u] = tc::read_shared<Pack<T, kV>>(ring + 16u * (j * kChunkUnits + tid + u * kStepWorkers));
          take(r, q, c);
        } else {
          for (int v = j * kChunkUnits + tid; v < units; v += kStepWorkers) {
            const Pack<T, kV> last[1] = {tc::read_shared<Pack<T, kV>>(ring + 16u * v)};
            take(r, last, c);
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float m = __shfl_xor_sync(0xFFFFFFFFu, r.m, o), s = __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
        join(r, m, s, c);
      }
      if (lane == 0) warp_run[warp] = r;
      // The list is read before this block lets the others go on: with the
      // gradient in the logits' place they would write over what it reads.
      wait(list_full(i), (uint32_t)((lists_read >> i) & 1));
      lists_read ^= 1u << i;
      const List &list = lists[i];
      tc::named_sync(1, kStepWorkers);
      if (warp == 0) {
        r = warp_run[lane % kStepWarps];
#pragma unroll
        for (int o = kStepWarps / 2; o > 0; o >>= 1) {
          const float m = __shfl_xor_sync(0xFFFFFFFFu, r.m, o), s = __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
          join(r, m, s, c);
        }
      }
      meet(r);
      Run total = {exchange[i][0].x, exchange[i][0].y};
      for (int q = 1; q < n_part; ++q) join(total, exchange[i][q].x, exchange[i][q].y, c);
      const bool live = list.live != 0;
      const float o = origin(total.m), inv_s = 1.0f / total.s;
      if (tid == 0) result[i] = total;
      const float scale = live ? weight * (a.grad_loss ? a.grad_loss[row] : 1.0f) * a.temperature : 0.0f;
      const float f_s = scale * inv_s;
      const bool same = ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
      T *body = g + c0;
      auto put = [&](int v, const Pack<T, kV> &q) {
        const Pack<T, kV> out = share_of(q, o, c, f_s);
        T *to = body + (int64_t)v * kV;
        if (same) {
          store_pack(to, out);
        } else {
#pragma unroll
          for (int i = 0; i < kV; ++i) to[i] = item(out, i);
        }
      };
      for (int j = 0; j < p.chunks; j += 2) {
        if (!live) {
          for (int v = j * kChunkUnits + tid; v < min(units, (j + 2) * kChunkUnits); v += kStepWorkers) {
#pragma unroll
            for (int i = 0; i < kV; ++i) body[(int64_t)v * kV + i] = Type<T>::down(0.0f);
          }
        } else if ((j + 2) * kChunkUnits <= units) {
          Pack<T, kV> q[kU];
#pragma unroll
          for (int u = 0; u < kU; ++u) q[u] = tc::read_shared<Pack<T, kV>>(ring + 16u * (j * kChunkUnits + tid + u * kStepWorkers));
#pragma unroll
          for (int u = 0; u < kU; ++u) put(j * kChunkUnits + tid + u * kStepWorkers, q[u]);
        } else {
          for (int v = j * kChunkUnits + tid; v < units; v += kStepWorkers) put(v, tc::read_shared<Pack<T, kV>>(ring + 16u * v));
        }
        __syncwarp();
        if (lane == 0) {
          tc::bar_arrive(used(j));
          if (j + 1 < p.chunks) tc::bar_arrive(used(j + 1));
        }
      }
      if (edge >= 0) g[edge] = Type<T>::down(live ? f_s * exp2_fast((at_edge - o) * c) : 0.0f);
      // the listed items over what was just written
      tc::named_sync(1, kStepWorkers);
      if (live) put_listed(list, a.k, g, b, e, o, c, scale, inv_s, tid, kStepWorkers);
      __syncwarp();
      if (lane == 0) tc::bar_arrive(list_free(i));
    }
  }
  __syncthreads();
  tc::cluster_sync();  // no block leaves while another writes to its exchange
}

template <typename T>
cudaError_t launch_typed(ss_handle *h, const distill_args &a, int32_t mode, cudaStream_t s) {
  const int64_t R = a.logits.n_rows, V = a.logits.n_cols;
  cudaLaunchAttribute at[1];
  auto config = [&](int64_t blocks, int threads, int smem, int n_part) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)n_part;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cfg;
  };
  // Blocks a row: while the rows alone leave SMs idle and a block keeps at
  // least 16 KB.
  const int64_t sms = std::max(1, h->sm_count), bytes = V * (int64_t)sizeof(T);
  int parts = 1;
  while (parts < kMostCluster && R * parts < 4 * sms && bytes / (2 * parts) >= 16384) parts *= 2;
  if (mode == DISTILL_STEP) {
    int on_chip = parts;
    while (on_chip < kMostCluster && (bytes + 32) / on_chip + 32 > (int64_t)kMostChunks * kChunk) on_chip *= 2;
    if ((bytes + 32) / on_chip + 32 <= (int64_t)kMostChunks * kChunk) {
      auto step = k_distill_step<T>;
      const cudaError_t e = ensure_dyn_smem(step, kStepSmem);
      if (e != cudaSuccess) return e;
      const cudaLaunchConfig_t cfg = config(R * on_chip, kStepThreads, kStepSmem, on_chip);
      return cudaLaunchKernelEx(&cfg, step, a, on_chip, h->d_status);
    }
    // wider rows: parts small enough that those of the resident blocks stay in
    // L2 for the second read
    parts = kMostCluster;
  }
  auto kernel = mode == DISTILL_FORWARD    ? k_distill<T, DISTILL_FORWARD>
                : mode == DISTILL_BACKWARD ? k_distill<T, DISTILL_BACKWARD>
                                           : k_distill<T, DISTILL_STEP>;
  const cudaLaunchConfig_t cfg = config(R * parts, kThreads, 0, parts);
  return cudaLaunchKernelEx(&cfg, kernel, a, parts, h->d_status);
}

}  // namespace

cudaError_t launch_distill(ss_handle *h, const distill_args &a, int32_t mode, cudaStream_t s, int *queued) {
  *queued = 1;
  switch (a.logits.type) {
    case SS_VALUES_F32:
      return launch_typed<float>(h, a, mode, s);
    case SS_VALUES_BF16:
      return launch_typed<__nv_bfloat16>(h, a, mode, s);
    default:
      return launch_typed<__half>(h, a, mode, s);
  }
}
