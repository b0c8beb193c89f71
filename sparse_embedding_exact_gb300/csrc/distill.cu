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
// maximum grows), then q = exp((z - M) / T) / S is written in a second one.
// The row is shared by a cluster of up to 8 blocks, which exchange their (M,
// S) through each other's shared memory, so a step is one launch and a row's
// second read finds it in L2.  The k entries are then written over by one
// thread each, the duplicates of an item summed in list order.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "dense.cuh"

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
template <int kN>
__device__ __forceinline__ void take(Run &a, const float (&z)[kN], float c) {
  float m = z[0];
#pragma unroll
  for (int i = 1; i < kN; ++i) m = fmaxf(m, z[i]);
  if (m > a.m) {
    a.s *= exp2_fast((a.m - m) * c);
    a.m = m;
  }
  const float o = origin(a.m);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kN; ++i) s += exp2_fast((z[i] - o) * c);
  a.s += s;
}

// A row's list in shared memory.
struct List {
  int64_t item[kMostK];  // -1: absent
  float p[kMostK];
  float z[kMostK];  // the student's logits of the present items
  float plogp;      // sum p_j log p_j
  int live;         // an entry is present
};

// The teacher's distribution of row `row`, by one warp.
template <typename T>
__device__ void read_list(const distill_args &a, int64_t row, const T *z, int32_t *status, List &l) {
  const int lane = threadIdx.x & 31;
  const float inv = 1.0f / a.teacher_temperature;
  float sc[kPerLane], most = -INFINITY;
  bool any = false;
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) {
    const int j = u * 32 + lane;
    sc[u] = -INFINITY;
    if (j < a.k) {
      int64_t item = a.items[row * a.k + j];
      const float score = a.scores[row * a.k + j];
      float zj = 0.0f;
      if (item >= a.logits.n_cols) {
        flag(status, DEV_OUT_OF_RANGE);
        item = -1;
      }
      if (item < 0 || score == -INFINITY) {
        item = -1;
      } else {
        zj = Type<T>::up(z[item]);
        if (zj == -INFINITY) item = -1;
      }
      if (item >= 0) {
        sc[u] = score;
        any = true;
        most = max_nan(most, score);
      } else {
        item = -1;
      }
      l.item[j] = item;
      l.z[j] = zj;
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
}

// Calls vec(first column, kVec values) on the aligned body of columns
// [b, e) of the row at z and one(column) on its ragged ends.
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
#pragma unroll
    for (int u = 0; u < 4; ++u) vec(b1 + (v + u * kThreads) * kV, p[u]);
  }
  for (; v < n; v += kThreads) vec(b1 + v * kV, load_pack<T, kV>(z + b1 + v * kV));
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
  const float inv_t = 1.0f / a.temperature, c = kLog2e / a.temperature;
  Run total = {-INFINITY, 0.0f};
  bool live = weight != 0.0f;
  if (live) {  // the same in every block of the cluster
    if (threadIdx.x < 32) read_list<T>(a, row, z, status, list);
    if (kMode != DISTILL_BACKWARD) {
      Run r = {-INFINITY, 0.0f};
      walk(
          z, b, e,
          [&](int64_t, const Pack<T, kV> &p) {
            float f[kV];
            widen(p, f);
            take(r, f, c);
          },
          [&](int64_t col) {
            const float f[1] = {Type<T>::up(z[col])};
            take(r, f, c);
          });
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
    float loss = 0.0f;
    if (live) {
      const float o = origin(total.m), log_s = logf(total.s);
      for (int j = threadIdx.x; j < a.k; j += 32)
        if (list.item[j] >= 0 && !(list.p[j] == 0.0f)) loss += list.p[j] * (log_s - (list.z[j] - o) * inv_t);
      loss = weight * a.temperature * a.temperature * (list.plogp + warp_sum(loss));
    }
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
        [&](int64_t col, const Pack<T, kV> &p) {
          float f[kV];
          widen(p, f);
#pragma unroll
          for (int i = 0; i < kV; ++i) f[i] = f_s * exp2_fast((f[i] - o) * c);
          const Pack<T, kV> out = narrow<T, kV>(f);
          if (same) {
            store_pack(g + col, out);
          } else {
#pragma unroll
            for (int i = 0; i < kV; ++i) g[col + i] = out.v[i];
          }
        },
        [&](int64_t col) { g[col] = Type<T>::down(f_s * exp2_fast((Type<T>::up(z[col]) - o) * c)); });
    __syncthreads();
    for (int j = threadIdx.x; j < a.k; j += kThreads) {
      const int64_t item = list.item[j];
      if (item < b || item >= e) continue;
      bool first = true;
      float p = 0.0f;
      for (int i = 0; i < a.k; ++i)
        if (list.item[i] == item) {
          if (i < j) first = false;
          p += list.p[i];
        }
      if (first) g[item] = Type<T>::down(scale * (exp2_fast((list.z[j] - o) * c) * inv_s - p));
    }
  } else {
    for (int64_t col = b + threadIdx.x; col < e; col += kThreads) g[col] = Type<T>::down(0.0f);
  }
}

template <typename T>
cudaError_t launch_typed(ss_handle *h, const distill_args &a, int32_t mode, cudaStream_t s) {
  const int64_t R = a.logits.n_rows, V = a.logits.n_cols;
  // Blocks a row: while the rows alone leave SMs idle and a block keeps at
  // least 16 KB.
  const int64_t want = 4 * (int64_t)std::max(1, h->sm_count);
  int parts = 1;
  while (parts < kMostCluster && R * parts < want && V / (2 * parts) * (int64_t)sizeof(T) >= 16384) parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(R * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)parts;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = parts > 1 ? 1 : 0;
  auto kernel = mode == DISTILL_FORWARD    ? k_distill<T, DISTILL_FORWARD>
                : mode == DISTILL_BACKWARD ? k_distill<T, DISTILL_BACKWARD>
                                           : k_distill<T, DISTILL_STEP>;
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
