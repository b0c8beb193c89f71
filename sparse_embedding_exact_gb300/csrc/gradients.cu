// The two products of a layer's gradient in one launch.
//
//   grad_x = gz w  (summed over the N features),  grad_w = gz^T x  (over the M rows)
//
// Both cost M N K multiply-adds, but their tiles do not: grad_x has few (M K /
// 256^2) with long sums where a layer is wide, grad_w many with short ones.  On
// their own grad_x leaves SMs idle (2500 x 1024 over 50,176 features: 40 tiles
// of 256 x 256 for 76 pairs of blocks; by blocks of 128 x 256 265 us, where 133
// are the tensor cores' time) and every launch its last turn.  Together they are
// dealt out in advance: one product's tiles evenly, the other's to whoever has
// less, so that all pairs end within a tile of each other.  Where
// grad_x's tiles are too few or too long for that, its sum is split into shares
// (`parts`), each added up in a float32 matrix of its own, which k_finish adds
// up in their order: no atomics, the same bits every time.
//
// Bound by the tensor cores.
#include <algorithm>

#include "product.cuh"

namespace {

using namespace dense;

constexpr int kBN = 256;

// Which tiles a pair of blocks takes: first units of grad_x (a part's tiles side
// by side), then tiles of grad_w.  Pairs below `more` may have other numbers of
// each than the others.
struct Deal {
  int32_t pairs, more;
  int32_t x_more, x_less, w_more, w_less;
  int32_t tiles_m, tiles_k, parts, stages_n, stages_m;
  int32_t units, tiles_w;
};

struct DealWalk {
  Deal d;
  int32_t pair, turn_x, turn_w;
  // The turn-th of a pair that has `mine` of them: turn by turn over all pairs,
  // then over those that have more turns.
  __device__ __forceinline__ int64_t number(int32_t turn, int32_t of_more, int32_t of_less) const {
    const int32_t all = min(of_more, of_less);
    if (turn < all) return (int64_t)turn * d.pairs + pair;
    const bool high = pair < d.more;
    return (int64_t)all * d.pairs + (int64_t)(turn - all) * (high ? d.more : d.pairs - d.more) + (high ? pair : pair - d.more);
  }
  __device__ __forceinline__ bool next(Tile &t) {
    while (turn_x < (pair < d.more ? d.x_more : d.x_less)) {
      const int64_t unit = number(turn_x++, d.x_more, d.x_less);
      if (unit >= d.units) continue;
      const int32_t tiles = d.tiles_m * d.tiles_k, part = (int32_t)unit / tiles, tile = (int32_t)unit % tiles;
      t.ta = tile % d.tiles_m;
      t.tb = tile / d.tiles_m;
      t.k0 = (int32_t)((int64_t)d.stages_n * part / d.parts);
      t.kb = (int32_t)((int64_t)d.stages_n * (part + 1) / d.parts) - t.k0;
      t.kind = 0;
      return true;
    }
    while (turn_w < (pair < d.more ? d.w_more : d.w_less)) {
      const int64_t tile = number(turn_w++, d.w_more, d.w_less);
      if (tile >= d.tiles_w) continue;
      t = {(int32_t)tile / d.tiles_k, (int32_t)tile % d.tiles_k, 0, d.stages_m, 1};
      return true;
    }
    return false;
  }
  // The part of a tile of grad_x, the last that next() gave.
  __device__ __forceinline__ int32_t part() const {
    return d.parts == 1 ? 0 : (int32_t)(number(turn_x - 1, d.x_more, d.x_less) / (d.tiles_m * d.tiles_k));
  }
};

struct Products {
  CUtensorMap a[2], b[2], out[2];
  uint32_t idesc[2];
  Deal deal;
  ss_dense y[2];        // grad_x or the parts (one under the other), and grad_w
  int32_t vec[2];       // their rows start on 16-byte boundaries
  const float *before;  // what earlier calls added up, or null
  int64_t ld_before, part_rows;
  const float *factor, *row_factor;
  int32_t row_step;
  int32_t *status;
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1) k_grad_products(const __grid_constant__ Products a) {
  const int lane = threadIdx.x & 31;
  const int64_t rank_rows = (int64_t)tc::cluster_rank() * kTileM;
  const int32_t pair = (int32_t)(blockIdx.x / 2);
  pair_products<kBN, kMajorByKind, kMajorMN, false, 1>(
      a.a, a.b, a.idesc, a.status, DealWalk{a.deal, pair, 0, 0},
      [&](const DealWalk &w, const Tile &t, int q, int quarter, uint32_t acc, uint32_t boxes, auto release) {
        ss_dense y = a.y[t.kind];
        int64_t under = 0;  // rows of the parts before this one
        if (t.kind == 0 && a.part_rows) {
          under = a.part_rows * w.part();
          y.n_rows = under + a.part_rows;
        }
        const int64_t m0 = t.ta * 2 * kTileM + rank_rows + q * 32, row = under + m0;
        const bool there = row < y.n_rows;
        float factor = 1.0f;
        if (t.kind == 0 && a.row_factor && row + lane < y.n_rows) factor = a.row_factor[(m0 + lane) * a.row_step];
        if (t.kind == 1 && a.factor) factor = *a.factor;
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
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) * factor;
          }
          if (!there || n0 >= y.n_cols) continue;
          if (t.kind == 0 && a.before && row + lane < y.n_rows) {
            const float *p = a.before + (row + lane) * a.ld_before + n0;  // rows of whole 32 values
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 f = reinterpret_cast<const float4 *>(p)[j];
              v[4 * j] += f.x;
              v[4 * j + 1] += f.y;
              v[4 * j + 2] += f.z;
              v[4 * j + 3] += f.w;
            }
          }
          if (t.kind == 0 && a.part_rows) {  // whole rows of the parts: the padding's values stay there
            float *p = static_cast<float *>(y.data) + (row + lane) * y.ld + n0;
            if (row + lane < y.n_rows) {
#pragma unroll
              for (int j = 0; j < 8; ++j) reinterpret_cast<float4 *>(p)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
          } else {
            put32<false>(y, &a.out[t.kind], a.vec[t.kind], boxes, lane, m0, n0, v);
          }
        }
      });
}

// What is left to add up: grad_x of its parts, and the sums of columns (a
// bias's gradient), each in a fixed order.  Blocks of the first kind take rows of
// grad_x, 2^an_x of them one (whole rows left few rows to few blocks: 16 x 4096 x
// 4096 bf16's gradients 44 us, so 31), then come those of 32 columns, eight threads
// a column.
struct Finish {
  const float *parts;
  int64_t ld;
  int32_t n;
  ss_dense out;
  int32_t blocks_x, an_x;
  const float *sums;
  int64_t sum_rows, sum_cols;
  float *sum_to;
};
template <typename T>
__global__ void __launch_bounds__(256) k_finish(const Finish a) {
  tc::wait_before();
  tc::let_next();
  if ((int)blockIdx.x < a.blocks_x) {
    for (int64_t row = blockIdx.x >> a.an_x; row < a.out.n_rows; row += a.blocks_x >> a.an_x)
      for (int64_t c = (int64_t)(blockIdx.x & ((1u << a.an_x) - 1)) * 256 + threadIdx.x; c < a.out.n_cols; c += (int64_t)256 << a.an_x) {
        float v = 0.0f;
#pragma unroll 4
        for (int p = 0; p < a.n; ++p) v += a.parts[((int64_t)p * a.out.n_rows + row) * a.ld + c];
        static_cast<T *>(a.out.data)[row * a.out.ld + c] = Type<T>::down(v);
      }
    return;
  }
  __shared__ float sm[8][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t c = (int64_t)((int)blockIdx.x - a.blocks_x) * 32 + lane;
  float v = 0.0f;
  if (c < a.sum_cols)
#pragma unroll 8
    for (int64_t r = g; r < a.sum_rows; r += 8) v += a.sums[r * a.sum_cols + c];
  sm[g][lane] = v;
  __syncthreads();
  if (g != 0 || c >= a.sum_cols) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) v += sm[k][lane];
  a.sum_to[c] = v;
}

int64_t up(int64_t x, int64_t y) { return (x + y - 1) / y; }
int64_t part_ld(int64_t K) { return up(K, 32) * 32; }

// Clocks of a tile: 590 a stage (512 are the tensor cores' own) and 3,500, or its
// epilogue, as measured over 16 and 64 stages.  (The estimate of a layer's kernel,
// linear.cu, has 600 and 7,000, as its tiles come one after the other without the
// 3,500 and its epilogue does more.)
int64_t clocks_of(int64_t stages) { return std::max<int64_t>(590 * stages + 3500, 6500); }
// The deal for grad_x in `parts` shares, and the clocks until its last pair is
// done.  One product's tiles are spread evenly, the other's go where there is
// room until the least possible end: whichever way round ends sooner.
Deal deal_of(const ss_handle *h, int64_t M, int64_t N, int64_t K, int64_t parts, bool with_x, bool with_w, int64_t *clocks) {
  Deal d = {};
  d.tiles_m = (int32_t)up(M, 256);
  d.tiles_k = (int32_t)up(K, 256);
  d.stages_n = (int32_t)up(N, 64);
  d.stages_m = (int32_t)up(M, 64);
  d.parts = (int32_t)parts;
  d.units = with_x ? d.tiles_m * d.tiles_k * d.parts : 0;
  d.tiles_w = with_w ? (int32_t)up(N, 256) * d.tiles_k : 0;
  const int64_t pairs = std::min<int64_t>(std::max(1, h->sm_count / 2), std::max<int64_t>(1, (int64_t)d.units + d.tiles_w));
  d.pairs = (int32_t)pairs;
  const int64_t cost_x = clocks_of(up(d.stages_n, parts)), cost_w = clocks_of(d.stages_m);
  int64_t best = INT64_MAX;
  for (int even = 0; even < 2; ++even) {
    const int64_t spread = even ? d.tiles_w : d.units, filled = even ? d.units : d.tiles_w;
    const int64_t cost_s = even ? cost_w : cost_x, cost_f = even ? cost_x : cost_w;
    const int64_t more = spread % pairs, n_less = spread / pairs, n_more = n_less + (more > 0);
    const int64_t less_end = n_less * cost_s, more_end = n_more * cost_s;
    auto room = [&](int64_t end) { return (pairs - more) * ((end - less_end) / cost_f) + more * ((end - more_end) / cost_f); };
    // from the mean on, over the ends at which a pair has room for one more
    int64_t lo = std::max(more_end, (filled * cost_f + less_end * (pairs - more) + more_end * more) / pairs);
    while (room(lo) < filled)
      lo = std::min(less_end + ((lo - less_end) / cost_f + 1) * cost_f, more_end + ((lo - more_end) / cost_f + 1) * cost_f);
    if (lo >= best) continue;
    best = lo;
    d.more = (int32_t)more;
    (even ? d.w_less : d.x_less) = (int32_t)n_less;
    (even ? d.w_more : d.x_more) = (int32_t)n_more;
    (even ? d.x_less : d.w_less) = (int32_t)((lo - less_end) / cost_f);
    (even ? d.x_more : d.w_more) = (int32_t)((lo - more_end) / cost_f);
  }
  if (clocks) *clocks = best;
  return d;
}

}  // namespace

int64_t grad_product_parts(const ss_handle *h, int64_t M, int64_t N, int64_t K, int64_t *estimate) {
  int64_t best = 1, least = INT64_MAX;
  for (const int64_t parts : {1, 2, 3, 4, 6, 8, 12, 16}) {
    if (parts > 1 && up(N, 64) / parts < 4) break;
    int64_t clocks;
    deal_of(h, M, N, K, parts, true, true, &clocks);
    // the parts written and read again, at 3,000 bytes a clock, and a launch
    if (parts > 1) clocks += 2 * parts * M * K * 4 / 3000 + 4000;
    if (clocks < least) {
      least = clocks;
      best = parts;
    }
  }
  if (estimate) *estimate = least;
  return best;
}
int64_t grad_part_bytes(int64_t M, int64_t K) { return align_up(M * part_ld(K) * 4); }

cudaError_t launch_grad_products(ss_handle *h, const grad_products &g, cudaStream_t s, int *queued) {
  const int64_t M = g.gz.n_rows, N = g.gz.n_cols, K = g.x.n_cols;
  const bool with_x = g.grad_x.data != nullptr, with_w = g.grad_w.data != nullptr;
  if (!with_x && !with_w && !g.sums) return cudaSuccess;
  Products p = {};
  const int64_t parts = std::min<int64_t>(g.parts, up(N, 64));
  p.deal = deal_of(h, M, N, K, parts, with_x, with_w, nullptr);
  p.factor = g.factor;
  p.row_factor = g.row_factor;
  p.row_step = g.row_step;
  p.status = h->d_status;
  cudaError_t e = cudaSuccess;
  if (with_x) {
    const bool direct = g.parts == 1 && g.ends;
    const ss_dense acc = {g.acc, M * g.parts, K, part_ld(K), SS_VALUES_F32};
    p.y[0] = direct ? g.grad_x : acc;
    p.part_rows = direct ? 0 : M;
    p.before = g.begun ? g.acc : nullptr;
    p.ld_before = part_ld(K);
    p.vec[0] = rows_aligned(p.y[0], 16);
    e = encode(&p.a[0], g.gz, 64, kTileM);
    if (e == cudaSuccess) e = encode(&p.b[0], g.wide, 64, 64);
    if (e == cudaSuccess && direct && p.vec[0]) e = encode_out(&p.out[0], p.y[0]);
    p.idesc[0] = idesc_of(g.gz, kMajorK, kMajorMN, 2 * kTileM, kBN);
  }
  if (e == cudaSuccess && with_w) {
    p.y[1] = g.grad_w;
    p.vec[1] = rows_aligned(g.grad_w, 16);
    e = encode(&p.a[1], g.gz, 64, 64);
    if (e == cudaSuccess) e = encode(&p.b[1], g.x, 64, 64);
    if (e == cudaSuccess && p.vec[1]) e = encode_out(&p.out[1], p.y[1]);
    p.idesc[1] = idesc_of(g.gz, kMajorMN, kMajorMN, 2 * kTileM, kBN);
  }
  if (!with_w) p.a[1] = p.a[0], p.b[1] = p.b[0];  // no tile of that kind, but the maps are fetched
  if (!with_x) p.a[0] = p.a[1], p.b[0] = p.b[1];
  constexpr int kSmem = PairRing<kBN, 1>::kSmem;
  if (e == cudaSuccess) e = ensure_dyn_smem(k_grad_products, kSmem);
  if (e != cudaSuccess) return e;
  if (with_x || with_w) {
    e = launch_beside(k_grad_products, (unsigned)(2 * p.deal.pairs), kPairThreads, kSmem, s, g.beside, p);
    *queued += 1;
  }
  const bool join = with_x && g.ends && g.parts > 1;
  if (e != cudaSuccess || (!join && !g.sums)) return e;
  Finish f = {};
  if (join) {
    f.parts = g.acc;
    f.ld = part_ld(K);
    f.n = g.parts;
    f.out = g.grad_x;
    const int64_t most = 8 * (int64_t)std::max(1, h->sm_count);
    while ((M << (f.an_x + 1)) <= most && ((int64_t)256 << f.an_x) < K) ++f.an_x;
    f.blocks_x = (int32_t)std::min<int64_t>(M << f.an_x, most >> f.an_x << f.an_x);
  }
  f.sums = g.sums;
  f.sum_rows = g.sum_rows;
  f.sum_cols = g.sum_cols;
  f.sum_to = g.sum_to;
  const unsigned blocks = (unsigned)(f.blocks_x + (g.sums ? up(g.sum_cols, 32) : 0));
  *queued += 1;
  auto kernel = g.grad_x.type == SS_VALUES_F32 ? k_finish<float> : g.grad_x.type == SS_VALUES_BF16 ? k_finish<__nv_bfloat16> : k_finish<__half>;
  return launch_beside(kernel, blocks, 256, 0, s, true, f);
}
