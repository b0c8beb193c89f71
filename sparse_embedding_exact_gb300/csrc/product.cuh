// Shared by the dense products (linear.cu, cross_entropy.cu): tiles and rings,
// the epilogue's boxes, products by pairs of blocks and tensor maps.
#pragma once

#include <algorithm>
#include <mutex>
#include <utility>

#include "tc.cuh"

namespace dense {

constexpr int kTileM = 128;     // rows of A a block's tile
constexpr int kRowBytes = 128;  // of the summed dimension a stage, both operands
constexpr int kSmemMost = 227 * 1024;
constexpr int kStaging = 32 * 64;  // an epilogue warp's box: 32 rows of 64 bytes

enum : int { kMajorK = 0, kMajorMN = 1, kMajorByKind = 2 };  // by a tile's kind: 0 along the sum, 1 across it

// ---------------------------------------------------------------- boxes
// An epilogue warp takes 32 rows x 32 columns at a time.  Its boxes in shared
// memory have 32 rows of 64 bytes in the 64-byte swizzle of tensor copies
// (16-byte unit j of row r at j ^ (r / 2 % 4)): eight lanes with a row each, or
// four with a row's units, meet no bank twice.
__device__ __forceinline__ uint32_t unit_at(uint32_t box, int row, int unit) {
  return box + (uint32_t)(row * 64 + ((unit ^ (row >> 1 & 3)) << 4));
}

// Writes kN values of 64 bytes together, this lane's row.
template <typename T, int kN>
__device__ __forceinline__ void put_row(uint32_t box, int lane, const float *v) {
  constexpr int kV = Type<T>::kVec;
#pragma unroll
  for (int j = 0; j < kN / kV; ++j) {
    float f[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) f[i] = v[j * kV + i];
    const Pack<T, kV> p = narrow<T, kV>(f);
    uint4 q;
    memcpy(&q, &p, 16);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(unit_at(box, lane, j)), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w)
                 : "memory");
  }
}
// The box's values to rows that start anywhere: row after row, the lanes along
// it.  16-bit values go two rows at a time in words, of columns 2 l and 2 l + 1
// where the row starts on a word, else of 2 l + 1 and 2 l + 2 between its first
// and its last value; one by one at the matrix's edge.
template <typename U, bool kWords>
__device__ __forceinline__ void store_ragged(const ss_dense &out, uint32_t box, int lane, int64_t m0, int64_t n) {
  constexpr int kCols = 64 / (int)sizeof(U), kPer = 16 / (int)sizeof(U);
  if constexpr (sizeof(U) == 2 && kWords) {
    if (n + 32 <= out.n_cols) {
      const int l = lane % 16;
      uint16_t *base = static_cast<uint16_t *>(out.data) + m0 * out.ld + n;
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int r = i / 2 * 4 + i % 2 + lane / 16 * 2;  // rows two apart start alike
        uint16_t *to = base + r * out.ld;
        const uint32_t w = tc::read_shared<uint32_t>(unit_at(box, r, l / 4) + (uint32_t)(l % 4 * 4));
        const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, w, 1);
        if (m0 + r >= out.n_rows) continue;
        if (reinterpret_cast<uintptr_t>(to) & 2) {
          if (l < 15) *reinterpret_cast<uint32_t *>(to + 2 * l + 1) = __funnelshift_r(w, next, 16);
          if (l % 15 == 0) to[l == 0 ? 0 : 31] = (uint16_t)(l == 0 ? w : w >> 16);
        } else {
          *reinterpret_cast<uint32_t *>(to + 2 * l) = w;
        }
      }
      return;
    }
  }
  U *to = static_cast<U *>(out.data) + m0 * out.ld + n + lane % kCols;
#pragma unroll 8
  for (int r = lane / kCols; r < 32; r += 32 / kCols) {
    const int c = lane % kCols;
    if (m0 + r < out.n_rows && n + c < out.n_cols)
      to[r * out.ld] = tc::read_shared<U>(unit_at(box, r, c / kPer) + (uint32_t)(c % kPer * sizeof(U)));
  }
}
// Writes 32 values of each lane's row (rows m0 + lane, columns n0 ..) to the
// matrix of `map`, through the warp's box.  kWords: 16-bit values to rows that
// start anywhere in words.  (A layer's epilogue with everything in it has no
// registers for them, nor have a gradient's two products: 4000 x 1001 x 2777 bf16
// with residual and kept pre-activation 95 us, value by value 91, its gradients 89
// and 87; with bias and activation alone 44 and 46.)
template <bool kWords>
__device__ __forceinline__ void put32(const ss_dense &out, const CUtensorMap *map, bool vec, uint32_t box, int lane, int64_t m0,
                                      int64_t n0, const float (&v)[32]) {
  const bool wide = out.type == SS_VALUES_F32;
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    if (part && !wide) break;
    const int64_t n = n0 + 16 * part;
    if (lane == 0) tc::store_wait_read();  // the box's last copy out
    __syncwarp();
    if (wide)
      put_row<float, 16>(box, lane, v + 16 * part);
    else if (out.type == SS_VALUES_BF16)
      put_row<__nv_bfloat16, 32>(box, lane, v);
    else
      put_row<__half, 32>(box, lane, v);
    if (vec) {
      tc::fence_async();
      __syncwarp();
      if (lane == 0) {
        if (n < out.n_cols && m0 < out.n_rows) tc::store_2d(map, box, (int)n, (int)m0);
        tc::store_commit();
      }
    } else {
      __syncwarp();
      if (wide)
        store_ragged<uint32_t, kWords>(out, box, lane, m0, n);
      else
        store_ragged<uint16_t, kWords>(out, box, lane, m0, n);
      __syncwarp();
    }
  }
}

// Calls f(i, p[i]) for 32 columns (`n` of them exist): the same addresses in
// every lane, four at a time where they are aligned.
template <typename F>
__device__ __forceinline__ void along32(const float *p, int64_t n, F f) {
  if (n >= 32 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 q = __ldg(reinterpret_cast<const float4 *>(p) + j);
      f(4 * j, q.x);
      f(4 * j + 1, q.y);
      f(4 * j + 2, q.z);
      f(4 * j + 3, q.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) f(i, i < n ? __ldg(p + i) : 0.0f);
  }
}

// ---------------------------------------------------------------- products by pairs of blocks
constexpr int kEpiWarps = 16;                   // four for each 32 tensor-memory lanes, a quarter of the columns each
constexpr int kPairThreads = 64 + 32 * kEpiWarps;

// kBoxesEach: staging boxes of an epilogue warp.
template <int kBN, int kBoxesEach>
struct PairRing {
  static constexpr int kBytesA = kTileM * kRowBytes, kBytesB = kBN / 2 * kRowBytes;
  static constexpr int kStage = kBytesA + kBytesB;  // a block's part
  static constexpr int kBoxes = kEpiWarps * kBoxesEach * kStaging;
  static constexpr int kStages = (kSmemMost - 2048 - kBoxes) / kStage;
  static constexpr int kSmem = kStages * kStage + kBoxes + 1024;
};

// A tile's place, its share of the summed dimension (stages k0 to k0 + kb) and,
// where a kernel has two products, whose it is.
struct Tile {
  int32_t ta, tb;
  int32_t k0, kb, kind;
};

// Every n-th tile of p's tiles_a x tiles_b, from `tile` on (fewer than 2^31, as the
// output is in memory); down groups of 8 tile rows, so that the tiles in flight
// share both operands in L2.
template <typename P>
struct TileWalk {
  const P &p;
  int32_t tile;
  __device__ __forceinline__ bool next(Tile &t) {
    if (tile >= p.tiles_a * p.tiles_b) return false;
    const int32_t group = 8 * p.tiles_b, in = tile % group, g0 = tile / group * 8, gh = min(8, p.tiles_a - g0);
    t = {g0 + in % gh, in / gh, 0, p.blocks_k, 0};
    tile += (int32_t)(gridDim.x / 2);
    return true;
  }
};

// The body of a persistent kernel of pairs of blocks (clusters of two, of
// kPairThreads): tiles of 256 x kBN of the products of `map_a` and `map_b` (one a
// kind, and an `idesc`), the ones that `walk` gives this pair.  Each tile goes to
// epi(w, tile, q, quarter, acc, boxes, release) in every epilogue warp, w the
// walk past this tile: rows q * 32 + lane of this
// block's 128, columns quarter * kBN / 4 on, accumulators from column 0 of the
// tile at tensor-memory address `acc`, the warp's boxes; it calls release()
// once, after its last load of them.  Copies out are waited for here.
template <int kBN, int kMajA, int kMajB, bool kF8, int kBoxesEach, typename Walk, typename Epi>
__device__ __forceinline__ void pair_products(const CUtensorMap *map_a, const CUtensorMap *map_b, const uint32_t *idesc,
                                              int32_t *status, const Walk walk, Epi epi) {
  using R = PairRing<kBN, kBoxesEach>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t bars[2 * R::kStages + 4];
  __shared__ uint32_t tmem_slot;
  __shared__ int stalled;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = (tc::smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t rank = tc::cluster_rank();
  auto full = [&](int s) { return tc::smem_u32(&bars[s]); };
  auto empty = [&](int s) { return tc::smem_u32(&bars[R::kStages + s]); };
  auto acc_full = [&](int b) { return tc::smem_u32(&bars[2 * R::kStages + b]); };
  auto acc_free = [&](int b) { return tc::smem_u32(&bars[2 * R::kStages + 2 + b]); };
  constexpr uint32_t kCols = 2 * kBN;
  if (tid == 0) {
    stalled = 0;
    for (int i = 0; i < 2 * R::kStages + 2; ++i) tc::bar_init(tc::smem_u32(&bars[i]), 1);
    for (int b = 0; b < 2; ++b) tc::bar_init(acc_free(b), 2 * kEpiWarps);
    tc::bar_init_fence();
    for (int i = 0; i < (kMajA == kMajorByKind ? 2 : 1); ++i) {
      tc::prefetch_map(map_a + i);
      tc::prefetch_map(map_b + i);
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(&tmem_slot)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    tc::fence_before();
  }
  __syncthreads();
  tc::cluster_sync();  // both blocks' barriers exist before either is signalled
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  tc::wait_before();
  tc::let_next();

  constexpr int kUnit = kF8 ? kRowBytes : kRowBytes / 2;

  // Stages and their phases are counted up by hand: a 64-bit remainder a stage
  // kept the copies' and the products' threads behind the tensor cores.
  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t phase = 1;  // of the slot's last reading; a slot's first wait passes
      int64_t issued = 0;
      bool ok = true;
      const uint32_t bars_there = tc::map_rank(full(0), 0);
      Walk w = walk;
      for (Tile t; ok && w.next(t);) {
        const int32_t row_a = (int32_t)(t.ta * 2 * kTileM + (int32_t)rank * kTileM), row_b = (int32_t)(t.tb * kBN + rank * (kBN / 2));
        const CUtensorMap *ma = map_a, *mb = map_b;
        bool across_a = kMajA == kMajorMN;
        if (kMajA == kMajorByKind) {
          ma += t.kind;
          mb += t.kind;
          across_a = t.kind != 0;
        }
        for (int k = t.k0; k < t.k0 + t.kb; ++k, ++issued) {
          if (!(ok = tc::bar_wait(empty(s), phase, status))) break;
          if (rank == 0) tc::bar_expect(full(s), 2 * R::kStage);
          const uint32_t bar = bars_there + 8u * (uint32_t)s;
          const uint32_t sa = ring + (uint32_t)(s * R::kStage), sb = sa + R::kBytesA;
          if (!across_a) {
            tc::load_2d_pair(sa, ma, k * kUnit, row_a, bar);
          } else {
#pragma unroll
            for (int i = 0; i < kTileM / 64; ++i) tc::load_2d_pair(sa + i * 8192, ma, row_a + 64 * i, k * kUnit, bar);
          }
          if (kMajB == kMajorK) {
            tc::load_2d_pair(sb, mb, k * kUnit, row_b, bar);
          } else {
#pragma unroll
            for (int i = 0; i < kBN / 128; ++i) tc::load_2d_pair(sb + i * 8192, mb, row_b + 64 * i, k * kUnit, bar);
          }
          if (++s == R::kStages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // The first block, whose barriers count both blocks' copies, waits for
      // the last one into each stage; neither block leaves before that.
      if (rank == 0)
        for (int i = 0; i < R::kStages; ++i) {
          const int64_t m = (issued + R::kStages - 1 - i) / R::kStages;
          if (m > 0) tc::bar_wait(full(i), (uint32_t)((m - 1) & 1), status);
        }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      int s = 0, n = 0;
      uint32_t phase = 0;
      bool ok = true;
      Walk w = walk;
      // The operands' descriptors in stage 0; a stage, a block of 16 rows or a
      // slab further on their addresses (in units of 16 bytes) grow.
      const uint64_t da_along = tc::desc_128b(ring, 16, 1024), da_across = tc::desc_128b(ring, 8192, 1024);
      const uint64_t db0 = kMajB == kMajorK ? tc::desc_128b(ring + R::kBytesA, 16, 1024) : tc::desc_128b(ring + R::kBytesA, 8192, 1024);
      for (Tile t; ok && w.next(t); ++n) {
        const int b = n & 1;
        if (n >= 2 && !(ok = tc::bar_wait(acc_free(b), (uint32_t)(((n - 2) >> 1) & 1), status))) break;
        tc::fence_after();
        const uint32_t d = tmem + (uint32_t)(b * kBN);
        const bool across_a = kMajA == kMajorByKind ? t.kind != 0 : kMajA == kMajorMN;
        const uint64_t da0 = across_a ? da_across : da_along, step_a = across_a ? 128 : 2;
        const uint32_t id = idesc[kMajA == kMajorByKind ? t.kind : 0];
        for (int k = 0; k < t.kb; ++k) {
          if (!(ok = tc::bar_wait(full(s), phase, status))) break;
          tc::fence_after();
          const uint64_t at = (uint64_t)(uint32_t)(s * (R::kStage / 16));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc::mma_pair<kF8>(d, da0 + at + (uint64_t)j * step_a, db0 + at + (uint64_t)(j * (kMajB == kMajorK ? 2 : 128)), id,
                              (k > 0 || j > 0) ? 1u : 0u);
          tc::commit_pair(empty(s));
          if (++s == R::kStages) {
            s = 0;
            phase ^= 1;
          }
        }
        tc::commit_pair(acc_full(b));
      }
    }
  } else {
    const int q = warp & 3, quarter = (warp - 2) >> 2;
    const uint32_t boxes = ring + (uint32_t)(R::kStages * R::kStage + (warp - 2) * kBoxesEach * kStaging);
    int n = 0;
    Walk w = walk;
    for (Tile t; w.next(t); ++n) {
      const int b = n & 1;
      // a wait that runs out is flagged and gone on from, as the warps may meet
      // at barriers of their own
      tc::bar_wait_on(acc_full(b), (uint32_t)((n >> 1) & 1), status, &stalled);
      tc::fence_after();
      epi(w, t, q, quarter, tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * kBN), boxes, [&] {
        tc::fence_before();  // read out: the products may write it again
        __syncwarp();
        if (lane == 0) tc::arrive_remote(tc::map_rank(acc_free(b), 0));
      });
    }
    if (lane == 0) tc::store_wait_all();
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();  // no block leaves while the other signals it or reads its operands
  if (warp == 1) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
  }
}

// ---------------------------------------------------------------- host side
// Launches a kernel that may start while the one before it in the stream ends:
// it sets itself up and waits for that one's end (tc::wait_before) before it
// touches its data.  The kernel before must be one of the same call.
template <typename... P, typename... A>
cudaError_t launch_beside(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s, bool beside, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = beside ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    cudaGetLastError();
  });
  return fn;
}

// A map of m (rows on 16-byte boundaries) for boxes of `inner` values x
// `outer` rows in the 128-byte swizzle; parts outside the matrix read as 0.
inline cudaError_t encode(CUtensorMap *map, const ss_dense &m, int inner, int outer) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = map_encoder();
  if (!fn) return cudaErrorNotSupported;
  const int64_t size = size_of(m.type);
  const cuuint64_t dims[2] = {(cuuint64_t)m.n_cols, (cuuint64_t)m.n_rows};
  // one row: its stride is never used, and any ld is allowed for it
  const cuuint64_t strides[1] = {(cuuint64_t)(m.n_rows > 1 ? m.ld * size : (m.n_cols * size + 15) / 16 * 16)};
  const cuuint32_t box[2] = {(cuuint32_t)inner, (cuuint32_t)outer}, elem[2] = {1, 1};
  return fn(map, size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, m.data, dims, strides,
            box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

inline int64_t padded_ld(const ss_dense &m) { return (m.n_cols + 15) / 16 * 16; }
inline int64_t align_up(int64_t b) { return (b + SS_SCRATCH_ALIGN - 1) / SS_SCRATCH_ALIGN * SS_SCRATCH_ALIGN; }
inline int64_t copy_bytes(const ss_dense &m) {
  return rows_aligned(m, 16) ? 0 : align_up(m.n_rows * padded_ld(m) * size_of(m.type));
}
// A map of an output for boxes of 64 bytes x 32 rows.
inline cudaError_t encode_out(CUtensorMap *map, const ss_dense &m) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = map_encoder();
  if (!fn) return cudaErrorNotSupported;
  const int64_t size = size_of(m.type);
  const cuuint64_t dims[2] = {(cuuint64_t)m.n_cols, (cuuint64_t)m.n_rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(m.n_rows > 1 ? m.ld * size : (m.n_cols * size + 15) / 16 * 16)};
  const cuuint32_t box[2] = {(cuuint32_t)(64 / size), 32}, elem[2] = {1, 1};
  return fn(map, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, m.data, dims, strides,
            box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

inline uint32_t idesc_of(const ss_dense &A, int majA, int majB, int m, int n) {
  const uint32_t type = A.type == SS_VALUES_BF16 ? 1 : 0;  // fp16 and e4m3: 0
  return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)majA << 15) | ((uint32_t)majB << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

}  // namespace dense
