// Tensor-core (tcgen05), asynchronous copy and mbarrier instructions of the
// dense operators.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "dense.cuh"

namespace tc {

constexpr long long kWaitNs = 2000000000ll;  // bounded waits: 2 s

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ long long global_ns() {
  long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// ---------------------------------------------------------------- barriers
__device__ __forceinline__ void bar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase of `parity` to complete, for at most kWaitNs; false
// (and a DEV_STALL flag) when it runs out.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, int32_t *status) {
  if (bar_try(bar, parity)) return true;
  const long long t0 = global_ns();
  for (;;) {
    for (int i = 0; i < 64; ++i)
      if (bar_try(bar, parity)) return true;
    if (global_ns() - t0 > kWaitNs) {
      dense::flag(status, DEV_STALL);
      return false;
    }
  }
}
// The same for code that must not leave its path when a wait runs out (the
// block's other barriers count on every thread): after kWaitNs it flags
// DEV_STALL and sets *stalled, to the time then in units of 2^20 ns (made odd,
// so not 0).  From then on it and the block's other waits go on for another
// kWaitNs together, so that copies under way land before the block leaves, and
// return whether their phases complete or not: whether they did.
__host__ __device__ constexpr int stall_time(long long ns) { return (int)(unsigned)(ns >> 20) | 1; }
__host__ __device__ constexpr bool stall_over(int stalled, long long ns) {
  return (int)((unsigned)(ns >> 20) - (unsigned)stalled) > (int)(kWaitNs >> 20);
}
static_assert(stall_time(0) != 0 && !stall_over(stall_time(5ll << 32), 5ll << 32) &&
                  !stall_over(stall_time(5ll << 32), (5ll << 32) + kWaitNs) &&
                  stall_over(stall_time(5ll << 32), (5ll << 32) + kWaitNs + (3ll << 20)) &&
                  !stall_over(stall_time((1ll << 52) - 1), (1ll << 52) + kWaitNs - (3ll << 20)) &&
                  stall_over(stall_time((1ll << 52) - 1), (1ll << 52) + kWaitNs + (3ll << 20)),
              "a second limit of kWaitNs from the stall on");
__device__ __forceinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, int32_t *status, volatile int *stalled) {
  const long long t0 = global_ns();
  for (;;) {
    for (int i = 0; i < 64; ++i)
      if (bar_try(bar, parity)) return true;
    const long long now = global_ns();
    if (const int s = *stalled) {
      if (stall_over(s, now)) return false;
    } else if (now - t0 > kWaitNs) {
      dense::flag(status, DEV_STALL);
      *stalled = stall_time(now);
    }
  }
}
__device__ __forceinline__ bool bar_wait_on(uint32_t bar, uint32_t parity, int32_t *status, volatile int *stalled) {
  return bar_try(bar, parity) || bar_wait_long(bar, parity, status, stalled);
}
// The same with the long wait out of line, for a kernel of many waits.
static __device__ __noinline__ bool bar_wait_apart(uint32_t bar, uint32_t parity, int32_t *status, volatile int *stalled) {
  return bar_wait_long(bar, parity, status, stalled);
}
__device__ __forceinline__ bool bar_wait_far(uint32_t bar, uint32_t parity, int32_t *status, volatile int *stalled) {
  return bar_try(bar, parity) || bar_wait_apart(bar, parity, status, stalled);
}
// The barrier `id` (1 to 15) of `threads` threads of the block.
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// ---------------------------------------------------------------- copies
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Plain bytes: both addresses 16-byte aligned, a multiple of 16 of them.
__device__ __forceinline__ void load_bulk(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// kBytes (4, 8 or 16) from one thread, both addresses aligned to them.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(kBytes) : "memory");
}
// A value of 2, 4 or 16 bytes at a shared address aligned to its size.
template <typename P>
__device__ __forceinline__ P read_shared(uint32_t at) {
  P v;
  if constexpr (sizeof(P) == 16) {
    uint4 q;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at) : "memory");
    memcpy(&v, &q, 16);
  } else if constexpr (sizeof(P) == 4) {
    uint32_t q;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(q) : "r"(at) : "memory");
    memcpy(&v, &q, 4);
  } else {
    static_assert(sizeof(P) == 2, "16, 4 or 2 bytes");
    uint16_t q;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(q) : "r"(at) : "memory");
    memcpy(&v, &q, 2);
  }
  return v;
}
// Writes a value of 2 or 4 bytes.
template <typename P>
__device__ __forceinline__ void write_shared(uint32_t at, P v) {
  if constexpr (sizeof(P) == 4) {
    uint32_t q;
    memcpy(&q, &v, 4);
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(q) : "memory");
  } else {
    static_assert(sizeof(P) == 2, "4 or 2 bytes");
    uint16_t q;
    memcpy(&q, &v, 2);
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(q) : "memory");
  }
}
// A box into this block's shared memory, counted on barrier `bar` (a
// cluster address) of either block of the pair.
__device__ __forceinline__ void load_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Shared memory to the box at (x, y), in this thread's bulk group; parts
// outside the matrix are not written.
__device__ __forceinline__ void store_2d(const CUtensorMap *map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map), "r"(src),
               "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Until all of this thread's store groups have read their source.
__device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// This thread's shared-memory writes before its later asynchronous copies.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---------------------------------------------------------------- tcgen05
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// Descriptor of an operand in the 128-byte swizzle at `addr` (its 8-row,
// 1024-byte pattern starts on a 1024-byte boundary).  K-major: rows of 128
// bytes, sbo = bytes between groups of 8 rows.  MN-major: lbo = bytes between
// slabs of 64 rows, sbo = bytes between groups of 8 K.
__device__ __forceinline__ uint64_t desc_128b(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// D[tmem] (+)= A B^T; kF8: e4m3 inputs, else the 16-bit type in idesc.
template <bool kF8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kF8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(accumulate));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(accumulate));
}
// The same over a pair of blocks: 256 rows of A, half of them and half of B's
// rows in each block's shared memory, each block's rows in its tensor memory.
template <bool kF8>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kF8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(accumulate));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(accumulate));
}
// Arrives on `bar` in both blocks of the pair once this thread's products so
// far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// 32 consecutive fp32 columns of this thread's tensor-memory lane, without the wait.
__device__ __forceinline__ void load_acc32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void load_acc_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// 16 consecutive fp32 columns of this thread's tensor-memory lane.
__device__ __forceinline__ void load_acc16(uint32_t addr, float (&f)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(r[i]);
}

// 32 columns of 16 tensor-memory lanes, without the wait: of columns 8 i + 2 (t % 4)
// and the next, thread t has those of lane t / 4 in r[4 i], r[4 i + 1] and those of
// lane t / 4 + 8 in r[4 i + 2], r[4 i + 3].
__device__ __forceinline__ void load_acc16x32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
// Four matrices of 8 x 8 16-bit values: thread t holds values (t / 4, 2 (t % 4))
// and the next of each, and the shared address of row t % 8 of matrix t / 8.
__device__ __forceinline__ void store_matrices(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// For kernels launched beside the end of the one before (launch_beside): until
// that one is done, and leave for the next one to be launched.
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Asks for the work of a cluster of this grid that has not started: the 16-byte
// answer goes to shared address `at` of every block of this cluster and counts
// on the barrier at `bar` there.
__device__ __forceinline__ void ask_for_cluster(uint32_t at, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 [%0], [%1];" ::"r"(at),
      "r"(bar)
      : "memory");
}
// The first block's x of the cluster that an answer gives, or -1: none left.
__device__ __forceinline__ int64_t cluster_given(uint32_t at) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.b32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n\t}\n"
      : "=r"(ok), "=r"(x)
      : "r"(at)
      : "memory");
  return ok ? (int64_t)x : -1;
}
// The address in the cluster of shared address `addr` of block `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
// Arrives on a barrier given by its address in the cluster.
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Two floats to shared memory of a block of the cluster, counted as 8 bytes on
// barrier `bar` there (both cluster addresses).  Unlike an arrival that
// releases to the cluster it does not wait for this thread's earlier stores.
__device__ __forceinline__ void send_remote(uint32_t at, float x, float y, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at), "f"(x), "f"(y), "r"(bar)
               : "memory");
}
// The float at shared address `addr` of block `rank` of the cluster.
__device__ __forceinline__ float load_remote(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(map_rank(addr, rank)) : "memory");
  return v;
}

}  // namespace tc
