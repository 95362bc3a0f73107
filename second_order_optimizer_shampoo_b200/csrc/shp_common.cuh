// Device helpers shared by the sm_100a kernels: mbarriers with bounded waits,
// TMA bulk-tensor loads, tcgen05 (TMEM allocation, MMA, commit, loads) and
// the shared-memory matrix descriptors of the 5th-generation tensor cores.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#define SHP_DEV __device__ __forceinline__

// Upper bound for every spin-wait, in SM clock cycles (~1 s at 2 GHz).  A wait
// that runs out records SHP_ETIMEOUT and lets the kernel unwind; nothing spins
// unbounded.
#ifndef SHP_SPIN_LIMIT
#define SHP_SPIN_LIMIT (2000000000LL)
#endif

namespace shp {

// Kernels this translation unit has run on the current device: the first
// thread of the first CTA of every kernel adds one (before any early exit).
static __device__ unsigned long long g_kernel_runs;
SHP_DEV void count_kernel_run() {
  if ((threadIdx.x | threadIdx.y | threadIdx.z | blockIdx.x | blockIdx.y | blockIdx.z) == 0)
    atomicAdd(&g_kernel_runs, 1ull);
}

SHP_DEV uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ----------------------------------------------------------------- mbarrier
SHP_DEV void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}
SHP_DEV void fence_barrier_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
SHP_DEV void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
SHP_DEV uint32_t mbar_try_wait(uint32_t addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(addr), "r"(parity)
      : "memory");
  return ok;
}
// Bounded wait on phase `parity`; returns false if `limit` cycles ran out or,
// when `abort` is given, once another role of the CTA has set it (so that a
// CTA whose wait gave up unwinds without every other waiter spinning to its
// own limit).
SHP_DEV bool mbar_wait(uint64_t* bar, uint32_t parity, const volatile int* abort = nullptr,
                       long long limit = SHP_SPIN_LIMIT) {
  const uint32_t addr = smem_u32(bar);
  if (mbar_try_wait(addr, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(addr, parity)) {
    if (clock64() - t0 > limit) return false;
    if (abort != nullptr && *abort) return false;
  }
  return true;
}

// A position in a ring of N stages: the slot and the parity of its current use.
// A producer waits with parity ^ 1, which a fresh barrier passes at once.
// Counting instead of dividing a running index by N keeps the one-thread issue
// loops short: their instructions, not the copies, set a ring's rate.
template <int N>
struct RingPos {
  uint32_t slot = 0, parity = 0;
  SHP_DEV void advance() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// try_wait that may suspend the thread for up to about 16 us: a polling warp
// takes issue slots and shared-memory cycles from the issuing threads beside it.
SHP_DEV uint32_t mbar_try_wait_long(uint32_t addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(addr), "r"(parity), "r"(16384u)
      : "memory");
  return ok;
}

// What the bounded waits of a CTA share, in shared memory.  `limit` is for a wait
// that ends with one step of a pipeline (a ring's stage, a chunk of an
// accumulator), however long the launch; `tile_limit` for one that spans whole
// tiles (the next tile's description, a stage that comes late in a tile), whose
// length follows the work: TILE_PATIENCE clocks more for each stage of the
// longest tile, hundreds of times what one takes (two tiles may pass during such
// a wait), so that no accepted size runs into it.
struct WaitState {
  int abort;  // set by the wait that gave up; the others then give up too (but see below)
  long long limit, tile_limit;
};
constexpr long long TILE_PATIENCE = 1 << 18;

// By one thread, before the block's first barrier.  `limit` 0: the usual one.
SHP_DEV void wait_state_init(volatile WaitState* ws, long long limit, int64_t tile_stages) {
  ws->abort = 0;
  ws->limit = limit > 0 ? limit : SHP_SPIN_LIMIT;
  ws->tile_limit = (limit > 0 ? limit : SHP_SPIN_LIMIT) + tile_stages * TILE_PATIENCE;
}

// Bounded wait by shared address; the abort flag is looked at only when the
// phase is not complete yet, and set on giving up.
SHP_DEV bool ring_wait(uint32_t bar, uint32_t parity, volatile WaitState* ws, bool tile = false) {
  if (mbar_try_wait_long(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait_long(bar, parity)) {
    if (ws->abort || clock64() - t0 > (tile ? ws->tile_limit : ws->limit)) {
      ws->abort = 1;
      return false;
    }
  }
  return true;
}
// The producers' form.  What a pair's producers load is counted on the leader's
// barriers, so both have to stop at the same stage, or the leader cannot tell when
// the last copy has landed.  They are woken by the same commits and the same tile
// descriptions, which end within microseconds of an abort; so a producer goes on
// for `limit` clocks after it has seen the flag, and stops when nothing has come.
SHP_DEV bool producer_wait(uint32_t bar, uint32_t parity, volatile WaitState* ws, bool tile) {
  if (mbar_try_wait_long(bar, parity)) return true;
  const long long t0 = clock64();
  long long seen = -1;
  while (!mbar_try_wait_long(bar, parity)) {
    const long long t = clock64();
    if (seen < 0 && ws->abort) seen = t;
    if ((seen >= 0 && t - seen > ws->limit) || t - t0 > (tile ? ws->tile_limit : ws->limit)) {
      ws->abort = 1;
      return false;
    }
  }
  return true;
}
// A whole warp waits; false for every lane if one lane's wait gave up, so that
// the warp leaves its loop together.
SHP_DEV bool warp_wait(uint32_t bar, uint32_t parity, volatile WaitState* ws, bool tile = false) {
  return __all_sync(0xffffffffu, ring_wait(bar, parity, ws, tile));
}

// The same wait for the loops that issue copies or MMAs, with every branch on a
// vote, so that the compiler can see that the warp stays together (see
// warp-uniform issue below).  Measured: a stage of the 4-bit product (10
// instructions, 128-column tiles) 290 -> 203 ns; 1 row over 8 groups, 4096 x 4096
// 15.6 -> 14.4 us.  In the scheduler warp the same form costs (14.4 -> 20 us).
// PRODUCER: for a stage of the ring, as producer_wait.
template <bool PRODUCER = false>
SHP_DEV bool issue_wait(uint32_t bar, uint32_t parity, volatile WaitState* ws) {
  if (__all_sync(0xffffffffu, mbar_try_wait_long(bar, parity))) return true;
  const long long t0 = clock64();
  while (!__all_sync(0xffffffffu, mbar_try_wait_long(bar, parity))) {
    if (__any_sync(0xffffffffu, (!PRODUCER && ws->abort) || clock64() - t0 > ws->limit)) {
      ws->abort = 1;
      return false;
    }
  }
  return true;
}

// One look at a barrier, by a whole warp: an issuing warp asks for its next stage
// while it still issues this one, which hides the answer's latency.
SHP_DEV bool warp_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, ok);
}

// Behind a wait on a phase that is complete: acquires what the other CTA of the
// pair released (or stored by st.async) with it.
SHP_DEV bool acquire_cluster(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// warp_wait that does so.
SHP_DEV bool warp_wait_cluster(uint32_t bar, uint32_t parity, volatile WaitState* ws,
                               bool tile = false) {
  return __all_sync(0xffffffffu,
                    ring_wait(bar, parity, ws, tile) && acquire_cluster(bar, parity));
}

// Limit of the wait a bounded-wait self-test points at a barrier nothing
// completes (about 10 ms): long enough to be a real wait, short for a test.
// (The grouped and 4-bit kernels' take SelfTest::stall clocks.)
#define SHP_SELFTEST_LIMIT (20000000LL)

// Bounded-wait self-test of a kernel: waits `stall` clocks (0: no test) on a
// barrier that nothing completes and raises the block's abort flag.  True if it did.
SHP_DEV bool selftest_wait(int stall, uint64_t* never, volatile int* abort_flag) {
  if (stall == 0 || mbar_wait(never, 0, nullptr, stall)) return false;
  *abort_flag = 1;
  return true;
}
// Its end: a block whose abort flag is up records the timeout (status null:
// an ordinary launch, which has none).
SHP_DEV void selftest_report(int* status, volatile const int* abort_flag) {
  if (status != nullptr && threadIdx.x == 0 && *abort_flag) atomicExch(status, 19);  // SHP_ETIMEOUT
}

SHP_DEV void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// ----------------------------------------------------------------- TMA
SHP_DEV void tma_prefetch_desc(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// 3-D tiled bulk-tensor load global -> shared, completion counted on `bar`.
// Coordinates are element indices {x (innermost), y, z}; x is always a
// multiple of 32 elements here, so x * element size is 16-byte aligned.
SHP_DEV void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Byte offset of 16-byte group g of row r in a box of 128-byte rows stored
// with the 128-byte swizzle.
SHP_DEV uint32_t sw128_off(int r, int g) {
  return static_cast<uint32_t>(r * 128 + ((g ^ (r & 7)) << 4));
}

// 3-D tiled bulk-tensor store shared -> global of the box at {x, y, z}, in
// this thread's bulk group; the tensor map clips rows and columns outside
// the tensor.  x * element size must be a multiple of 16 bytes.
SHP_DEV void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
SHP_DEV void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// This thread's committed bulk stores have finished reading shared memory.
SHP_DEV void bulk_wait_read_all() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
// This thread's committed bulk stores are complete.
SHP_DEV void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Orders this thread's generic-proxy shared-memory accesses before later
// async-proxy (TMA) accesses to them.
SHP_DEV void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ----------------------------------------------------------------- tcgen05
SHP_DEV void tmem_alloc(uint32_t* dst_smem, uint32_t ncols) {  // whole warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst_smem)),
               "r"(ncols));
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
SHP_DEV void tmem_dealloc(uint32_t taddr, uint32_t ncols) {  // whole warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols));
}
SHP_DEV void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
SHP_DEV void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D(tmem) (+)= A(smem) * B(smem), issued by one thread.
SHP_DEV void mma_tf32(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                      uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::tf32 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
SHP_DEV void mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                     uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
// Arrive once on `bar` when every MMA issued so far by this thread completes.
SHP_DEV void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}
// 32 lanes x 32 consecutive 32-bit columns: thread t gets lane (base + t).  Load and
// wait are one statement, so that nothing that uses the registers can move between.
SHP_DEV void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// The same for 64 columns, as bits.
SHP_DEV void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]),
        "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]),
        "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
        "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]),
        "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}

// ----------------------------------------------------------------- CTA pairs
// A cluster of two CTAs on two SMs runs one tcgen05 MMA of M = 256: each CTA
// holds 128 rows of A and half of B; the even CTA (rank 0) issues the MMAs.
SHP_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// All threads of both CTAs; the two CTAs of a cluster are co-scheduled.
SHP_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}
// shared::cluster address of the same shared variable in CTA `rank`.
SHP_DEV uint32_t mapa_shared(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// TMA load into this CTA's shared memory whose completion is counted on an
// mbarrier that may live in the peer CTA (`mbar` is a shared::cluster address).
SHP_DEV void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t mbar, int x, int y,
                              int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
SHP_DEV void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {  // one warp in each CTA
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst_smem)),
               "r"(ncols));
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
SHP_DEV void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols));
}
SHP_DEV void mma_tf32_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::tf32 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
SHP_DEV void mma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
// Arrive on an mbarrier given by its shared::cluster address (may be the peer's).
SHP_DEV void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
// Arrival on an mbarrier of either CTA that hands back tensor memory or a tile
// slot: the reads before it are complete (tcgen05.wait::ld and a tcgen05 fence, or
// shuffles of the values), and no memory write has to become visible with it, so it
// need not wait for this thread's outstanding stores as a releasing arrival does.
SHP_DEV void mbar_arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
// Arrive once on the mbarrier at this offset in every CTA of `mask` when the
// pair's MMAs issued so far complete.
SHP_DEV void mma_commit_pair(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(mask)
      : "memory");
}

// ----------------------------------------------------- warp-uniform issue
// The copy and MMA instructions take their operands from uniform registers.
// Inside an `if (lane == 0)` block the compiler keeps everything in per-thread
// registers and moves each operand across before each instruction: 70 to 90
// clocks per instruction, measured, which bounds kernels whose stages need
// many.  So an issuing warp runs its loop as a whole on warp-uniform values,
// and one elected lane (`on`) executes the instruction under a predicate.
SHP_DEV uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}
// A value every lane holds, as one the compiler knows to be warp-uniform.
SHP_DEV int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
SHP_DEV uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

SHP_DEV void mbar_expect_tx_if(uint32_t on, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%1], %2;\n\t}" ::"r"(on),
      "r"(bar), "r"(bytes)
      : "memory");
}
SHP_DEV void tma_3d_if(uint32_t on, uint32_t dst, const CUtensorMap* map, uint32_t mbar, int x,
                       int y, int z) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%1], [%2, {%4, %5, %6}], [%3];\n\t}" ::"r"(on),
      "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
SHP_DEV void tma_4d_if(uint32_t on, uint32_t dst, const CUtensorMap* map, uint32_t mbar, int x,
                       int y, int z, int w) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
      "@q cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%1], [%2, {%4, %5, %6, %7}], [%3];\n\t}" ::"r"(on),
      "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
SHP_DEV void tma_3d_pair_if(uint32_t on, uint32_t dst, const CUtensorMap* map, uint32_t mbar,
                            int x, int y, int z) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%1], [%2, {%4, %5, %6}], [%3];\n\t}" ::"r"(on),
      "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
SHP_DEV void tma_4d_pair_if(uint32_t on, uint32_t dst, const CUtensorMap* map, uint32_t mbar,
                            int x, int y, int z, int w) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
      "@q cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%1], [%2, {%4, %5, %6, %7}], [%3];\n\t}" ::"r"(on),
      "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
SHP_DEV void mma_f16_pair_if(uint32_t on, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %0, 0;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%1], %2, %3, %4, p;\n\t}" ::"r"(on),
      "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
SHP_DEV void mma_commit_pair_if(uint32_t on, uint32_t bar, uint16_t mask) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%1], %2;\n\t}" ::"r"(on),
      "r"(bar), "h"(mask)
      : "memory");
}

// ------------------------------------------------- dynamic tile scheduling
// A scheduler warp of a pair's leader CTA finds the pair's next tile and passes
// its description (eight integers, the first >= 0) to the roles of both CTAs
// through two slots, so that looking a tile up runs ahead of the work.
//
// Where tiles are handed out, the grid has one cluster (CTA pair) per tile, of
// which only those that fit run: a running pair that wants another tile cancels
// the launch of a waiting one and does that one's work (cluster launch
// control).  The hardware hands tiles out as pairs become free, with no counter
// in memory to clear or to share between launches.
struct TileSlots {
  uint64_t full[2];   // per CTA: the slot holds a tile (or -1: no more)
  uint64_t empty[2];  // leader: every consumer of both CTAs has read it
  uint64_t asked;     // leader: the answer has arrived
  alignas(16) uint4 answer;
  alignas(16) int tile[2][8];
};

// Asks for another cluster; 16 bytes arrive in `answer`, counted on `bar`.
SHP_DEV void try_cancel_cluster(uint32_t answer, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
      " [%0], [%1];" ::"r"(answer),
      "r"(bar)
      : "memory");
}
// First CTA index (x) of the cancelled cluster, or -1 if none was left.
SHP_DEV int cancelled_cta(uint32_t answer) {
  int x = -1;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t.reg .b32 y, z;\n\t"
      "ld.shared.b128 a, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, _}, a;\n\t}"
      : "+r"(x)
      : "r"(answer)
      : "memory");
  return x;
}
// Stores a tile in a CTA's slot (cluster address), 32 bytes counted on its
// barrier, on which this thread also arrives.
SHP_DEV void slot_store(uint32_t addr, const int (&v)[8], uint32_t bar) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], 32;" ::"r"(bar)
               : "memory");
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
            addr + 16u * i),
        "r"(v[4 * i]), "r"(v[4 * i + 1]), "r"(v[4 * i + 2]), "r"(v[4 * i + 3]), "r"(bar)
        : "memory");
}

SHP_DEV void tile_slots_init(TileSlots* ts, int consumers) {
  for (int i = 0; i < 2; ++i) {
    mbar_init(&ts->full[i], 1);
    mbar_init(&ts->empty[i], consumers);
  }
  mbar_init(&ts->asked, 1);
}

// The scheduler, a whole warp of the leader.  Tiles come from the launch's
// waiting clusters (handed_out) or are every `step`-th from `t`.  find(t, v)
// describes tile t, or is false if there is no such tile: then none follows it
// in turn, and of those handed out (a grid sized by an upper bound) it is
// dropped.  Every wait is bounded; the answer to a question is waited for without a
// look at the abort flag, as it is written into this CTA's shared memory.
template <class Find>
SHP_DEV void schedule_tiles(TileSlots* ts, bool handed_out, int t, int step, Find find,
                            volatile WaitState* ws) {
  const int lane = threadIdx.x & 31;
  RingPos<2> at;
  uint32_t asked = 0;
  for (;;) {
    if (!warp_wait_cluster(smem_u32(&ts->empty[at.slot]), at.parity ^ 1u, ws, true)) return;
    int v[8] = {-1, 0, 0, 0, 0, 0, 0, 0};
    if (handed_out) {
      do {
        if (lane == 0) {
          mbar_arrive_expect_tx(&ts->asked, 16);
          try_cancel_cluster(smem_u32(&ts->answer), smem_u32(&ts->asked));
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&ts->asked, asked, nullptr, ws->limit))) return;
        asked ^= 1u;
        t = cancelled_cta(smem_u32(&ts->answer));
        fence_proxy_async_smem();  // read before the next answer is written
        t = uniform(t);
        __syncwarp();
      } while (t >= 0 && !find(t / 2, v));
    } else {
      t += step;
      if (!find(t, v)) t = -1;
    }
    if (t < 0) v[0] = -1;
    if (lane < 2)
      slot_store(mapa_shared(smem_u32(ts->tile[at.slot]), lane), v,
                 mapa_shared(smem_u32(&ts->full[at.slot]), lane));
    if (t < 0) return;
    at.advance();
  }
}

// A consumer warp's view: next() gives the following tile's description to every
// lane, v[0] = -1 when there is none left (or a wait gave up).
struct TileFeed {
  TileSlots* ts;
  volatile WaitState* ws;
  RingPos<2> at;
  template <bool PRODUCER>
  SHP_DEV void next(int (&v)[8]) {
    v[0] = -1;
    const uint32_t bar = smem_u32(&ts->full[at.slot]);
    const bool ok = PRODUCER ? producer_wait(bar, at.parity, ws, true)
                             : ring_wait(bar, at.parity, ws, true);
    if (!__all_sync(0xffffffffu, ok && acquire_cluster(bar, at.parity))) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = uniform(const_cast<volatile int*>(ts->tile[at.slot])[i]);
    // The shuffles have consumed what every lane read, so the slot may be written
    // again; a releasing arrival would wait for the epilogue warps' stores besides
    // (8192 rows over 64 blocks 99 -> 109 us, 64 gradients of 1024^2 72 -> 83).
    if ((threadIdx.x & 31) == 0)
      mbar_arrive_relaxed(mapa_shared(smem_u32(&ts->empty[at.slot]), 0));
    at.advance();
  }
};

// Shared-memory matrix descriptor (sm_100 layout version 1).
//   start address, leading-dimension byte offset and stride-dimension byte
//   offset are stored >> 4; `layout` is the swizzle mode:
//     2 = 128-byte swizzle of 16-byte chunks (period 8 rows of 128 B),
//     1 = 128-byte swizzle of 32-byte chunks (period 4 rows of 128 B), the
//         only MN-major layout the tensor cores accept for 32-bit operands.
//   K-major operand: the leading offset is unused (16) and the stride offset
//   is the distance between 8-row core groups (1024 B).
//   MN-major operand: the leading offset is the distance between 128-byte MN
//   chunks and the stride offset the distance between K groups of one swizzle
//   period (8 rows = 1024 B for layout 2, 4 rows = 512 B for layout 1).
SHP_DEV uint64_t smem_desc(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes,
                           uint32_t layout) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo_bytes >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((sbo_bytes >> 4) & 0x3FFFu) << 32;
  d |= 1ull << 46;  // descriptor version for sm_100
  d |= static_cast<uint64_t>(layout & 7u) << 61;
  return d;
}

// Instruction descriptor for kind::tf32 / kind::f16 with fp32 accumulation.
//   fmt: 1 = BF16, 2 = TF32 (both operands the same type).
__host__ __device__ constexpr uint32_t instr_desc(uint32_t fmt, bool a_mn, bool b_mn, int M,
                                                  int N) {
  return (1u << 4)                              // D format fp32
         | (fmt << 7) | (fmt << 10)             // A, B formats
         | (static_cast<uint32_t>(a_mn) << 15)  // A major: 0 K, 1 MN
         | (static_cast<uint32_t>(b_mn) << 16)  // B major
         | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Round to the nearest TF32 value (ties away from zero), kept in fp32 format.
SHP_DEV float tf32_round(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return __uint_as_float(r);
}

SHP_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
SHP_DEV double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace shp
