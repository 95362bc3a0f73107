// Products of rows grouped by expert (weight block) on the sm_100a tensor
// cores: the forward product of an expert layer, the gradient of its input
// and the gradient of its weight blocks, which the Shampoo statistics take.
//
//   rows      Y[t]  = X[t] W_e  (or X[t] W_e^T),  t in [off_e, off_{e+1})
//   wgrad     G_e   = A_e^T B_e (+ G_e),  A_e, B_e the rows [off_e, off_{e+1})
//
// bf16 operands, fp32 accumulation.  The group boundaries are read on the
// device, so nothing waits for the host.  Both kernels are persistent CTA-pair
// kernels (one tcgen05 MMA of M = 256 over two SMs, tiles up to 256 x 256, TMA
// ring, two TMEM accumulators so that the epilogue of one tile runs beside the
// main loop of the next), like the batched product of gemm_tc.cu; what differs
// is where tiles come from (a scheduler warp that scans the offsets), the ragged
// edges, and the fp32 sums:
//   - row tiles start at any row; rows of the next group that a tile's box
//     also holds are multiplied but not stored (a row of Y depends on its own
//     row of X alone);
//   - wgrad contracts over rows, where a neighbour's rows would enter the
//     sum: the last, partial stage of a group is landed on a barrier of its
//     own, one warp clears the rows behind the group in shared memory (both
//     operands, so that 0 * Inf cannot arise), and only then is the stage
//     handed to the MMA, which issues just the 16-row steps it needs;
//   - the tensor cores add into their accumulator with truncation, a bias of
//     about half an ulp per MMA that grows with the length of the sum, so
//     fp32 results are summed in chunks of CHUNK_KB stages: each chunk is
//     read out of TMEM and added to running sums in registers, rounded to
//     nearest, while the next chunk's MMAs run.  bf16 results take chunks of
//     LONG_KB stages: 256 MMAs' bias, at most 2^-16 of a sum of one sign, moves
//     one bf16 result in 500 to its neighbour, and a longer contraction's is no
//     larger.  Up to that length a chunk is the whole sum and is stored as it
//     leaves the accumulator (chunks of CHUNK_KB for bf16 too: 65536 rows over
//     16 groups, 4096 x 1024, 405 us against 372, and 1024 x 4096 466 against
//     381; the error against the exact product is its rounding's, 1.7e-3 of the
//     norm, either way).
#include <cuda_bf16.h>
#include <string.h>

#include "internal.h"
#include "shp_common.cuh"

namespace shp {

namespace {

constexpr int BK = 64;                // contraction elements per stage: 128-byte rows
constexpr int A_BYTES = 128 * 128;    // per CTA and stage: 128 rows (columns) of A
constexpr int CHUNK_KB = 8;  // stages per fp32 chunk: sums of 512 products inside the tensor core
constexpr int LONG_KB = 64;  // stages per chunk of a bf16 result: sums of 4096 products
constexpr int EPI_WARPS = 8;
constexpr int EPI_BOX = 4096;  // one warp's 32 x 32 fp32 store box

SHP_DEV void tma_reduce_add_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group"
      " [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Group e covers the rows [lo, hi): the offsets clamped to 0..T and to
// non-negative lengths, so that no offset array reaches outside the operands.
struct Groups {
  const int64_t* off;
  int n;
  int T;
  SHP_DEV void range(int e, int& lo, int& hi) const {
    int64_t a = __ldg(off + e), b = __ldg(off + e + 1);
    a = a < 0 ? 0 : (a > T ? T : a);
    b = b < a ? a : (b > T ? T : b);
    lo = static_cast<int>(a);
    hi = static_cast<int>(b);
  }
};

// A tile of the rows product: `count` rows from row t0 in group e, weight
// columns from n0.
struct RowTile {
  int e, t0, count, n0;
};

// Looks row tiles up by number.  Tiles are numbered over the groups in order; a
// group of len rows has ceil(len / NT) row tiles of equal size (up to the MMA's
// granule of 16), each with every column tile.  find() is called by whole warps
// and looks at 32 groups per step.
template <int NT>
struct RowTiles {
  const Groups g;
  const int tiles_n;
  int e0 = 0;    // first group of the window
  int base = 0;  // tiles before the window
  SHP_DEV RowTiles(const Groups& groups, int N) : g(groups), tiles_n((N + 255) / 256) {}
  SHP_DEV bool find(int t, RowTile& x) {
    if (t < base) e0 = base = 0;
    const int lane = threadIdx.x & 31;
    while (e0 < g.n) {
      int a = 0, b = 0;
      if (e0 + lane < g.n) g.range(e0 + lane, a, b);
      const int cnt = (b - a + NT - 1) / NT * tiles_n;
      int inc = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const unsigned in = __ballot_sync(0xffffffffu, t < base + inc);
      if (in != 0) {
        const int src = __ffs(in) - 1;
        const int r = t - base - __shfl_sync(0xffffffffu, inc - cnt, src);
        const int lo = __shfl_sync(0xffffffffu, a, src), hi = __shfl_sync(0xffffffffu, b, src);
        const int tiles = (hi - lo + NT - 1) / NT;
        const int per = ((hi - lo + tiles - 1) / tiles + 15) & ~15;  // <= NT
        x.e = uniform(e0 + src);
        x.t0 = uniform(lo + r / tiles_n * per);
        x.count = uniform(min(per, hi - x.t0));
        x.n0 = uniform(r % tiles_n * 256);
        return true;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
      e0 += 32;
    }
    return false;  // a number beyond the last tile
  }
};

// A role's walk over its pair's tiles: its own, which every role looks up while
// the block sets up, then the scheduler's.
struct RowWalk {
  TileFeed feed;
  RowTile own;
  bool have, first = true;
  SHP_DEV RowWalk(TileSlots* ts, volatile WaitState* ws) : feed{ts, ws}, have(false) {}
  template <bool PRODUCER = false>
  SHP_DEV bool next(RowTile& x) {
    if (first) {
      first = false;
      x = own;
      return have;
    }
    int v[8];
    feed.next<PRODUCER>(v);
    x.e = v[0];
    x.t0 = v[1];
    x.count = v[2];
    x.n0 = v[3];
    return x.e >= 0;
  }
};

// ---------------------------------------------------------- rows product
//
// k_grouped_rows computes the transposed tile, D (columns of W x rows of X):
// the 256 columns of W are the MMA's M (128 per CTA of the pair) and the rows
// of the group its N, any multiple of 16 up to NT.  So the time of the MMAs
// follows the rows a group has, and few rows cost little more than streaming
// W; with the rows as M = 256 a single row cost as much as 256.
// NT (64, 128 or 256 rows; rows_per_tile()) is a tile's height: a stage is 16 KB
// of W and up to NT * 64 bytes of X per CTA.
// Epilogue: a lane holds one column of Y.  bf16: lanes trade halves so that 16
// lanes store 64 contiguous bytes of a row, directly and only inside the group.
// fp32: whole 32-row chunks go through shared memory and leave as bulk stores
// (stored directly, 4 bytes per lane, a 256 x 256 tile took 9700 clocks of
// stores, more than the MMAs of K = 1024: 65536 rows x 1024 x 4096 590 us, now 481),
// partial ones directly.
//
// Bound and rate: tensor pipe for long groups (65536 rows over 16 groups, 4096 x
// 1024: 361 to 381 us = 1520 to 1443 TFLOP/s in a short run, 533 clocks per stage of 512), HBM
// for short ones (64 rows over 64 groups, 1024 x 4096: 45.7 us for 280 MB of W =
// 6.1 TB/s).
struct RowsParams {
  Groups g;
  int N, K;
  int w_chunks;  // W [K][N] is mapped as 64-column chunks: both of a CTA in one box
  int dynamic;   // tiles are handed out; else taken in turn
  void* out;
  SelfTest test;
};

// What a tile's sums become: bf16 of one accumulator, bf16 or fp32 of summed chunks.
enum RowsOut { ROWS_BF16, ROWS_BF16_CHUNKS, ROWS_F32 };

template <int NT, bool F32>
struct RowsCfg {
  static constexpr int X_BYTES = NT / 2 * 128;
  static constexpr int STAGE = A_BYTES + X_BYTES;
  static constexpr int BOXES = F32 ? EPI_WARPS * EPI_BOX : 0;
  static constexpr int TAIL = BOXES + 320 + static_cast<int>(sizeof(TileSlots));
  static constexpr int STAGES = (232448 - 1024 - TAIL) / STAGE;
  static constexpr int SMEM = 1024 + STAGES * STAGE + TAIL;
  static constexpr int THREADS = 32 * (2 + EPI_WARPS + 1);
};

// 32 rows of a bf16 tile, from row r0 of it on: v holds this lane's column, nb + lane.
// Lane l stores columns nb + (l & ~1), + 1 of the even (odd) rows.
SHP_DEV void store_bf16_rows(const RowsParams& p, const RowTile& x, int r0, int nb, int lane,
                             const float* v) {
  const int odd = lane & 1;
  const bool in = nb + lane < p.N;  // N is even: a pair is in or out
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) +
                     static_cast<int64_t>(x.t0 + r0 + odd) * p.N + nb + lane - odd;
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
    const __nv_bfloat162 w = odd ? __floats2bfloat162_rn(got, v[j + 1])
                                 : __floats2bfloat162_rn(v[j], got);
    if (in && r0 + j + odd < x.count)
      *reinterpret_cast<__nv_bfloat162*>(o + static_cast<int64_t>(j) * p.N) = w;
  }
}

template <int NT, bool W_MN, RowsOut OUT>
__global__ void __launch_bounds__(RowsCfg<NT, OUT == ROWS_F32>::THREADS, 1)
    k_grouped_rows(const __grid_constant__ CUtensorMap tW, const __grid_constant__ CUtensorMap tX,
                   const __grid_constant__ CUtensorMap tX32,
                   const __grid_constant__ CUtensorMap tY, RowsParams p) {
  count_kernel_run();
  constexpr bool F32 = OUT == ROWS_F32, CHUNKS = OUT != ROWS_BF16;
  constexpr int CHUNK = F32 ? CHUNK_KB : LONG_KB;
  using C = RowsCfg<NT, F32>;
  constexpr int STAGES = C::STAGES;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int KB = (p.K + BK - 1) / BK;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* boxes = smem + STAGES * C::STAGE;
  TileSlots* slots = reinterpret_cast<TileSlots*>(boxes + C::BOXES);
  uint64_t* full = reinterpret_cast<uint64_t*>(slots + 1);
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;
  uint64_t* acce = accf + 2;
  uint64_t* drain = acce + 2;  // all MMAs of this pair complete
  uint64_t* never = drain + 1;  // completed by nothing: the self-test's wait
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
  volatile WaitState* ws = reinterpret_cast<volatile WaitState*>(never + 2);
  static_assert((2 * STAGES + 7) * 8 + sizeof(WaitState) <= 320, "barriers");

  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&accf[u], 1);
      mbar_init(&acce[u], 2 * EPI_WARPS);
    }
    mbar_init(drain, 1);
    mbar_init(never, 1);
    // consumers: producer and epilogue warps of both CTAs, MMA warp
    tile_slots_init(slots, 2 * (EPI_WARPS + 1) + 1);
    wait_state_init(ws, p.test.limit, KB);
    fence_barrier_init();
    tma_prefetch_desc(&tW);
    tma_prefetch_desc(&tX);
    tma_prefetch_desc(&tX32);
    if (F32) tma_prefetch_desc(&tY);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 2 * NT);
  RowTiles<NT> tiles(p.g, p.N);
  RowWalk walk(slots, ws);
  RowTile x;
  const int turn = static_cast<int>(blockIdx.x) / 2;
  walk.have = tiles.find(turn, walk.own);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // peer barriers initialised, both TMEM allocations done
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  if (warp == 0) {
    // ---------------- TMA producer (both CTAs): its 128 columns of W and its
    // half of the tile's rows, in boxes of 32
    const uint32_t on = elect_one(), lead = on & (leader ? 1u : 0u);
    RingPos<STAGES> ring;
    const uint32_t stages = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty);
    const uint32_t fleader = uniform(mapa_shared(full0, 0));
    bool stop = false;
    while (!stop && walk.next<true>(x)) {
      const int n0 = x.n0 + static_cast<int>(rank) * 128;
      const int half = ((x.count + 15) & ~15) / 2;  // rows per CTA
      const int t0 = x.t0 + static_cast<int>(rank) * half;
      // X in one box of NT / 2 rows, or in 32-row boxes where that moves less
      const bool small = half <= NT / 4;
      const int boxes = (half + 31) / 32;
      const uint32_t tx = 2 * (A_BYTES + (small ? boxes * 4096u : C::X_BYTES));
      for (int k0 = 0; k0 < p.K; k0 += BK) {
        if (!issue_wait<true>(empty0 + ring.slot * 8, ring.parity ^ 1u, ws)) {
          stop = true;
          break;
        }
        const uint32_t sw = stages + ring.slot * C::STAGE, sx = sw + A_BYTES;
        const uint32_t fbar = fleader + ring.slot * 8;
        mbar_expect_tx_if(lead, full0 + ring.slot * 8, tx);
        if (W_MN && p.w_chunks) {
          tma_4d_pair_if(on, sw, &tW, fbar, 0, k0, n0 >> 6, x.e);
        } else if (W_MN) {
          tma_3d_pair_if(on, sw, &tW, fbar, n0, k0, x.e);
          tma_3d_pair_if(on, sw + BK * 128, &tW, fbar, n0 + 64, k0, x.e);
        } else {
          tma_3d_pair_if(on, sw, &tW, fbar, k0, n0, x.e);
        }
        if (!small) {
          tma_3d_pair_if(on, sx, &tX, fbar, k0, t0, 0);
        } else {
          for (int i = 0; i < boxes; ++i)
            tma_3d_pair_if(on, sx + i * 4096, &tX32, fbar, k0, t0 + i * 32, 0);
        }
        ring.advance();
      }
    }
    // no copy may be in flight when the CTAs exit, also where a wait gave up and
    // no MMA waits for it (the leader's barriers count the peer's copies too)
    for (int k = 0; leader && k < STAGES; ++k, ring.advance())
      if (!mbar_wait(&full[ring.slot], ring.parity ^ 1u, nullptr, ws->limit)) break;
  } else if (warp == 1) {
    const bool gave_up = selftest_wait(p.test.stall, never, &ws->abort);
    if (leader) {
      // ---------------- MMA issuer (leader of the pair)
      const uint32_t on = elect_one();
      RingPos<STAGES> ring;
      RingPos<2> au;  // accumulator
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
      const uint32_t accf0 = smem_u32(accf), acce0 = smem_u32(acce);
      const uint64_t wdesc = W_MN ? smem_desc(smem_u32(smem), BK * 128, 1024u, 2u)
                                  : smem_desc(smem_u32(smem), 16, 1024u, 2u);
      const uint64_t xdesc = smem_desc(smem_u32(smem) + A_BYTES, 16, 1024u, 2u);
      constexpr uint64_t WSTEP = (W_MN ? 16 * 128 : 32) >> 4, XSTEP = 32 >> 4;
      bool stop = gave_up;
      while (!stop && walk.next(x)) {
        const uint32_t idesc = instr_desc(1u, W_MN, false, 256, (x.count + 15) & ~15);
        for (int c0 = 0; c0 < KB && !stop; c0 += CHUNKS ? CHUNK : KB, au.advance()) {
          const int c1 = CHUNKS ? min(c0 + CHUNK, KB) : KB;
          if (!issue_wait(acce0 + au.slot * 8, au.parity ^ 1u, ws)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t dacc = tmem + au.slot * NT;
          for (int kb = c0; kb < c1; ++kb) {
            if (!issue_wait(full0 + ring.slot * 8, ring.parity, ws)) {
              stop = true;
              break;
            }
            tc_fence_after();
            const uint64_t at = static_cast<uint64_t>(ring.slot) * (C::STAGE >> 4);
#pragma unroll
            for (int ks = 0; ks < BK / 16; ++ks)
              mma_f16_pair_if(on, dacc, wdesc + at + ks * WSTEP, xdesc + at + ks * XSTEP, idesc,
                              (kb > c0 || ks > 0) ? 1u : 0u);
            mma_commit_pair_if(on, empty0 + ring.slot * 8, 3);
            ring.advance();
          }
          mma_commit_pair_if(on, accf0 + au.slot * 8, 3);
        }
      }
      mma_commit_pair_if(on, smem_u32(drain), 3);  // after every MMA issued above
    }
  } else if (warp == 2 + EPI_WARPS) {
    // ---------------- scheduler (leader)
    if (leader && walk.have)
      schedule_tiles(
          slots, p.dynamic != 0, turn, static_cast<int>(gridDim.x) / 2,
          [&](int t, int(&v)[8]) {
            if (!tiles.find(t, x)) return false;
            v[0] = x.e;
            v[1] = x.t0;
            v[2] = x.count;
            v[3] = x.n0;
            return true;
          },
          ws);
  } else {
    // ---------------- epilogue warps (both CTAs, each on its TMEM rows): warp
    // (q, h) takes the W columns of lane quarter q and the 32-row chunks
    // h, h + 2, ... of the tile
    constexpr int NC = NT / 64;  // chunks per warp
    const int q = warp & 3, h = (warp - 2) >> 2;
    const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16);
    int it = 0;
    bool stop = false;
    while (!stop && walk.next(x)) {
      const int nb = x.n0 + static_cast<int>(rank) * 128 + q * 32;  // this warp's first column
      if (CHUNKS) {
        float acc[NC * 32];
#pragma unroll
        for (int j = 0; j < NC * 32; ++j) acc[j] = 0.f;
        for (int c0 = 0; c0 < KB; c0 += CHUNK, ++it) {
          const int u = it & 1;
          if (!warp_wait(smem_u32(&accf[u]), (it >> 1) & 1, ws)) {
            stop = true;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            if ((2 * c + h) * 32 < x.count) {
              float v[32];
              tmem_ld32(trow + static_cast<uint32_t>(u * NT + (2 * c + h) * 32), v);
#pragma unroll
              for (int j = 0; j < 32; ++j) acc[c * 32 + j] += v[j];
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_relaxed(mapa_shared(smem_u32(&acce[u]), 0));
        }
        if (stop) break;
        if (!F32) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if ((2 * c + h) * 32 < x.count)
              store_bf16_rows(p, x, (2 * c + h) * 32, nb, lane, acc + c * 32);
        } else if (nb < p.N) {
          uint8_t* box = boxes + (warp - 2) * EPI_BOX;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const int r0 = (2 * c + h) * 32;
            if (r0 + 32 <= x.count) {  // whole chunks leave as bulk stores
              if (lane == 0) bulk_wait_read_all();  // the last store has read the box
              __syncwarp();
#pragma unroll
              for (int j = 0; j < 32; ++j)
                *reinterpret_cast<float*>(box + sw128_off(j, lane >> 2) + (lane & 3) * 4) =
                    acc[c * 32 + j];
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_3d(&tY, box, nb, x.t0 + r0, 0);
                bulk_commit();
              }
            } else if (r0 < x.count && nb + lane < p.N) {
              float* o = static_cast<float*>(p.out) + static_cast<int64_t>(x.t0 + r0) * p.N + nb + lane;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (r0 + j < x.count) o[static_cast<int64_t>(j) * p.N] = acc[c * 32 + j];
            }
          }
        }
      } else {
        const int u = it & 1;
        if (!warp_wait(smem_u32(&accf[u]), (it >> 1) & 1, ws)) break;
        ++it;
        tc_fence_after();
        // store_bf16_rows, written out: called, the compiler works the row addresses out
        // again for every 32 rows (72 registers, not 114; 8192 rows over 64 blocks of
        // 1024 x 4096: 101.1 us, not 99.8)
        const int odd = lane & 1;
        const bool in = nb + lane < p.N;  // N is even: a pair is in or out
#pragma unroll 1
        for (int r0 = h * 32; r0 < x.count; r0 += 64) {
          float v[32];
          tmem_ld32(trow + static_cast<uint32_t>(u * NT + r0), v);
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) +
                             static_cast<int64_t>(x.t0 + r0 + odd) * p.N + nb + lane - odd;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
            const __nv_bfloat162 w = odd ? __floats2bfloat162_rn(got, v[j + 1])
                                         : __floats2bfloat162_rn(v[j], got);
            if (in && r0 + j + odd < x.count)
              *reinterpret_cast<__nv_bfloat162*>(o + static_cast<int64_t>(j) * p.N) = w;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(mapa_shared(smem_u32(&acce[u]), 0));
      }
    }
    if (F32) {
      if (lane == 0) bulk_wait_all();  // nothing outlives the CTA's shared memory
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();  // every role of this CTA has left its loop
  // so the pair's MMAs have only to complete, which a limit of a stage bounds
  if (warp == 1) mbar_wait(drain, 0, nullptr, ws->limit);
  selftest_report(p.test.status, &ws->abort);
  // releasing: this CTA's arrivals on the other's barriers land before it exits
  cluster_sync();
  if (warp == 1) tmem_dealloc_pair(tmem, 2 * NT);
}

// -------------------------------------------------------- weight gradient
//
// k_grouped_wgrad: 256 x 256 tiles of G_e, both operands MN-major (rows of A
// and B are the contraction), a 128-column half of each per CTA.  A tile's time
// follows its group's rows, so tiles are handed out as pairs become free, and
// where they are long the largest groups' first: for 16 groups of 0.3 to 13
// thousand rows the busiest pair has 1 % more stages than the mean, in a fixed
// rotation 10 %.
// Bound and rate: tensor pipe for long groups (that case, 1024 x 4096,
// accumulated: 414 us = 1328 TFLOP/s in a short run), the stores of G for short
// ones (64 groups of 256 rows, 1024^2: 61 us for 335 MB = 5.5 TB/s; a kernel that
// only stores such tiles takes 50 us for their 268 MB).

constexpr int STAGE_BYTES = 2 * A_BYTES;
constexpr int STAGES = 6;
constexpr int BN = 256;
constexpr int THREADS = 32 * (2 + EPI_WARPS + 2);

constexpr int SORT_MAX = 256;  // groups that are put in order (each thread compares all)

// order[i] = the group of the i-th largest size (ties by number).  Called by all
// threads of a block of at least SORT_MAX; `len` is scratch in shared memory.
SHP_DEV void sort_groups(const Groups& g, uint16_t* order, int* len) {
  const int e = static_cast<int>(threadIdx.x);
  if (e < g.n) {
    int lo, hi;
    g.range(e, lo, hi);
    len[e] = hi - lo;
  }
  __syncthreads();
  if (e < g.n) {
    int rank = 0;
    for (int j = 0; j < g.n; ++j) rank += len[j] > len[e] || (len[j] == len[e] && j < e);
    order[rank] = static_cast<uint16_t>(e);
  }
}

constexpr int GSMEM = 1024 + STAGES * STAGE_BYTES + EPI_WARPS * EPI_BOX + 320 +
                      static_cast<int>(sizeof(TileSlots)) + SORT_MAX * 2;
static_assert(GSMEM <= 232448, "weight-gradient kernel exceeds shared memory");

struct WgradParams {
  Groups g;
  int M, N;
  int accumulate;
  int chunks;   // A and B are mapped as 64-column chunks: both of a CTA in one box
  int sorted;   // the largest groups' tiles first
  int dynamic;  // tiles are handed out; else taken in turn
  SelfTest test;
};

// One tile: group e, tile (m0, n0), kb stages from row k0; `tail` valid rows in
// the last stage (0: all 64).  Clearing a partial stage and handing it over
// takes longer than a stage's MMAs, so it is loaded TAIL_EARLY stages ahead of
// its turn (`tail_at`: its place in the order of loading; -1: none) and used
// last: 64 groups of 250 rows, 1024 x 1024: 77 -> 72 us (of 256 rows: 64 us).
constexpr int TAIL_EARLY = STAGES - 2;  // the stages behind it still fit in the ring
struct Tile {
  int e, m0, n0, k0, len, kb, tail, tail_at;
};

// A role's walk over its pair's tiles: its own, then the scheduler's.
struct Walk {
  const WgradParams& p;
  const uint16_t* order;  // groups by falling size; null: in their own order
  TileFeed feed;
  int tiles_n, per_e;
  bool first = true;
  Tile own;
  SHP_DEV Walk(const WgradParams& q, const uint16_t* o, TileSlots* ts, volatile WaitState* ws)
      : p(q), order(o), feed{ts, ws} {
    tiles_n = (q.N + BN - 1) / BN;
    per_e = tiles_n * ((q.M + 255) / 256);
  }
  SHP_DEV bool find(int t, Tile& x) const {
    if (t >= per_e * p.g.n) return false;
    const int i = t / per_e, r = t % per_e;
    x.e = order != nullptr ? uniform(static_cast<int>(order[i])) : i;
    int lo, hi;
    p.g.range(x.e, lo, hi);
    x.m0 = r / tiles_n * 256;
    x.n0 = r % tiles_n * BN;
    x.k0 = uniform(lo);
    rows(x, uniform(hi - lo));
    return true;
  }
  SHP_DEV static void rows(Tile& x, int len) {
    x.len = len;
    x.kb = (len + BK - 1) / BK;
    x.tail = len % BK;
    x.tail_at = x.tail == 0 ? -1 : max(0, x.kb - 1 - TAIL_EARLY);
  }
  template <bool PRODUCER = false>
  SHP_DEV bool next(Tile& x) {
    if (first) {
      first = false;
      x = own;
      return true;
    }
    int v[8];
    feed.next<PRODUCER>(v);
    x.e = v[0];
    x.m0 = v[1];
    x.n0 = v[2];
    x.k0 = v[3];
    rows(x, v[4]);
    return x.e >= 0;
  }
};

__global__ void __launch_bounds__(THREADS, 1)
    k_grouped_wgrad(const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tB,
                    const __grid_constant__ CUtensorMap tO, WgradParams p) {
  count_kernel_run();
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* boxes = smem + STAGES * STAGE_BYTES;
  TileSlots* slots = reinterpret_cast<TileSlots*>(boxes + EPI_WARPS * EPI_BOX);
  uint64_t* full = reinterpret_cast<uint64_t*>(slots + 1);
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;
  uint64_t* acce = accf + 2;
  uint64_t* tailb = acce + 2;        // per stage: a partial stage of this CTA has landed
  uint64_t* clearb = tailb + STAGES;  // per stage (leader): the peer's half is cleared
  uint64_t* drain = clearb + STAGES;  // all MMAs of this pair complete
  uint64_t* never = drain + 1;        // completed by nothing: the self-test's wait
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
  volatile WaitState* ws = reinterpret_cast<volatile WaitState*>(never + 2);
  uint16_t* order = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(full) + 320);
  static_assert((4 * STAGES + 7) * 8 + sizeof(WaitState) <= 320, "barriers");
  const bool sorted = p.sorted != 0;

  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tailb[s], 1);
      mbar_init(&clearb[s], 1);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&accf[u], 1);
      mbar_init(&acce[u], 2 * EPI_WARPS);
    }
    mbar_init(drain, 1);
    mbar_init(never, 1);
    // consumers: producer, epilogue and clearing warps of both CTAs, MMA warp
    tile_slots_init(slots, 2 * (EPI_WARPS + 2) + 1);
    wait_state_init(ws, p.test.limit, p.g.T / BK + 1);
    fence_barrier_init();
    tma_prefetch_desc(&tA);
    tma_prefetch_desc(&tB);
    tma_prefetch_desc(&tO);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 2 * BN);
  if (sorted) {
    sort_groups(p.g, order, reinterpret_cast<int*>(smem));
    fence_proxy_async_smem();  // before the copies that reuse the space
  }
  Walk walk(p, sorted ? order : nullptr, slots, ws);
  Tile x;
  const int turn = static_cast<int>(blockIdx.x) / 2;
  if (!sorted) walk.find(turn, walk.own);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // peer barriers initialised, both TMEM allocations done
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  if (sorted) walk.find(turn, walk.own);
  if (warp == 0) {
    // ---------------- TMA producer (both CTAs)
    const uint32_t on = elect_one(), lead = on & (leader ? 1u : 0u);
    RingPos<STAGES> ring;
    const uint32_t stages = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty);
    const uint32_t tail0 = smem_u32(tailb), fleader = uniform(mapa_shared(full0, 0));
    uint32_t tails = 0, tpar = 0;  // per slot: its last use is a partial stage; tailb's next phase
    bool stop = false;
    while (!stop && walk.next<true>(x)) {
      const int m0 = x.m0 + static_cast<int>(rank) * 128;
      const int nb0 = x.n0 + static_cast<int>(rank) * 128;
      int k0 = x.k0;
      for (int l = 0; l < x.kb; ++l) {
        if (!issue_wait<true>(empty0 + ring.slot * 8, ring.parity ^ 1u, ws)) {
          stop = true;
          break;
        }
        const uint32_t sa = stages + ring.slot * STAGE_BYTES, sb = sa + A_BYTES;
        if (l == x.tail_at) {
          // partial stage: this CTA's halves, for the clearing warp
          const uint32_t bar = tail0 + ring.slot * 8;
          const int kt = x.k0 + (x.kb - 1) * BK;
          tails |= 1u << ring.slot;
          tpar ^= 1u << ring.slot;
          mbar_expect_tx_if(on, bar, STAGE_BYTES);
          if (p.chunks) {
            tma_4d_if(on, sa, &tA, bar, 0, kt, m0 >> 6, 0);
            tma_4d_if(on, sb, &tB, bar, 0, kt, nb0 >> 6, 0);
          } else {
            for (int i = 0; i < 2; ++i) {
              tma_3d_if(on, sa + i * BK * 128, &tA, bar, m0 + i * 64, kt, 0);
              tma_3d_if(on, sb + i * BK * 128, &tB, bar, nb0 + i * 64, kt, 0);
            }
          }
        } else {
          const uint32_t fbar = fleader + ring.slot * 8;
          tails &= ~(1u << ring.slot);
          mbar_expect_tx_if(lead, full0 + ring.slot * 8, 2 * STAGE_BYTES);
          if (p.chunks) {
            tma_4d_pair_if(on, sa, &tA, fbar, 0, k0, m0 >> 6, 0);
            tma_4d_pair_if(on, sb, &tB, fbar, 0, k0, nb0 >> 6, 0);
          } else {
            for (int i = 0; i < 2; ++i) {
              tma_3d_pair_if(on, sa + i * BK * 128, &tA, fbar, m0 + i * 64, k0, 0);
              tma_3d_pair_if(on, sb + i * BK * 128, &tB, fbar, nb0 + i * 64, k0, 0);
            }
          }
          k0 += BK;
        }
        ring.advance();
      }
    }
    // no copy may be in flight when the CTAs exit, also where a wait gave up and
    // no MMA waits for it: partial stages land on this CTA's own barriers, the
    // others of both CTAs on the leader's
    for (int k = 0; k < STAGES; ++k, ring.advance()) {
      const uint32_t s = ring.slot;
      if ((tails >> s) & 1)
        mbar_wait(&tailb[s], ((tpar >> s) & 1) ^ 1u, nullptr, ws->limit);
      else if (leader)
        mbar_wait(&full[s], ring.parity ^ 1u, nullptr, ws->limit);
    }
  } else if (warp == 1) {
    const bool gave_up = selftest_wait(p.test.stall, never, &ws->abort);
    if (leader) {
      // ---------------- MMA issuer (leader of the pair)
      const uint32_t idesc = instr_desc(1u, true, true, 256, BN);
      const uint32_t on = elect_one();
      RingPos<STAGES> ring;
      RingPos<2> au;  // accumulator
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
      const uint32_t accf0 = smem_u32(accf), acce0 = smem_u32(acce);
      const uint64_t adesc = smem_desc(smem_u32(smem), BK * 128, 1024u, 2u);
      const uint64_t bdesc = smem_desc(smem_u32(smem) + A_BYTES, BK * 128, 1024u, 2u);
      constexpr uint64_t KSTEP = 16 * 128 >> 4;
      bool stop = gave_up;
      while (!stop && walk.next(x)) {
        int l = 0;                 // place in the order of loading
        RingPos<STAGES> tail = ring;  // where the partial stage is
        for (int kb = 0; kb < x.kb; ++kb) {
          const int c = kb % CHUNK_KB;
          if (c == 0 && !issue_wait(acce0 + au.slot * 8, au.parity ^ 1u, ws)) {
            stop = true;
            break;
          }
          if (l++ == x.tail_at) {
            tail = ring;
            ring.advance();
            ++l;
          }
          const bool last = kb == x.kb - 1, partial = last && x.tail != 0;
          const RingPos<STAGES> at = partial ? tail : ring;
          if (!issue_wait(full0 + at.slot * 8, at.parity, ws)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t dacc = tmem + au.slot * BN;
          const uint64_t da = static_cast<uint64_t>(at.slot) * (STAGE_BYTES >> 4);
          if (!partial) {
            ring.advance();
#pragma unroll
            for (int ks = 0; ks < BK / 16; ++ks)
              mma_f16_pair_if(on, dacc, adesc + da + ks * KSTEP, bdesc + da + ks * KSTEP, idesc,
                              (c > 0 || ks > 0) ? 1u : 0u);
          } else {
            for (int ks = 0; ks < (x.tail + 15) / 16; ++ks)
              mma_f16_pair_if(on, dacc, adesc + da + ks * KSTEP, bdesc + da + ks * KSTEP, idesc,
                              (c > 0 || ks > 0) ? 1u : 0u);
          }
          mma_commit_pair_if(on, empty0 + at.slot * 8, 3);
          if (last || c == CHUNK_KB - 1) {
            mma_commit_pair_if(on, accf0 + au.slot * 8, 3);
            au.advance();
          }
        }
      }
      mma_commit_pair_if(on, smem_u32(drain), 3);  // after every MMA issued above
    }
  } else if (warp < 2 + EPI_WARPS) {
    // ---------------- epilogue warps (both CTAs, each on its TMEM rows)
    const int q = warp & 3, h = (warp - 2) >> 2;
    uint8_t* box = boxes + (warp - 2) * EPI_BOX;
    const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * 128u;
    int it = 0;
    bool stop = false;
    while (!stop && walk.next(x)) {
      const int row0 = x.m0 + static_cast<int>(rank) * 128 + q * 32;
      const int c0 = x.n0 + h * 128;
      float acc[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) acc[j] = 0.f;
      const int nc = (x.kb + CHUNK_KB - 1) / CHUNK_KB;
      for (int c = 0; c < nc; ++c, ++it) {
        const int u = it & 1;
        if (!warp_wait(smem_u32(&accf[u]), (it >> 1) & 1, ws)) {
          stop = true;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float v[32];
          tmem_ld32(trow + static_cast<uint32_t>(u * BN + g * 32), v);
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[g * 32 + j] += v[j];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(mapa_shared(smem_u32(&acce[u]), 0));
      }
      if (stop) break;
      if (p.accumulate && nc == 0) continue;  // an empty group leaves G as it is
      if (row0 >= p.M) continue;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int cb = c0 + g * 32;
        if (cb >= p.N) continue;
        // the warp's box, or, when no more tiles come, a box of its own for
        // each store in the stages, which nothing reads or fills any more
        uint8_t* bx = p.dynamic ? box : smem + ((warp - 2) * 4 + g) * EPI_BOX;
        if (p.dynamic) {
          if (lane == 0) bulk_wait_read_all();  // the last store has read the box
          __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4*>(bx + sw128_off(lane, i)) =
              make_float4(acc[g * 32 + 4 * i], acc[g * 32 + 4 * i + 1], acc[g * 32 + 4 * i + 2],
                          acc[g * 32 + 4 * i + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (p.accumulate)
            tma_reduce_add_3d(&tO, bx, cb, row0, x.e);
          else
            tma_store_3d(&tO, bx, cb, row0, x.e);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait_all();  // nothing outlives the CTA's shared memory
    __syncwarp();
  } else if (warp == 2 + EPI_WARPS + 1) {
    // ---------------- scheduler (leader)
    if (leader)
      schedule_tiles(
          slots, p.dynamic != 0, turn, static_cast<int>(gridDim.x) / 2,
          [&](int t, int(&v)[8]) {
            if (!walk.find(t, x)) return false;
            v[0] = x.e;
            v[1] = x.m0;
            v[2] = x.n0;
            v[3] = x.k0;
            v[4] = x.len;
            return true;
          },
          ws);
  } else {
    // ---------------- clearing warp: rows behind the group in its last stage
    int kit = 0;
    uint32_t par = 0;  // phase of each stage's tailb and clearb
    while (walk.next(x)) {
      const int s = (kit + max(x.tail_at, 0)) % STAGES;
      kit = (kit + x.kb) % STAGES;
      if (x.tail == 0) continue;
      if (!warp_wait(smem_u32(&tailb[s]), (par >> s) & 1, ws, true)) break;
      uint8_t* st = smem + s * STAGE_BYTES;
      const int r1 = (x.tail + 15) / 16 * 16;
      // four 64-column chunks (two of A, two of B) of 64 rows of 128 bytes
      for (int r = x.tail + (lane >> 3); r < r1; r += 4) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(st + c * BK * 128 + r * 128 + (lane & 7) * 16) =
              make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      // the leader hands the stage over once both halves are cleared
      if (!leader) {
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&clearb[s]), 0));
      } else {
        if (!warp_wait_cluster(smem_u32(&clearb[s]), (par >> s) & 1, ws)) break;
        if (lane == 0) mbar_arrive(&full[s]);
      }
      par ^= 1u << s;
    }
  }

  tc_fence_before();
  __syncthreads();  // every role of this CTA has left its loop
  // so the pair's MMAs have only to complete, which a limit of a stage bounds
  if (warp == 1) mbar_wait(drain, 0, nullptr, ws->limit);
  selftest_report(p.test.status, &ws->abort);
  // releasing: this CTA's arrivals on the other's barriers land before it exits
  cluster_sync();
  if (warp == 1) tmem_dealloc_pair(tmem, 2 * BN);
}

// A launch of `pairs` CTA pairs.
cudaLaunchConfig_t pair_grid(int64_t pairs, int threads, int smem, cudaStream_t st,
                             cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (pairs > 1 ? pairs : 1)), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = 2;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int NT, bool W_MN, RowsOut OUT>
cudaError_t launch_rows(const CUtensorMap& w, const CUtensorMap& x, const CUtensorMap& x32,
                        const CUtensorMap& y, RowsParams p, int T, cudaStream_t st) {
  using C = RowsCfg<NT, OUT == ROWS_F32>;
  auto kern = k_grouped_rows<NT, W_MN, OUT>;
  static std::atomic<uint64_t> done{0};
  const LaunchInfo li = launch_info(reinterpret_cast<const void*>(kern), C::SMEM, done);
  if (li.err != cudaSuccess) return li.err;
  // every group with rows has at most one row tile more than its full ones
  const int64_t tiles = (T / NT + static_cast<int64_t>(p.g.n < T ? p.g.n : T)) * ((p.N + 255) / 256);
  // Handing tiles out pays where their rows, and so their times, differ: 16384
  // rows over 32 skewed groups, 512 x 2048, 44 us against 50 in turn (equal
  // groups: 47 and 46).  Few rows per group cost the same everywhere, and asking
  // for tiles is in the way: 16 rows over 64 groups, 1024 x 4096, 26.4 us
  // against 25.6.  (Largest groups first, as in the weight gradient, did not
  // pay here: 46 us.)
  const int64_t pairs = li.sms / 2;
  p.dynamic = tiles > pairs && T > 32 * static_cast<int64_t>(p.g.n) ? 1 : 0;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg =
      pair_grid(p.dynamic || tiles < pairs ? tiles : pairs, C::THREADS, C::SMEM, st, &attr);
  return cudaLaunchKernelEx(&cfg, kern, w, x, x32, y, p);
}

template <int NT, bool W_MN>
cudaError_t dispatch_out(const CUtensorMap& w, const CUtensorMap& x, const CUtensorMap& x32,
                         const CUtensorMap& y, bool f32, const RowsParams& p, int T,
                         cudaStream_t st) {
  if (f32) return launch_rows<NT, W_MN, ROWS_F32>(w, x, x32, y, p, T, st);
  return p.K > LONG_KB * BK ? launch_rows<NT, W_MN, ROWS_BF16_CHUNKS>(w, x, x32, y, p, T, st)
                      : launch_rows<NT, W_MN, ROWS_BF16>(w, x, x32, y, p, T, st);
}

template <int NT>
cudaError_t dispatch_rows(const void* X, const CUtensorMap& w, bool w_mn, bool f32,
                          const RowsParams& p, int T, cudaStream_t st) {
  CUtensorMap x, x32, y;
  memset(&y, 0, sizeof(y));
  if (f32 && !tensor_map(&y, p.out, 4, p.N, T, 1, p.N, 0, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  if (!tensor_map(&x, X, 2, p.K, T, 1, p.K, 0, BK, NT / 2, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tensor_map(&x32, X, 2, p.K, T, 1, p.K, 0, BK, 32, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  return w_mn ? dispatch_out<NT, true>(w, x, x32, y, f32, p, T, st)
              : dispatch_out<NT, false>(w, x, x32, y, f32, p, T, st);
}

// Rows per tile.  The host knows the mean size of a group only, so it counts as
// if all were equal: rounds of tiles over the SM pairs, times a tile's cost,
// which grows with its rows beyond streaming W (a tile of 256 rows takes 1.6
// times one of 16, measured).  Equal counts: with several rounds the larger
// tile (fewer reads of W where groups differ: 8192 skewed rows over 64 blocks
// of 1024 x 4096, 106 us against 116 with 128 and 145 with 64), in one round
// the smaller (16 blocks of 4096 x 1024 with 16 rows each: 29 us against 32).
int rows_per_tile(int64_t T, int64_t N, int64_t groups, int64_t pairs) {
  const int64_t tn = (N + 255) / 256;
  const int64_t used = groups < T ? groups : T, mean = (T + used - 1) / used;
  int best = 0;
  double best_cost = 0;
  int64_t best_rounds = 0;
  for (int nt = 64; nt <= 256; nt *= 2) {
    const int64_t per_group = (mean + nt - 1) / nt;
    const int64_t rounds = (used * per_group * tn + pairs - 1) / pairs;
    const double rows = static_cast<double>(mean) / static_cast<double>(per_group);
    const double cost = static_cast<double>(rounds) * (1.0 + rows / 340.0);
    if (best == 0 || cost < best_cost || (cost == best_cost && best_rounds > 1)) {
      best = nt;
      best_cost = cost;
      best_rounds = rounds;
    }
  }
  return best;
}

}  // namespace

cudaError_t grouped_rows(const void* X, const int64_t* offsets, const void* W, bool w_trans,
                         void* Y, int T, int K, int N, int groups, bool f32, cudaStream_t st,
                         const SelfTest& selftest) {
  RowsParams p;
  memset(&p, 0, sizeof(p));
  p.g = Groups{offsets, groups, T};
  p.N = N;
  p.K = K;
  p.out = Y;
  p.test = selftest;
  CUtensorMap w;
  const int64_t kn = static_cast<int64_t>(K) * N;
  bool ok;
  if (w_trans) {
    ok = tensor_map(&w, W, 2, K, N, groups, K, kn, BK, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  } else if (N % 64 == 0) {
    p.w_chunks = 1;
    ok = tensor_map4(&w, W, 2, {64, K, N / 64, groups}, {N, 64, kn}, {64, BK, 2, 1},
                     CU_TENSOR_MAP_SWIZZLE_128B);
  } else {
    ok = tensor_map(&w, W, 2, N, K, groups, N, kn, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (!ok) return cudaErrorInvalidValue;
  const LaunchInfo li = device_info();
  if (li.err != cudaSuccess) return li.err;
  switch (rows_per_tile(T, N, groups, li.sms / 2)) {
    case 64: return dispatch_rows<64>(X, w, !w_trans, f32, p, T, st);
    case 128: return dispatch_rows<128>(X, w, !w_trans, f32, p, T, st);
    default: return dispatch_rows<256>(X, w, !w_trans, f32, p, T, st);
  }
}

cudaError_t grouped_wgrad(const void* A, const void* B, const int64_t* offsets, float* G, int T,
                          int M, int N, int groups, bool accumulate, cudaStream_t st,
                          const SelfTest& selftest) {
  WgradParams p;
  memset(&p, 0, sizeof(p));
  CUtensorMap a, b, o;
  bool ok = tensor_map(&o, G, 4, N, M, groups, N, static_cast<int64_t>(M) * N, 32, 32,
                       CU_TENSOR_MAP_SWIZZLE_128B);
  if (T == 0) {
    a = b = o;  // no group has a row: never loaded from
  } else if (M % 64 == 0 && N % 64 == 0) {
    p.chunks = 1;
    ok = ok &&
         tensor_map4(&a, A, 2, {64, T, M / 64, 1}, {M, 64, static_cast<int64_t>(T) * M},
                     {64, BK, 2, 1}, CU_TENSOR_MAP_SWIZZLE_128B) &&
         tensor_map4(&b, B, 2, {64, T, N / 64, 1}, {N, 64, static_cast<int64_t>(T) * N},
                     {64, BK, 2, 1}, CU_TENSOR_MAP_SWIZZLE_128B);
  } else {
    ok = ok && tensor_map(&a, A, 2, M, T, 1, M, 0, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B) &&
         tensor_map(&b, B, 2, N, T, 1, N, 0, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (!ok) return cudaErrorInvalidValue;
  p.g = Groups{offsets, groups, T};
  p.M = M;
  p.N = N;
  p.accumulate = accumulate ? 1 : 0;
  p.test = selftest;
  const int64_t tiles = static_cast<int64_t>(groups) * ((M + 255) / 256) * ((N + BN - 1) / BN);
  static std::atomic<uint64_t> done{0};
  const LaunchInfo li = launch_info(reinterpret_cast<const void*>(k_grouped_wgrad), GSMEM, done);
  if (li.err != cudaSuccess) return li.err;
  const int64_t pairs = li.sms / 2;
  p.dynamic = tiles > pairs ? 1 : 0;
  // Largest groups first ends even (16 skewed groups of about 4096 rows, 4096 x
  // 1024: 421 us against 450), but puts the tiles that are all MMAs before those
  // that are all stores: with few rows per tile mixing them is better (64 skewed
  // groups of about 256 rows, 1024^2: 86 us sorted, 81 not; of 128 rows, 1024 x
  // 4096: 241 and 229; from about 512 rows on, 43 and 52).
  p.sorted = p.dynamic && groups <= SORT_MAX && T >= 512 * static_cast<int64_t>(groups) ? 1 : 0;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg =
      pair_grid(p.dynamic || tiles < pairs ? tiles : pairs, THREADS, GSMEM, st, &attr);
  return cudaLaunchKernelEx(&cfg, k_grouped_wgrad, a, b, o, p);
}

uint64_t kernel_runs_grouped() {
  unsigned long long v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kernel_runs, sizeof(v)) != cudaSuccess) return 0;
  return v;
}

}  // namespace shp
