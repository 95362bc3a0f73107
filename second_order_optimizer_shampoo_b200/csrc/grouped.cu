// Products of rows grouped by expert (weight block) on the sm_100a tensor
// cores: the forward product of an expert layer, the gradient of its input
// and the gradient of its weight blocks, which the Shampoo statistics take.
//
//   rows      Y[t]  = X[t] W_e  (or X[t] W_e^T),  t in [off_e, off_{e+1})
//   wgrad     G_e   = A_e^T B_e (+ G_e),  A_e, B_e the rows [off_e, off_{e+1})
//
// bf16 operands, fp32 accumulation.  The group boundaries are read on the
// device, so nothing waits for the host.  k_grouped is a persistent CTA-pair
// kernel (one tcgen05 MMA of M = 256 over two SMs, 256 x 256 tiles, TMA ring,
// two TMEM accumulators so that the epilogue of one tile runs beside the main
// loop of the next), like the batched product of gemm_tc.cu; what differs is
// where tiles come from (a warp-wide scan of the offsets), the ragged edges,
// and the fp32 sums:
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
//     nearest, while the next chunk's MMAs run.  bf16 results take one chunk.
#include <cuda_bf16.h>
#include <string.h>

#include "internal.h"
#include "shp_common.cuh"

namespace shp {

namespace {

constexpr int ROWB = 128;                 // bytes of one row of a stage tile
constexpr int BK = 64;                    // contraction elements per stage
constexpr int A_BYTES = 128 * ROWB;       // per CTA: 128 rows (columns) of A ...
constexpr int STAGE_BYTES = 2 * A_BYTES;  // ... and 128 of B
constexpr int STAGES = 6;
constexpr int BN = 256;
constexpr int CHUNK_KB = 8;  // stages per fp32 chunk: sums of 512 products inside the tensor core
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (2 + EPI_WARPS + 1);
constexpr int EPI_BOX = 4096;  // one warp's 32-row store box
constexpr int GSMEM = 1024 + STAGES * STAGE_BYTES + EPI_WARPS * EPI_BOX + 320;
static_assert(GSMEM <= 232448, "grouped kernel exceeds shared memory");

SHP_DEV void tma_reduce_add_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group"
      " [%0, {%2, %3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

SHP_DEV void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

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

// Walks the row tiles of all groups in order.  find(t) is called by a whole
// warp with increasing t and leaves the group and the tile's number within
// it; 32 groups are looked at per step.
struct RowTiles {
  Groups g;
  int rows_per_tile, tiles_n;
  int e0 = 0;    // first group of the window
  int base = 0;  // tiles before the window
  int lo = 0, hi = 0, e = 0;
  SHP_DEV bool find(int t, int& r) {
    const int lane = threadIdx.x & 31;
    while (e0 < g.n) {
      int a = 0, b = 0, cnt = 0;
      if (e0 + lane < g.n) {
        g.range(e0 + lane, a, b);
        cnt = (b - a + rows_per_tile - 1) / rows_per_tile * tiles_n;
      }
      int inc = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const unsigned in = __ballot_sync(0xffffffffu, t < base + inc);
      if (in != 0) {
        const int src = __ffs(in) - 1;
        r = t - base - __shfl_sync(0xffffffffu, inc - cnt, src);
        lo = __shfl_sync(0xffffffffu, a, src);
        hi = __shfl_sync(0xffffffffu, b, src);
        e = e0 + src;
        return true;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
      e0 += 32;
    }
    return false;
  }
};

struct GroupedParams {
  Groups g;
  int M;  // wgrad: rows of G (columns of A); rows product: unused
  int N, K;
  void* out;
  int accumulate;
};

// One tile: group e, tile rows from m0 (a row of X, or a row of G), columns
// from n0, `kb` stages of contraction starting at row / column k0; `tail`
// valid rows in the last stage (0: all 64).
struct Tile {
  int e, m0, n0, k0, kb, tail, mend;
};

// The tiles of a CTA pair in order; every role of the kernel walks the same
// sequence.  Called by whole warps.
template <bool WG>
struct Walk {
  const GroupedParams& p;
  RowTiles rt;
  int t, step, tiles_n, per_e;
  SHP_DEV Walk(const GroupedParams& q, int first, int stride) : p(q), t(first), step(stride) {
    tiles_n = (q.N + BN - 1) / BN;
    per_e = tiles_n * ((q.M + 255) / 256);
    rt.g = q.g;
    rt.rows_per_tile = 256;
    rt.tiles_n = tiles_n;
  }
  SHP_DEV bool next(Tile& x) {
    if (WG) {
      if (t >= per_e * p.g.n) return false;
      x.e = t / per_e;
      const int r = t % per_e;
      int lo, hi;
      p.g.range(x.e, lo, hi);
      x.m0 = r / tiles_n * 256;
      x.mend = p.M;
      x.n0 = r % tiles_n * BN;
      x.k0 = lo;
      x.kb = (hi - lo + BK - 1) / BK;
      x.tail = (hi - lo) % BK;
    } else {
      int r;
      if (!rt.find(t, r)) return false;
      x.e = rt.e;
      x.m0 = rt.lo + r / tiles_n * 256;
      x.mend = rt.hi;
      x.n0 = r % tiles_n * BN;
      x.k0 = 0;
      x.kb = (p.K + BK - 1) / BK;
      x.tail = 0;
    }
    t += step;
    return true;
  }
};

template <bool WG, bool B_MN, bool F32>
__global__ void __launch_bounds__(THREADS, 1)
    k_grouped(const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tB,
              const __grid_constant__ CUtensorMap tO, GroupedParams p) {
  count_kernel_run();
  constexpr bool A_MN = WG;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int ncl = static_cast<int>(gridDim.x) / 2, cl = static_cast<int>(blockIdx.x) / 2;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* boxes = smem + STAGES * STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(boxes + EPI_WARPS * EPI_BOX);
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;
  uint64_t* acce = accf + 2;
  uint64_t* tailb = acce + 2;        // per stage: a partial stage of this CTA has landed
  uint64_t* clearb = tailb + STAGES;  // per stage (leader): the peer's half is cleared
  uint64_t* drain = clearb + STAGES;  // all MMAs of this pair complete
  volatile int* abort_flag = reinterpret_cast<volatile int*>(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1) + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tA);
    tma_prefetch_desc(&tB);
    tma_prefetch_desc(&tO);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 2 * BN);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // peer barriers initialised, both TMEM allocations done
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  Walk<WG> walk(p, cl, ncl);
  Tile x;
  if (warp == 0) {
    // ---------------- TMA producer (both CTAs)
    int kit = 0;
    bool stop = false;
    while (!stop && walk.next(x)) {
      const int m0 = x.m0 + static_cast<int>(rank) * 128;
      const int nb0 = x.n0 + static_cast<int>(rank) * 128;
      if (lane == 0) {
        for (int kb = 0; kb < x.kb; ++kb, ++kit) {
          const int s = kit % STAGES;
          if (kit >= STAGES &&
              (*abort_flag || !mbar_wait(&empty[s], ((kit / STAGES) - 1) & 1, abort_flag))) {
            *abort_flag = 1;
            stop = true;
            break;
          }
          uint8_t* sa = smem + s * STAGE_BYTES;
          uint8_t* sb = sa + A_BYTES;
          const int k0 = x.k0 + kb * BK;
          if (WG && x.tail != 0 && kb == x.kb - 1) {
            // partial stage: this CTA's halves, for the clearing warp
            mbar_arrive_expect_tx(&tailb[s], STAGE_BYTES);
            for (int i = 0; i < 2; ++i) {
              tma_load_3d(sa + i * BK * 128, &tA, &tailb[s], m0 + i * 64, k0, 0);
              tma_load_3d(sb + i * BK * 128, &tB, &tailb[s], nb0 + i * 64, k0, 0);
            }
            continue;
          }
          const uint32_t fbar = mapa_shared(smem_u32(&full[s]), 0);
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * STAGE_BYTES);
          if (A_MN) {
            for (int i = 0; i < 2; ++i)
              tma_load_3d_pair(sa + i * BK * 128, &tA, fbar, m0 + i * 64, k0, 0);
          } else {
            tma_load_3d_pair(sa, &tA, fbar, k0, m0, 0);
          }
          const int eb = WG ? 0 : x.e;
          if (B_MN) {
            for (int i = 0; i < 2; ++i)
              tma_load_3d_pair(sb + i * BK * 128, &tB, fbar, nb0 + i * 64, k0, eb);
          } else {
            tma_load_3d_pair(sb, &tB, fbar, k0, nb0, eb);
          }
        }
      }
      stop = __shfl_sync(0xffffffffu, stop ? 1 : 0, 0) != 0;
    }
    // a wait that gave up leaves copies in flight that no MMA waits for: let
    // them land (bounded) before the CTAs exit
    if (stop && leader && lane == 0) {
      for (int k = kit > STAGES ? kit - STAGES : 0; k < kit; ++k)
        mbar_wait(&full[k % STAGES], (k / STAGES) & 1);
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------- MMA issuer (leader of the pair)
      const uint32_t idesc = instr_desc(1u, A_MN, B_MN, 256, BN);
      const uint32_t mn_lbo = BK * 128;
      int kit = 0, it = 0;  // stages and accumulator chunks so far
      bool stop = false;
      while (!stop && walk.next(x)) {
        if (lane == 0) {
          for (int c0 = 0; c0 < x.kb && !stop; c0 += F32 ? CHUNK_KB : x.kb, ++it) {
            const int c1 = F32 ? min(c0 + CHUNK_KB, x.kb) : x.kb;
            const int u = it & 1, use = it >> 1;
            if (use >= 1 && (*abort_flag || !mbar_wait(&acce[u], (use - 1) & 1, abort_flag))) {
              *abort_flag = 1;
              stop = true;
              break;
            }
            tc_fence_after();
            const uint32_t dacc = tmem + static_cast<uint32_t>(u * BN);
            for (int kb = c0; kb < c1; ++kb, ++kit) {
              const int s = kit % STAGES;
              if (*abort_flag || !mbar_wait(&full[s], (kit / STAGES) & 1, abort_flag)) {
                *abort_flag = 1;
                stop = true;
                break;
              }
              int steps = BK / 16;
              if (WG && x.tail != 0 && kb == x.kb - 1) {
                steps = (x.tail + 15) / 16;
                fence_cluster();  // the peer's half was cleared by its own warp
              }
              tc_fence_after();
              const uint32_t sa = smem_u32(smem + s * STAGE_BYTES), sb = sa + A_BYTES;
#pragma unroll
              for (int ks = 0; ks < BK / 16; ++ks) {
                if (WG && ks >= steps) break;
                const uint64_t ad = A_MN ? smem_desc(sa + ks * 16 * 128, mn_lbo, 1024u, 2u)
                                         : smem_desc(sa + ks * 32, 16, 1024u, 2u);
                const uint64_t bd = B_MN ? smem_desc(sb + ks * 16 * 128, mn_lbo, 1024u, 2u)
                                         : smem_desc(sb + ks * 32, 16, 1024u, 2u);
                mma_f16_pair(dacc, ad, bd, idesc, (kb > c0 || ks > 0) ? 1u : 0u);
              }
              mma_commit_pair(&empty[s], 3);
            }
            mma_commit_pair(&accf[u], 3);
          }
        }
        stop = __shfl_sync(0xffffffffu, stop ? 1 : 0, 0) != 0;
      }
      if (lane == 0) mma_commit_pair(drain, 3);  // after every MMA issued above
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
      const int row = row0 + lane;
      const bool whole = WG ? row0 < x.mend : row0 + 32 <= x.mend;  // a box store covers it
      const int64_t rbase = static_cast<int64_t>(row) * p.N;
      if (F32) {
        float acc[128];
#pragma unroll
        for (int j = 0; j < 128; ++j) acc[j] = 0.f;
        const int nc = (x.kb + CHUNK_KB - 1) / CHUNK_KB;
        for (int c = 0; c < nc; ++c, ++it) {
          const int u = it & 1;
          if (!warp_wait(&accf[u], (it >> 1) & 1, abort_flag)) {
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
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&acce[u]), 0));
        }
        if (stop) break;
        if (WG && p.accumulate && nc == 0) continue;  // an empty group leaves G as it is
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int cb = c0 + g * 32;
          if (cb < p.N) {
            if (whole) {
              if (lane == 0) bulk_wait_read_all();  // the previous store has read the box
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float4*>(box + sw128_off(lane, i)) =
                    make_float4(acc[g * 32 + 4 * i], acc[g * 32 + 4 * i + 1],
                                acc[g * 32 + 4 * i + 2], acc[g * 32 + 4 * i + 3]);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                if (WG && p.accumulate)
                  tma_reduce_add_3d(&tO, box, cb, row0, x.e);
                else
                  tma_store_3d(&tO, box, cb, row0, WG ? x.e : 0);
                bulk_commit();
              }
            } else if (!WG && row < x.mend) {
              float* o = static_cast<float*>(p.out) + rbase + cb;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (cb + 4 * i < p.N)
                  *reinterpret_cast<float4*>(o + 4 * i) =
                      make_float4(acc[g * 32 + 4 * i], acc[g * 32 + 4 * i + 1],
                                  acc[g * 32 + 4 * i + 2], acc[g * 32 + 4 * i + 3]);
            }
          }
        }
      } else {
        const int u = it & 1;
        if (!warp_wait(&accf[u], (it >> 1) & 1, abort_flag)) break;
        ++it;
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int cb = c0 + g * 64;
          uint32_t w[32];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float v[32];
            tmem_ld32(trow + static_cast<uint32_t>(u * BN + g * 64 + k * 32), v);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
              w[16 * k + j] = *reinterpret_cast<const uint32_t*>(&t);
            }
          }
          if (g == 1) {  // the accumulator is in registers: hand it back
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&acce[u]), 0));
          }
          if (cb < p.N) {
            if (whole) {
              if (lane == 0) bulk_wait_read_all();
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4*>(box + sw128_off(lane, i)) =
                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_3d(&tO, box, cb, row0, 0);
                bulk_commit();
              }
            } else if (row < x.mend) {
              __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + rbase + cb;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (cb + 8 * i < p.N)
                  *reinterpret_cast<uint4*>(o + 8 * i) =
                      make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();  // nothing outlives the CTA's shared memory
    __syncwarp();
  } else if (WG) {
    // ---------------- clearing warp: rows behind the group in its last stage
    int kit = 0;
    uint32_t par = 0;  // phase of each stage's tailb and clearb
    while (walk.next(x)) {
      kit += x.kb;
      if (x.tail == 0) continue;
      const int s = (kit - 1) % STAGES;
      if (!warp_wait(&tailb[s], (par >> s) & 1, abort_flag)) break;
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
        if (!warp_wait(&clearb[s], (par >> s) & 1, abort_flag)) break;
        fence_cluster();
        if (lane == 0) mbar_arrive(&full[s]);
      }
      par ^= 1u << s;
    }
  }

  if (warp == 1) mbar_wait(drain, 0);  // bounded; immediate unless a wait above gave up
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) tmem_dealloc_pair(tmem, 2 * BN);
}

template <bool WG, bool B_MN, bool F32>
cudaError_t launch_grouped(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o,
                           const GroupedParams& p, int64_t max_tiles, cudaStream_t st) {
  auto kern = k_grouped<WG, B_MN, F32>;
  static std::atomic<uint64_t> done{0};
  const LaunchInfo li = launch_info(reinterpret_cast<const void*>(kern), GSMEM, done);
  if (li.err != cudaSuccess) return li.err;
  int64_t ncl = li.sms / 2;
  if (ncl > max_tiles) ncl = max_tiles;
  if (ncl < 1) ncl = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * ncl), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = GSMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, b, o, p);
}

}  // namespace

cudaError_t grouped_rows(const void* X, const int64_t* offsets, const void* W, bool w_trans,
                         void* Y, int T, int K, int N, int groups, bool f32, cudaStream_t st) {
  CUtensorMap a, b, o;
  const int64_t kn = static_cast<int64_t>(K) * N;
  bool ok = tensor_map(&a, X, 2, K, T, 1, K, 0, BK, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  ok = ok && (w_trans ? tensor_map(&b, W, 2, K, N, groups, K, kn, BK, 128,
                                   CU_TENSOR_MAP_SWIZZLE_128B)
                      : tensor_map(&b, W, 2, N, K, groups, N, kn, 64, BK,
                                   CU_TENSOR_MAP_SWIZZLE_128B));
  ok = ok && tensor_map(&o, Y, f32 ? 4 : 2, N, T, 1, N, 0, f32 ? 32 : 64, 32,
                        CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return cudaErrorInvalidValue;
  GroupedParams p;
  memset(&p, 0, sizeof(p));
  p.g = Groups{offsets, groups, T};
  p.N = N;
  p.K = K;
  p.out = Y;
  // every group has at most one partial tile
  const int64_t tiles = (T / 256 + static_cast<int64_t>(groups < T ? groups : T)) * ((N + BN - 1) / BN);
  if (w_trans)
    return f32 ? launch_grouped<false, false, true>(a, b, o, p, tiles, st)
               : launch_grouped<false, false, false>(a, b, o, p, tiles, st);
  return f32 ? launch_grouped<false, true, true>(a, b, o, p, tiles, st)
             : launch_grouped<false, true, false>(a, b, o, p, tiles, st);
}

cudaError_t grouped_wgrad(const void* A, const void* B, const int64_t* offsets, float* G, int T,
                          int M, int N, int groups, bool accumulate, cudaStream_t st) {
  CUtensorMap a, b, o;
  bool ok = true;
  if (T > 0) {
    ok = tensor_map(&a, A, 2, M, T, 1, M, 0, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B) &&
         tensor_map(&b, B, 2, N, T, 1, N, 0, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  ok = ok && tensor_map(&o, G, 4, N, M, groups, N, static_cast<int64_t>(M) * N, 32, 32,
                        CU_TENSOR_MAP_SWIZZLE_128B);
  if (!ok) return cudaErrorInvalidValue;
  if (T == 0) a = b = o;  // no group has a row: never loaded from
  GroupedParams p;
  memset(&p, 0, sizeof(p));
  p.g = Groups{offsets, groups, T};
  p.M = M;
  p.N = N;
  p.out = G;
  p.accumulate = accumulate ? 1 : 0;
  const int64_t tiles = static_cast<int64_t>(groups) * ((M + 255) / 256) * ((N + BN - 1) / BN);
  return launch_grouped<true, true, true>(a, b, o, p, tiles, st);
}

uint64_t kernel_runs_grouped() {
  unsigned long long v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kernel_runs, sizeof(v)) != cudaSuccess) return 0;
  return v;
}

}  // namespace shp
