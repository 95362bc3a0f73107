// Microscaled 4-bit floating point (MXFP4): quantisation, its inverse and the
// product of two quantised operands on the sm_100a tensor cores.
//
// Format (OCP Microscaling Formats v1.0): a block of 32 values x_i shares the
// scale 2^e, e = floor(log2 max|x_i|) - 2, kept as the byte e + 127; a value
// is a 4-bit float (sign, 2 exponent bits, 1 mantissa bit: 0, .5, 1, 1.5, 2,
// 3, 4, 6) of x_i / 2^e, rounded to nearest with ties to even and saturated
// at 6 (so that max|x| in (7, 8) 2^e is clipped by up to a quarter).
//
// Layout: a matrix of R rows and C columns has rows of Cp / 2 bytes, Cp = C
// rounded up to whole blocks, element 2j in the low nibble of byte j, zero
// codes behind C.  Its scales come in tiles of 128 rows x 4 blocks, 512 bytes,
// tile (i, j) at (i * ceil(Cp / 128) + j) * 512, row r and block k of a tile at
// byte (r % 32) * 16 + (r / 32) * 4 + k: the order in which one
// tcgen05.cp.32x128b brings a tile's scales into tensor memory.  Scales of
// rows and blocks outside the matrix are zero bytes.
#include <cuda_bf16.h>
#include <string.h>

#include "internal.h"
#include "shp_common.cuh"

namespace shp {

namespace {

// ------------------------------------------------------------ quantisation

constexpr int QT = 128;       // rows and columns of a quantiser tile
constexpr int QLD = QT + 4;   // floats per tile row in shared memory (see k_mx4_quantize)
constexpr int QSMEM = QT * QLD * 4;

// Codes of eight values, the first in the lowest nibble.
SHP_DEV uint32_t e2m1x8(const float* y) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// One block of 32 values: its scale byte, and its codes in q[0..3].  The scale
// is a power of two, so dividing by it is exact (a quotient small enough to
// underflow rounds to the zero code either way).  The largest magnitude is
// compared as bits: a block that holds a NaN or an Inf gets the NaN scale and
// zero codes.
SHP_DEV uint32_t quantize_block(float* x, uint32_t* q) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  if (top >= 0x7f800000u) {
    q[0] = q[1] = q[2] = q[3] = 0;
    return 255u;
  }
  // floor(log2) is the exponent field - 127 (below it the scale is 2^-127)
  const int sb = max(static_cast<int>(top >> 23) - 2, 0);
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - sb) << 23);  // 2^(127 - sb)
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] *= inv;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = e2m1x8(x + 8 * i);
  return static_cast<uint32_t>(sb);
}

// One orientation's outputs: codes of `lines` lines (rows, or columns of X)
// of `len` values, and their scale tiles.
struct Mx4Out {
  uint8_t* q;
  uint8_t* s;
};

// A CTA quantises one 128 x 128 tile of X, read once (16-byte loads, a warp
// per row), along either axis or both.  The tile is kept as fp32 in shared
// memory with rows of 132 floats: threads that own a row read it 16 bytes at
// a time and threads that own a column 4 bytes at a time, both without bank
// conflicts.  A thread quantises two neighbouring blocks of a line, so its
// codes are 32 contiguous bytes, and the tile's scales leave as one 512-byte
// run.
template <bool BF16>
__global__ void __launch_bounds__(256)
    k_mx4_quantize(const void* X, int rows, int cols, int tiles_r, int tiles_c, Mx4Out orow,
                   Mx4Out ocol) {
  count_kernel_run();
  extern __shared__ __align__(16) float xs[];
  __shared__ uint32_t sc[2][128];
  const int64_t t = blockIdx.x;
  const int tc = static_cast<int>(t % tiles_c);
  const int tr = static_cast<int>(t / tiles_c % tiles_r);
  const int64_t b = t / tiles_c / tiles_r;
  const int r0 = tr * QT, c0 = tc * QT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t base = b * rows * static_cast<int64_t>(cols) + c0 + 4 * lane;
  const bool cin = c0 + 4 * lane < cols;  // cols is a multiple of 4
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + warp + 8 * (8 * half + i);
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (cin && r < rows) {
        const int64_t at = base + r * static_cast<int64_t>(cols);
        if (BF16) {
          const uint2 u = __ldg(reinterpret_cast<const uint2*>(
              static_cast<const __nv_bfloat16*>(X) + at));
          v[i] = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                             __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
        } else {
          v[i] = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(X) + at));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float4*>(xs + (warp + 8 * (8 * half + i)) * QLD + 4 * lane) = v[i];
  }
  __syncthreads();
  const int line = threadIdx.x & 127, h = threadIdx.x >> 7;  // blocks 2h, 2h + 1 of a line
#pragma unroll 1
  for (int o = 0; o < 2; ++o) {
    const Mx4Out out = o == 0 ? orow : ocol;
    if (out.q == nullptr) continue;
    const int lines = o == 0 ? rows : cols, len = o == 0 ? cols : rows;
    const int l0 = o == 0 ? r0 : c0, p0 = o == 0 ? c0 : r0;
    const int blocks = (len + 31) / 32;
    const int tl = o == 0 ? tr : tc, tp = o == 0 ? tc : tr;
    const int tiles_l = o == 0 ? tiles_r : tiles_c, tiles_p = o == 0 ? tiles_c : tiles_r;
    uint32_t bytes = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float x[32];
      const int p = 64 * h + 32 * k;
      if (o == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(xs + line * QLD + p + 4 * i);
          x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = xs[(p + i) * QLD + line];
      }
      uint32_t q[4];
      bytes |= quantize_block(x, q) << (8 * k);
      if (l0 + line < lines && (p0 + p) / 32 < blocks)
        *reinterpret_cast<uint4*>(out.q + ((b * lines + l0 + line) * blocks + (p0 + p) / 32) * 16) =
            make_uint4(q[0], q[1], q[2], q[3]);
    }
    // word (r % 32) * 4 + r / 32 of the tile holds a line's four scale bytes
    if (h == 1) sc[0][(line & 31) * 4 + (line >> 5)] = bytes << 16;
    __syncthreads();
    if (h == 0) sc[1][(line & 31) * 4 + (line >> 5)] = sc[0][(line & 31) * 4 + (line >> 5)] | bytes;
    __syncthreads();
    if (h == 0)
      reinterpret_cast<uint32_t*>(out.s)[((b * tiles_l + tl) * tiles_p + tp) * 128 + line] =
          sc[1][line];
    __syncthreads();
  }
}

// Eight values per thread: a coalesced 4-byte read of codes, 16 or 32 bytes
// written.  Values are exact in either type (one mantissa bit, and exponents
// down to 2^-128).
template <bool BF16>
__global__ void __launch_bounds__(256)
    k_mx4_dequantize(const uint8_t* Q, const uint8_t* S, int rows, int cols, int64_t batch,
                     void* X) {
  count_kernel_run();
  const int groups = (cols + 7) / 8, blocks = (cols + 31) / 32;
  const int tiles_r = (rows + 127) / 128, tiles_c = (blocks + 3) / 4;
  const int64_t n = batch * rows * groups;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int g = static_cast<int>(i % groups);
    const int64_t br = i / groups;
    const int r = static_cast<int>(br % rows);
    const int64_t b = br / rows;
    const uint32_t codes =
        __ldg(reinterpret_cast<const uint32_t*>(Q + br * blocks * 16 + g * 4));
    const int k = g / 4;
    const uint32_t sb = __ldg(S + (((b * tiles_r + r / 128) * tiles_c + k / 4) * 512 +
                                   (r % 32) * 16 + (r % 128) / 32 * 4 + k % 4));
    const float scale = sb == 0 ? __uint_as_float(0x00400000u)
                                : __uint_as_float(sb == 255 ? 0x7fc00000u : sb << 23);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t c = codes >> (4 * j);
      // exponent field 0: 0 or .5; otherwise (1 + m / 2) 2^(e - 1)
      const uint32_t m = c & 7u;
      const float a = m < 2 ? 0.5f * static_cast<float>(m)
                            : __uint_as_float((((m >> 1) + 126u) << 23) | ((m & 1u) << 22));
      v[j] = ((c & 8u) ? -a : a) * scale;
    }
    const int64_t at = br * cols + g * 8;
    if (BF16) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&p);
      }
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(X) + at;
      if (cols % 8 == 0) {
        *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        for (int j = 0; j < 8 && g * 8 + j < cols; ++j) o[j] = __float2bfloat16_rn(v[j]);
      }
    } else {
      float* o = static_cast<float*>(X) + at;
      if (cols % 4 == 0) {
        *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
        if (g * 8 + 4 < cols) *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        for (int j = 0; j < 8 && g * 8 + j < cols; ++j) o[j] = v[j];
      }
    }
  }
}

// ----------------------------------------------------------------- product
//
// C[b] = A[b] B[b]^T (A: M x K, B: N x K, both quantised along K).
// k_mx4_gemm is a persistent CTA-pair kernel: one block-scaled tcgen05.mma
// (kind::mxf4, K = 64, M = 256 over two SMs, N = 256) per 64 columns of K;
// the tensor core multiplies each block's sum by both scales.  A stage is 256
// columns: 128-byte rows of codes (128 of A and 128 of B per CTA) and the
// scale tiles of this CTA's 128 rows of A and of all 256 rows of B, which
// tcgen05.cp moves into tensor memory in front of the stage's MMAs.
//
// Tensor memory (512 columns): two 256-column accumulators at 0 and 192 and
// two stages of scales behind them at 448.  The accumulators share 64 columns:
// the epilogue drains those first and hands them back, so the next tile's
// MMAs run beside the rest of this tile's epilogue.
//
// fp32 results are summed in chunks of CHUNK_KB stages (32 MMAs) in the tensor
// core, which adds with truncation, and over chunks in registers.

constexpr int BN = 256;
constexpr int MK = 256;            // codes per stage row: 128 bytes
constexpr int TILE_BYTES = 128 * 128;
constexpr int SF_BYTES = 3 * 1024;  // 2 tiles of A's rows, 2 x 2 of B's
constexpr int STAGE_BYTES = 2 * TILE_BYTES + SF_BYTES;
constexpr int STAGES = 5;
constexpr int CHUNK_KB = 8;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (2 + EPI_WARPS);
constexpr int EPI_BOX = 4096;
constexpr int GSMEM = 1024 + STAGES * STAGE_BYTES + EPI_WARPS * EPI_BOX + 256;
constexpr int ACC1 = 192;    // second accumulator's first column
constexpr int SF_COL = 448;  // scales: per stage 8 columns of A, 16 of B
static_assert(STAGE_BYTES % 1024 == 0, "swizzled tiles start on 1024-byte boundaries");
static_assert(GSMEM <= 232448, "product kernel exceeds shared memory");
static_assert(ACC1 + BN == SF_COL && SF_COL + 2 * 24 <= 512, "tensor memory");

// One scale tile (32 rows of 16 bytes) to four columns of tensor memory,
// repeated in all four lane quarters, in both CTAs of the pair (each from its
// own shared memory).
SHP_DEV void tmem_cp_scales_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc)
               : "memory");
}

SHP_DEV void mma_mxf4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                           uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X"
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
}

// Instruction descriptor of the block-scaled kinds: E2M1 operands (format 1),
// E8M0 scales; `sf` (0 or 2) picks the two bytes of a scale column that this
// MMA's two blocks use, for both operands.
__host__ __device__ constexpr uint32_t instr_desc_mxf4(int M, int N, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(M >> 4) << 24) | (sf << 29);
}

struct Mx4Params {
  int M, N, K;
  int tiles_m, tiles_n;
  int64_t batch;
  int rb_a, rb_b;  // 128-row scale tiles per matrix of A and B
  void* out;
};

template <bool F32>
__global__ void __launch_bounds__(THREADS, 1)
    k_mx4_gemm(const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tAs,
               const __grid_constant__ CUtensorMap tB, const __grid_constant__ CUtensorMap tBs,
               const __grid_constant__ CUtensorMap tO, Mx4Params p) {
  count_kernel_run();
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int ncl = static_cast<int>(gridDim.x) / 2, cl = static_cast<int>(blockIdx.x) / 2;
  const int per_b = p.tiles_m * p.tiles_n;
  const int ntiles = static_cast<int>(per_b * p.batch);
  const int KB = (p.K + MK - 1) / MK;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* boxes = smem + STAGES * STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(boxes + EPI_WARPS * EPI_BOX);
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;  // accumulator u complete
  uint64_t* acce = accf + 2;        // shared columns drained, and all of the accumulator before
  uint64_t* drain = acce + 1;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1) + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&accf[0], 1);
    mbar_init(&accf[1], 1);
    mbar_init(acce, 2 * EPI_WARPS);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tA);
    tma_prefetch_desc(&tAs);
    tma_prefetch_desc(&tB);
    tma_prefetch_desc(&tBs);
    tma_prefetch_desc(&tO);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // peer barriers initialised, both TMEM allocations done
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (both CTAs)
      int kit = 0;
      bool stop = false;
      for (int t = cl; t < ntiles && !stop; t += ncl) {
        const int b = t / per_b, r = t % per_b;
        const int tm = r / p.tiles_n, tn = r % p.tiles_n;
        const int m0 = tm * 256 + static_cast<int>(rank) * 128;
        const int nb0 = tn * BN + static_cast<int>(rank) * 128;
        const int za = b * p.rb_a + tm * 2 + static_cast<int>(rank);
        const int zb = b * p.rb_b + tn * 2;
        for (int kb = 0; kb < KB; ++kb, ++kit) {
          const int s = kit % STAGES;
          if (kit >= STAGES &&
              (*abort_flag || !mbar_wait(&empty[s], ((kit / STAGES) - 1) & 1, abort_flag))) {
            *abort_flag = 1;
            stop = true;
            break;
          }
          uint8_t* sa = smem + s * STAGE_BYTES;
          uint8_t* sf = sa + 2 * TILE_BYTES;
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * STAGE_BYTES);
          const uint32_t fbar = mapa_shared(smem_u32(&full[s]), 0);
          tma_load_3d_pair(sa, &tA, fbar, kb * 64, m0, b);  // codes move as 16-bit units
          tma_load_3d_pair(sa + TILE_BYTES, &tB, fbar, kb * 64, nb0, b);
          tma_load_3d_pair(sf, &tAs, fbar, 0, kb * 2, za);
          tma_load_3d_pair(sf + 1024, &tBs, fbar, 0, kb * 2, zb);
          tma_load_3d_pair(sf + 2048, &tBs, fbar, 0, kb * 2, zb + 1);
        }
      }
      // a wait that gave up leaves copies in flight that no MMA waits for: let
      // them land (bounded) before the CTAs exit
      if (stop && leader) {
        for (int k = kit > STAGES ? kit - STAGES : 0; k < kit; ++k)
          mbar_wait(&full[k % STAGES], (k / STAGES) & 1);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------- MMA issuer (leader of the pair)
      int kit = 0, it = 0;
      bool stop = false;
      for (int t = cl; t < ntiles && !stop; t += ncl) {
        for (int c0 = 0; c0 < KB && !stop; c0 += F32 ? CHUNK_KB : KB, ++it) {
          const int c1 = F32 ? min(c0 + CHUNK_KB, KB) : KB;
          const int u = it & 1;
          if (it >= 1 && (*abort_flag || !mbar_wait(acce, (it - 1) & 1, abort_flag))) {
            *abort_flag = 1;
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t dacc = tmem + static_cast<uint32_t>(u * ACC1);
          for (int kb = c0; kb < c1; ++kb, ++kit) {
            const int s = kit % STAGES;
            if (*abort_flag || !mbar_wait(&full[s], (kit / STAGES) & 1, abort_flag)) {
              *abort_flag = 1;
              stop = true;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + s * STAGE_BYTES), sb = sa + TILE_BYTES;
            const uint32_t sf = sb + TILE_BYTES;
            const uint32_t tsa = tmem + static_cast<uint32_t>(SF_COL + (kit & 1) * 24);
            const uint32_t tsb = tsa + 8;
            const int left = p.K - kb * MK;  // columns of this stage inside the matrix
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if (k * 128 >= left) break;
              tmem_cp_scales_pair(tsa + k * 4, smem_desc(sf + k * 512, 128, 128, 0));
              tmem_cp_scales_pair(tsb + k * 8, smem_desc(sf + 1024 + k * 512, 128, 128, 0));
              tmem_cp_scales_pair(tsb + k * 8 + 4, smem_desc(sf + 2048 + k * 512, 128, 128, 0));
            }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              if (ks * 64 >= left) break;
              mma_mxf4_pair(dacc, smem_desc(sa + ks * 32, 16, 1024u, 2u),
                            smem_desc(sb + ks * 32, 16, 1024u, 2u),
                            instr_desc_mxf4(256, BN, (ks & 1) * 2), tsa + (ks >> 1) * 4,
                            tsb + (ks >> 1) * 8, (kb > c0 || ks > 0) ? 1u : 0u);
            }
            mma_commit_pair(&empty[s], 3);
          }
          mma_commit_pair(&accf[u], 3);
        }
      }
      mma_commit_pair(drain, 3);  // after every MMA issued above
    }
  } else {
    // ---------------- epilogue warps 2..9 (both CTAs, each on its TMEM rows)
    const int q = warp & 3, h = (warp - 2) >> 2;
    uint8_t* box = boxes + (warp - 2) * EPI_BOX;
    const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16);
    int it = 0;
    bool stop = false;
    for (int t = cl; t < ntiles && !stop; t += ncl) {
      const int b = t / per_b, r = t % per_b;
      const int row0 = r / p.tiles_n * 256 + static_cast<int>(rank) * 128 + q * 32;
      // warp half h owns columns 128h .. 128h + 127 and reads its two 64-column
      // parts in the order that drains the shared columns first: they are the
      // upper part of half 1 in accumulator 0, the lower part of half 0 in 1
      const int n0 = r % p.tiles_n * BN + h * 128;
      if (F32) {
        float acc[128];
#pragma unroll
        for (int j = 0; j < 128; ++j) acc[j] = 0.f;
        for (int c0 = 0; c0 < KB; c0 += CHUNK_KB, ++it) {
          const int u = it & 1;
          if (!warp_wait(&accf[u], (it >> 1) & 1, abort_flag)) {
            stop = true;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float v[32];
            tmem_ld32(trow + static_cast<uint32_t>(u * ACC1 + h * 128 + (g ^ (2 * h)) * 32), v);
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[g * 32 + j] += v[j];
            if (g == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(acce), 0));
            }
          }
        }
        if (stop) break;
        if (row0 < p.M) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int cb = n0 + (g ^ (2 * h)) * 32;
            if (cb >= p.N) continue;
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
              tma_store_3d(&tO, box, cb, row0, b);
              bulk_commit();
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
          const int part = (g ^ h) * 64;
          uint32_t w[32];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float v[32];
            tmem_ld32(trow + static_cast<uint32_t>(u * ACC1 + h * 128 + part + k * 32), v);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
              w[16 * k + j] = *reinterpret_cast<const uint32_t*>(&x);
            }
          }
          if (g == 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(acce), 0));
          }
          if (row0 < p.M && n0 + part < p.N) {
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(box + sw128_off(lane, i)) =
                  make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&tO, box, n0 + part, row0, b);
              bulk_commit();
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();  // nothing outlives the CTA's shared memory
    __syncwarp();
  }

  if (warp == 1) mbar_wait(drain, 0);  // bounded; immediate unless a wait above gave up
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

cudaError_t mx4_quantize(const void* X, bool bf16, int rows, int cols, int64_t batch, uint8_t* Q,
                         uint8_t* S, uint8_t* Qt, uint8_t* St, cudaStream_t st) {
  const int tr = static_cast<int>(ceil_div(rows, QT)), tc = static_cast<int>(ceil_div(cols, QT));
  const int64_t tiles = batch * tr * tc;
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  auto kern = bf16 ? k_mx4_quantize<true> : k_mx4_quantize<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, QSMEM);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(tiles), 256, QSMEM, st>>>(X, rows, cols, tr, tc, Mx4Out{Q, S},
                                                         Mx4Out{Qt, St});
  return cudaGetLastError();
}

cudaError_t mx4_dequantize(const uint8_t* Q, const uint8_t* S, int rows, int cols, int64_t batch,
                           void* X, bool bf16, cudaStream_t st) {
  const int64_t n = batch * rows * ceil_div(cols, 8);
  int64_t blocks = ceil_div(n, 256);
  if (blocks > 148 * 64) blocks = 148 * 64;  // grid-stride: many waves per SM
  if (bf16)
    k_mx4_dequantize<true><<<static_cast<unsigned>(blocks), 256, 0, st>>>(Q, S, rows, cols, batch, X);
  else
    k_mx4_dequantize<false><<<static_cast<unsigned>(blocks), 256, 0, st>>>(Q, S, rows, cols, batch, X);
  return cudaGetLastError();
}

cudaError_t mx4_gemm(const uint8_t* A, const uint8_t* As, const uint8_t* B, const uint8_t* Bs,
                     void* C, bool f32, int M, int N, int K, int64_t batch, cudaStream_t st) {
  Mx4Params p;
  memset(&p, 0, sizeof(p));
  p.M = M;
  p.N = N;
  p.K = K;
  p.batch = batch;
  p.tiles_m = static_cast<int>(ceil_div(M, 256));
  p.tiles_n = static_cast<int>(ceil_div(N, BN));
  p.rb_a = static_cast<int>(ceil_div(M, 128));
  p.rb_b = static_cast<int>(ceil_div(N, 128));
  p.out = C;
  const int kt = static_cast<int>(ceil_div(K, 128));
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n * batch;
  if (tiles > INT32_MAX / 2 || batch * p.rb_a > INT32_MAX || batch * p.rb_b > INT32_MAX)
    return cudaErrorInvalidValue;
  CUtensorMap a, as, b, bs, o;
  const int64_t u = K / 4;  // 16-bit units per row of codes
  if (!tensor_map(&a, A, 2, u, M, batch, u, u * M, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tensor_map(&b, B, 2, u, N, batch, u, u * N, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tensor_map(&as, As, 4, 128, kt, batch * p.rb_a, 128, 128 * kt, 128, 2,
                  CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !tensor_map(&bs, Bs, 4, 128, kt, batch * p.rb_b, 128, 128 * kt, 128, 2,
                  CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !tensor_map(&o, C, f32 ? 4 : 2, N, M, batch, N, static_cast<int64_t>(M) * N, f32 ? 32 : 64, 32,
                  CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto kern = f32 ? k_mx4_gemm<true> : k_mx4_gemm<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GSMEM);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int64_t ncl = sms / 2;
  if (ncl > tiles) ncl = tiles;
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
  return cudaLaunchKernelEx(&cfg, kern, a, as, b, bs, o, p);
}

uint64_t kernel_runs_mx4() {
  unsigned long long v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kernel_runs, sizeof(v)) != cudaSuccess) return 0;
  return v;
}

}  // namespace shp
