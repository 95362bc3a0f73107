// Microscaled 4-bit floating point (MXFP4): quantisation, its inverse and the
// product of two quantised operands on the sm_100a tensor cores.
//
// Format (OCP Microscaling Formats v1.0): a block of 32 values x_i shares the
// scale 2^e, e = floor(log2 max|x_i|) - 2, kept as the byte e + 127; a value
// is a 4-bit float (sign, 2 exponent bits, 1 mantissa bit: 0, .5, 1, 1.5, 2,
// 3, 4, 6) of x_i / 2^e, rounded to nearest with ties to even and saturated
// at 6 (magnitudes in (6, 8) 2^e come out as 6 2^e).
//
// Layout: a matrix of R rows and C columns has rows of Cp / 2 bytes, Cp = C
// rounded up to whole blocks, element 2j in the low nibble of byte j, zero
// codes behind C.  Its scales come in tiles of 128 rows x 4 blocks, 512 bytes,
// tile (i, j) at (i * ceil(Cp / 128) + j) * 512, row r and block k of a tile at
// byte (r % 32) * 16 + (r / 32) * 4 + k: the order in which one
// tcgen05.cp.32x128b brings a tile's scales into tensor memory.  Scales of
// rows and blocks outside the matrix are zero bytes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <string.h>

#include "internal.h"
#include "shp_common.cuh"

namespace shp {

namespace {

// ------------------------------------------------------------ quantisation

constexpr int QT = 128;  // rows and columns of a quantiser tile

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

// k_mx4_quantize reads X once, in 128 x 128 tiles, along either axis or both.
// It moves bytes and computes little, so one persistent CTA per SM keeps
// several tiles in flight: warp 16 brings them by TMA (zero fill outside X)
// into a ring, 16 warps quantise, a block of 32 values per thread and
// orientation, and the codes and the 512 scale bytes of a tile leave as bulk
// stores (which clip the edge).  The tile stays in X's type, in boxes of
// 128-byte rows with the 128-byte swizzle: a warp whose lanes own 32 rows
// (16-byte reads) and one whose lanes own 32 columns both read it without bank
// conflicts, so one copy serves both orientations.  Bound by HBM: 16 x 4096 x
// 1024 fp32 along both axes 60 us = 5.65 TB/s, along one 53 us = 5.76.
constexpr int QTHREADS = 512;
constexpr int QSTG = 2 * 8192 + 2 * 512;  // codes and scales of both orientations

template <bool BF16>
struct QCfg {
  static constexpr int TILE = QT * QT * (BF16 ? 2 : 4);
  static constexpr int STAGES = BF16 ? 5 : 3;
  static constexpr int SMEM = 1024 + STAGES * TILE + QSTG + 128;
};

struct QParams {
  int tiles_r, tiles_c;
  int64_t tiles;
  uint8_t* s[2];  // scale tiles per orientation (null: not wanted)
  SelfTest test;
};

SHP_DEV void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
SHP_DEV void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(QTHREADS) : "memory"); }

template <bool BF16>
__global__ void __launch_bounds__(QTHREADS + 32, 1)
    k_mx4_quantize(const __grid_constant__ CUtensorMap tX, const __grid_constant__ CUtensorMap tQ,
                   const __grid_constant__ CUtensorMap tQt, QParams p) {
  count_kernel_run();
  using C = QCfg<BF16>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* stg = smem + C::STAGES * C::TILE;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg + QSTG);
  uint64_t* empty = full + C::STAGES;
  uint64_t* never = empty + C::STAGES;  // completed by nothing: the self-test's wait
  volatile int* abort_flag = reinterpret_cast<volatile int*>(never + 1);
  if (threadIdx.x == 0) {
    mbar_init(never, 1);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], QTHREADS / 32);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t per_b = static_cast<int64_t>(p.tiles_r) * p.tiles_c;
  const long long limit = p.test.limit > 0 ? p.test.limit : SHP_SPIN_LIMIT;
  if (warp == QTHREADS / 32) {
    if (lane == 0) {
      tma_prefetch_desc(&tX);
      int it = 0;
      for (int64_t t = blockIdx.x; t < p.tiles; t += gridDim.x, ++it) {
        const int s = it % C::STAGES;
        if (it >= C::STAGES && !mbar_wait(&empty[s], ((it / C::STAGES) - 1) & 1, nullptr, limit))
          break;
        const int b = static_cast<int>(t / per_b), r = static_cast<int>(t % per_b);
        const int c0 = r % p.tiles_c * QT, r0 = r / p.tiles_c * QT;
        mbar_arrive_expect_tx(&full[s], C::TILE);
        constexpr int W = BF16 ? 64 : 32;  // columns per box
        for (int i = 0; i < QT / W; ++i)
          tma_load_3d(smem + s * C::TILE + i * QT * 128, &tX, &full[s], c0 + i * W, r0, b);
      }
      // no copy may be in flight when the CTA exits, also where the consumers
      // gave up and do not wait for it
      for (int i = it > C::STAGES ? it - C::STAGES : 0; i < it; ++i)
        mbar_wait(&full[i % C::STAGES], (i / C::STAGES) & 1, nullptr, limit);
    }
    return;
  }
  const int line = threadIdx.x & 127, k = threadIdx.x >> 7;  // block k of a row, or column, `line`
  int it = 0;
  for (int64_t t = blockIdx.x; t < p.tiles; t += gridDim.x, ++it) {
    const int s = it % C::STAGES;
    const uint8_t* tile = smem + s * C::TILE;
    // a wait that gives up is acted on behind the barrier below, by all warps
    // together (only consumers set the flag)
    if (it == 0) selftest_wait(p.test.stall, never, abort_flag);
    if (!mbar_wait(&full[s], (it / C::STAGES) & 1, nullptr, limit)) *abort_flag = 1;
    uint32_t q[2][4], sb[2];
    if (p.s[0] != nullptr) {
      float x[32];
      if (BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 u = *reinterpret_cast<const uint4*>(
              tile + (k >> 1) * QT * 128 + sw128_off(line, (k & 1) * 4 + i));
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 v =
              *reinterpret_cast<const float4*>(tile + k * QT * 128 + sw128_off(line, i));
          x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
        }
      }
      sb[0] = quantize_block(x, q[0]);
    }
    if (p.s[1] != nullptr) {
      float x[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int r = 32 * k + i;  // r & 7 == i & 7
        if (BF16)
          x[i] = __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(
                     tile + (line >> 6) * QT * 128 + sw128_off(r, (line & 63) >> 3) +
                     (line & 7) * 2)) << 16);
        else
          x[i] = *reinterpret_cast<const float*>(tile + (line >> 5) * QT * 128 +
                                                 sw128_off(r, (line & 31) >> 2) + (line & 3) * 4);
      }
      sb[1] = quantize_block(x, q[1]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    if (threadIdx.x == 0) bulk_wait_read_all();  // the last tile's stores have read the staging
    consumers_sync();
    if (*abort_flag) break;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      if (p.s[o] == nullptr) continue;
      *reinterpret_cast<uint4*>(stg + o * 8192 + line * 64 + ((k ^ ((line >> 1) & 3)) << 4)) =
          make_uint4(q[o][0], q[o][1], q[o][2], q[o][3]);
      stg[2 * 8192 + o * 512 + (line & 31) * 16 + (line >> 5) * 4 + k] =
          static_cast<uint8_t>(sb[o]);
    }
    fence_proxy_async_smem();
    consumers_sync();
    if (threadIdx.x == 0) {
      const int b = static_cast<int>(t / per_b), r = static_cast<int>(t % per_b);
      const int tc = r % p.tiles_c, tr = r / p.tiles_c;
      if (p.s[0] != nullptr) {
        tma_store_3d(&tQ, stg, tc * 32, tr * QT, b);
        bulk_store(p.s[0] + t * 512, stg + 2 * 8192, 512);
      }
      if (p.s[1] != nullptr) {
        tma_store_3d(&tQt, stg + 8192, tr * 32, tc * QT, b);
        bulk_store(p.s[1] + (b * per_b + static_cast<int64_t>(tc) * p.tiles_r + tr) * 512,
                   stg + 2 * 8192 + 512, 512);
      }
      bulk_commit();
    }
  }
  if (threadIdx.x == 0) bulk_wait_all();
  selftest_report(p.test.status, abort_flag);
}

// Two codes (one byte of `w`) as fp32.
SHP_DEV void e2m1x2(uint32_t w, float& a, float& b) {
  uint32_t h;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
      : "=r"(h)
      : "r"(w));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  a = f.x;
  b = f.y;
}

// A CTA restores one 128 x 128 tile; a warp's store is one (fp32: 4 values per
// lane) or two (bf16: 8 values per lane) contiguous row segments, and each
// lane has eight loads of codes in flight.  Values are exact in either type
// (one mantissa bit, exponents down to 2^-128).  Bound by HBM: 16 x 4096 x 1024 to
// fp32 54 us = 5.6 TB/s.
template <bool BF16>
__global__ void __launch_bounds__(256)
    k_mx4_dequantize(const uint8_t* Q, const uint8_t* S, int rows, int cols, int tiles_r,
                     int tiles_c, void* X) {
  count_kernel_run();
  constexpr int V = BF16 ? 8 : 4;         // values per lane
  constexpr int RW = V * 32 / QT;         // rows per warp access
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tc = static_cast<int>(blockIdx.x % tiles_c);
  const int64_t br = blockIdx.x / tiles_c;
  const int tr = static_cast<int>(br % tiles_r);
  const int64_t b = br / tiles_r;
  const int blocks = (cols + 31) / 32;
  const int c = tc * QT + (lane * V) % QT;  // first column of this lane
  if (c >= cols) return;
  const uint8_t* tile = S + static_cast<int64_t>(blockIdx.x) * 512 + (c % QT) / 32;
  const int64_t first = b * rows + tr * QT;
  const uint8_t* q = Q + first * blocks * 16 + c / 2;
  const int n = rows - tr * QT < QT ? rows - tr * QT : QT;
  const bool wide = cols % V == 0;  // whole, aligned groups
#pragma unroll
  for (int half = 0; half < 2 / RW; ++half) {
    uint32_t code[8], sb[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = (8 * (8 * half + i) + warp) * RW + lane * V / QT;
      code[i] = sb[i] = 0;
      if (r < n) {
        const uint8_t* at = q + static_cast<int64_t>(r) * blocks * 16;
        code[i] = BF16 ? __ldg(reinterpret_cast<const uint32_t*>(at))
                       : __ldg(reinterpret_cast<const uint16_t*>(at));
        sb[i] = __ldg(tile + (r & 31) * 16 + (r >> 5) * 4);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = (8 * (8 * half + i) + warp) * RW + lane * V / QT;
      if (r >= n) continue;
      const float scale = __uint_as_float(sb[i] == 0 ? 0x00400000u
                                                     : (sb[i] == 255 ? 0x7fc00000u : sb[i] << 23));
      float v[V];
#pragma unroll
      for (int j = 0; j < V / 2; ++j) e2m1x2(code[i] >> (8 * j), v[2 * j], v[2 * j + 1]);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] *= scale;
      const int64_t at = (first + r) * cols + c;
      if (BF16) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(X) + at;
        if (wide) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * j], v[(2 * j + 1) % V]);
            w[j] = *reinterpret_cast<const uint32_t*>(&x);
          }
          *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (c + j < cols) o[j] = __float2bfloat16_rn(v[j]);
        }
      } else {
        float* o = static_cast<float*>(X) + at;
        if (wide) {
          *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (c + j < cols) o[j] = v[j];
        }
      }
    }
  }
}

// ----------------------------------------------------------------- product
//
// C[b] = A[b] B[b]^T (A: M x K, B: N x K, both quantised along K).
// k_mx4_gemm is a persistent CTA-pair kernel: one block-scaled tcgen05.mma
// (kind::mxf4, K = 64, M = 256 over two SMs, N = NB = 256 or 128) per 64 columns
// of K; the tensor core multiplies each block's sum by both scales.  A stage is
// 256 columns: 128-byte rows of codes (128 of A and NB / 2 of B per CTA) and the
// scale tiles of this CTA's 128 rows of A and of all NB rows of B, which
// tcgen05.cp moves into tensor memory in front of the stage's MMAs.
//
// Tensor memory (512 columns): two accumulators at 0 and 192 and two stages of
// scales behind them at 448.  Accumulators of 256 columns share 64: the epilogue
// drains those first and hands them back, so the next tile's MMAs run beside the
// rest of this tile's epilogue.
//
// The issuing warp needs ten or so instructions per stage beside its waits, so
// where a stage's MMAs are short it sets the rate: it asks whether the next stage
// is full while it still issues this one (NB = 128: 203 -> 173 ns per stage).
//
// fp32 results are summed in chunks of CHUNK_KB stages (32 MMAs) in the tensor
// core, which adds with truncation, and over chunks in registers; bf16 results in
// chunks of LONG_KB stages (256 MMAs: a bias of at most 2^-16 of a sum of one sign,
// however long the contraction), which is the whole sum, stored as it leaves the
// accumulator, where K is no longer.
//
// Bound and rate: a stage of NB = 256 brings 35 KB into each SM for 512 clocks of
// MMAs, 68 bytes per clock, about what the path from L2 delivers: 8192 x 8192 x
// 4096 95 to 98 us = 5.6 to 5.8 PFLOP/s in a short run, about 550 clocks per stage;
// under the power cap 114 to 119 us.

constexpr int MK = 256;  // codes per stage row: 128 bytes
constexpr int CHUNK_KB = 8;   // stages per chunk of an fp32 result
constexpr int LONG_KB = 64;   // stages per chunk of a bf16 result
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (2 + EPI_WARPS);
constexpr int EPI_BOX = 4096;
constexpr int ACC1 = 192;    // second accumulator's first column
constexpr int SF_COL = 448;  // scales: per stage 8 columns of A, 16 of B
static_assert(ACC1 + 256 == SF_COL && SF_COL + 2 * 24 <= 512, "tensor memory");

// NB columns of C per tile.
template <int NB>
struct GCfg {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = NB / 2 * 128;
  static constexpr int SB = NB > 128 ? 2 : 1;  // 128-row scale tiles of B
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + (1 + SB) * 1024;
  static constexpr int STAGES = NB == 256 ? 5 : 7;
  static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + EPI_WARPS * EPI_BOX + 256;
  static_assert(STAGE_BYTES % 1024 == 0, "swizzled tiles start on 1024-byte boundaries");
  static_assert(SMEM <= 232448, "product kernel exceeds shared memory");
};

// One scale tile (32 rows of 16 bytes) to four columns of tensor memory,
// repeated in all four lane quarters, in both CTAs of the pair (each from its
// own shared memory).
SHP_DEV void tmem_cp_scales_pair_if(uint32_t on, uint32_t taddr, uint64_t sdesc) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
      "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%1], %2;\n\t}" ::"r"(on),
      "r"(taddr), "l"(sdesc)
      : "memory");
}

SHP_DEV void mma_mxf4_pair_if(uint32_t on, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                              uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %0, 0;\n\t"
      "setp.ne.b32 p, %7, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X"
      " [%1], %2, %3, %4, [%5], [%6], p;\n\t}" ::"r"(on),
      "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
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
  SelfTest test;
};

// What a tile's sums become: bf16 of one accumulator, bf16 or fp32 of summed chunks.
enum GemmOut { PROD_BF16, PROD_BF16_CHUNKS, PROD_F32 };

template <int NB, GemmOut OUT>
__global__ void __launch_bounds__(THREADS, 1)
    k_mx4_gemm(const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tAs,
               const __grid_constant__ CUtensorMap tB, const __grid_constant__ CUtensorMap tBs,
               const __grid_constant__ CUtensorMap tO, Mx4Params p) {
  count_kernel_run();
  using C = GCfg<NB>;
  constexpr int STAGES = C::STAGES, STAGE_BYTES = C::STAGE_BYTES;
  constexpr bool F32 = OUT == PROD_F32, CHUNKS = OUT != PROD_BF16;
  constexpr int CHUNK = F32 ? CHUNK_KB : LONG_KB;
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
  uint64_t* never = drain + 1;  // completed by nothing: the self-test's wait
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
  volatile WaitState* ws = reinterpret_cast<volatile WaitState*>(never + 2);
  static_assert((2 * STAGES + 6) * 8 + sizeof(WaitState) <= 256, "barriers");

  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&accf[0], 1);
    mbar_init(&accf[1], 1);
    mbar_init(acce, 2 * EPI_WARPS);
    mbar_init(drain, 1);
    mbar_init(never, 1);
    wait_state_init(ws, p.test.limit, 0);
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
  const uint32_t tmem = uniform(*tmem_slot);

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs)
    const uint32_t on = elect_one(), lead = on & (leader ? 1u : 0u);
    RingPos<STAGES> ring;
    const uint32_t stages = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty);
    const uint32_t fleader = uniform(mapa_shared(full0, 0));
    bool stop = false;
    for (int t = cl; t < ntiles && !stop; t += ncl) {
      const int b = t / per_b, r = t % per_b;
      const int tm = r / p.tiles_n, tn = r % p.tiles_n;
      const int m0 = tm * 256 + static_cast<int>(rank) * 128;
      const int nb0 = tn * NB + static_cast<int>(rank) * (NB / 2);
      const int za = b * p.rb_a + tm * 2 + static_cast<int>(rank);
      const int zb = b * p.rb_b + tn * NB / 128;
      for (int kb = 0; kb < KB; ++kb) {
        if (!issue_wait<true>(empty0 + ring.slot * 8, ring.parity ^ 1u, ws)) {
          stop = true;
          break;
        }
        const uint32_t sa = stages + ring.slot * STAGE_BYTES, sf = sa + C::A_BYTES + C::B_BYTES;
        const uint32_t fbar = fleader + ring.slot * 8;
        mbar_expect_tx_if(lead, full0 + ring.slot * 8, 2 * STAGE_BYTES);
        tma_3d_pair_if(on, sa, &tA, fbar, kb * 64, m0, b);  // codes move as 16-bit units
        tma_3d_pair_if(on, sa + C::A_BYTES, &tB, fbar, kb * 64, nb0, b);
        tma_3d_pair_if(on, sf, &tAs, fbar, 0, kb * 2, za);
        tma_4d_pair_if(on, sf + 1024, &tBs, fbar, 0, kb * 2, zb, 0);
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
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
      const uint32_t accf0 = smem_u32(accf), acce0 = smem_u32(acce);
      const uint64_t adesc = smem_desc(smem_u32(smem), 16, 1024u, 2u);
      const uint64_t bdesc = smem_desc(smem_u32(smem) + C::A_BYTES, 16, 1024u, 2u);
      const uint64_t sdesc = smem_desc(smem_u32(smem) + C::A_BYTES + C::B_BYTES, 128, 128, 0);
      uint32_t u = 0, pe = 1;  // accumulator; parity of acce's last use
      uint32_t sf = 0;         // scale buffer
      bool stop = gave_up, ready = false;
      for (int t = cl; t < ntiles && !stop; t += ncl) {
        for (int c0 = 0; c0 < KB && !stop; c0 += CHUNKS ? CHUNK : KB, u ^= 1u, pe ^= 1u) {
          const int c1 = CHUNKS ? min(c0 + CHUNK, KB) : KB;
          if (!issue_wait(acce0, pe, ws)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t dacc = tmem + u * ACC1;
          for (int kb = c0; kb < c1; ++kb) {
            if (!ready && !issue_wait(full0 + ring.slot * 8, ring.parity, ws)) {
              stop = true;
              break;
            }
            tc_fence_after();
            const uint64_t at = static_cast<uint64_t>(ring.slot) * (STAGE_BYTES >> 4);
            const uint32_t tsa = tmem + SF_COL + sf * 24, tsb = tsa + 8;
            sf ^= 1u;
            const int left = p.K - kb * MK;  // columns of this stage inside the matrix
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if (k * 128 >= left) break;
              tmem_cp_scales_pair_if(on, tsa + k * 4, sdesc + at + k * 32);
              tmem_cp_scales_pair_if(on, tsb + k * 8, sdesc + at + 64 + k * 32);
              if (C::SB == 2) tmem_cp_scales_pair_if(on, tsb + k * 8 + 4, sdesc + at + 128 + k * 32);
            }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              if (ks * 64 >= left) break;
              mma_mxf4_pair_if(on, dacc, adesc + at + ks * 2, bdesc + at + ks * 2,
                               instr_desc_mxf4(256, NB, (ks & 1) * 2), tsa + (ks >> 1) * 4,
                               tsb + (ks >> 1) * 8, (kb > c0 || ks > 0) ? 1u : 0u);
            }
            const uint32_t ebar = empty0 + ring.slot * 8;
            ring.advance();
            ready = warp_test(full0 + ring.slot * 8, ring.parity);
            mma_commit_pair_if(on, ebar, 3);
          }
          mma_commit_pair_if(on, accf0 + u * 8, 3);
        }
      }
      mma_commit_pair_if(on, smem_u32(drain), 3);  // after every MMA issued above
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
      // warp half h owns half of the tile's columns; where they are 128 it reads
      // its two 64-column parts in the order that drains the shared columns first:
      // they are the upper part of half 1 in accumulator 0, the lower part of half
      // 0 in 1
      const int c0 = h * (NB / 2);
      const int n0 = r % p.tiles_n * NB + c0;
      // a 32-row x 64-column part as bf16 pairs w[0..31], through the box
      auto store_bf16 = [&](int part, const uint32_t* w) {
        if (row0 >= p.M || n0 + part >= p.N) return;
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
      };
      auto pair_bf16 = [](float lo, float hi) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&x);
      };
      if (CHUNKS) {
        constexpr int PARTS = NB / 64;
        const int flip = NB == 256 ? 2 * h : 0;
        float acc[NB / 2];
#pragma unroll
        for (int j = 0; j < NB / 2; ++j) acc[j] = 0.f;
        for (int kc = 0; kc < KB; kc += CHUNK, ++it) {
          const int u = it & 1;
          if (!warp_wait(smem_u32(&accf[u]), (it >> 1) & 1, ws)) {
            stop = true;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < PARTS; ++g) {
            float v[32];
            tmem_ld32(trow + static_cast<uint32_t>(u * ACC1 + c0 + (g ^ flip) * 32), v);
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[g * 32 + j] += v[j];
            if (g == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_relaxed(mapa_shared(smem_u32(acce), 0));
            }
          }
        }
        if (stop) break;
        if (!F32) {
#pragma unroll
          for (int g = 0; g < PARTS; g += 2) {
            uint32_t w[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
              w[j] = pair_bf16(acc[g * 32 + 2 * j], acc[g * 32 + 2 * j + 1]);
            store_bf16((g ^ flip) * 32, w);
          }
        } else if (row0 < p.M) {
#pragma unroll
          for (int g = 0; g < PARTS; ++g) {
            const int cb = n0 + (g ^ flip) * 32;
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
        if (!warp_wait(smem_u32(&accf[u]), (it >> 1) & 1, ws)) break;
        ++it;
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < (NB == 256 ? 2 : 1); ++g) {
          const int part = NB == 256 ? (g ^ h) * 64 : 0;
          uint32_t w[64];
          tmem_ld64(trow + static_cast<uint32_t>(u * ACC1 + c0 + part), w);
          if (g == 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(mapa_shared(smem_u32(acce), 0));
          }
#pragma unroll
          for (int j = 0; j < 32; ++j)
            w[j] = pair_bf16(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
          store_bf16(part, w);
        }
      }
    }
    if (lane == 0) bulk_wait_all();  // nothing outlives the CTA's shared memory
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();  // every role of this CTA has left its loop
  // so the pair's MMAs have only to complete, which a limit of a stage bounds
  if (warp == 1) mbar_wait(drain, 0, nullptr, ws->limit);
  selftest_report(p.test.status, &ws->abort);
  // releasing: this CTA's arrivals on the other's barriers land before it exits
  cluster_sync();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

namespace {

template <bool BF16>
cudaError_t launch_quantize(const CUtensorMap& x, const CUtensorMap& q, const CUtensorMap& qt,
                            const QParams& p, cudaStream_t st) {
  using C = QCfg<BF16>;
  static_assert(C::SMEM <= 232448, "quantiser exceeds shared memory");
  auto kern = k_mx4_quantize<BF16>;
  static std::atomic<uint64_t> done{0};
  const LaunchInfo li = launch_info(reinterpret_cast<const void*>(kern), C::SMEM, done);
  if (li.err != cudaSuccess) return li.err;
  // (the self-test: one CTA, so that it has more tiles than its ring holds)
  const int64_t ctas = p.test.stall > 0 ? 1 : li.sms;
  const unsigned grid = static_cast<unsigned>(p.tiles < ctas ? p.tiles : ctas);
  kern<<<grid, QTHREADS + 32, C::SMEM, st>>>(x, q, qt, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t mx4_quantize(const void* X, bool bf16, int rows, int cols, int64_t batch, uint8_t* Q,
                         uint8_t* S, uint8_t* Qt, uint8_t* St, cudaStream_t st,
                         const SelfTest& selftest) {
  QParams p;
  p.test = selftest;
  p.tiles_r = static_cast<int>(ceil_div(rows, QT));
  p.tiles_c = static_cast<int>(ceil_div(cols, QT));
  p.tiles = batch * p.tiles_r * p.tiles_c;
  p.s[0] = S;
  p.s[1] = St;
  // codes as 16-bit units: 8 per block of 32
  const int64_t uc = ceil_div(cols, 32) * 8, ur = ceil_div(rows, 32) * 8;
  CUtensorMap x, q, qt;
  memset(&q, 0, sizeof(q));
  memset(&qt, 0, sizeof(qt));
  if (!tensor_map(&x, X, bf16 ? 2 : 4, cols, rows, batch, cols, static_cast<int64_t>(rows) * cols,
                  bf16 ? 64 : 32, QT, CU_TENSOR_MAP_SWIZZLE_128B) ||
      (S != nullptr && !tensor_map(&q, Q, 2, uc, rows, batch, uc, uc * rows, 32, QT,
                                   CU_TENSOR_MAP_SWIZZLE_64B)) ||
      (St != nullptr && !tensor_map(&qt, Qt, 2, ur, cols, batch, ur, ur * cols, 32, QT,
                                    CU_TENSOR_MAP_SWIZZLE_64B)))
    return cudaErrorInvalidValue;
  return bf16 ? launch_quantize<true>(x, q, qt, p, st) : launch_quantize<false>(x, q, qt, p, st);
}

cudaError_t mx4_dequantize(const uint8_t* Q, const uint8_t* S, int rows, int cols, int64_t batch,
                           void* X, bool bf16, cudaStream_t st) {
  const int tr = static_cast<int>(ceil_div(rows, QT)), tc = static_cast<int>(ceil_div(cols, QT));
  const unsigned grid = static_cast<unsigned>(batch * tr * tc);
  if (bf16)
    k_mx4_dequantize<true><<<grid, 256, 0, st>>>(Q, S, rows, cols, tr, tc, X);
  else
    k_mx4_dequantize<false><<<grid, 256, 0, st>>>(Q, S, rows, cols, tr, tc, X);
  return cudaGetLastError();
}

namespace {

template <int NB, GemmOut OUT>
cudaError_t launch_gemm(const uint8_t* A, const uint8_t* As, const uint8_t* B, const uint8_t* Bs,
                        void* O, Mx4Params p, cudaStream_t st) {
  using C = GCfg<NB>;
  constexpr bool F32 = OUT == PROD_F32;
  p.tiles_m = static_cast<int>(ceil_div(p.M, 256));
  p.tiles_n = static_cast<int>(ceil_div(p.N, NB));
  const int64_t kt = ceil_div(p.K, 128);
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.batch;
  if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
  CUtensorMap a, as, b, bs, o;
  const int64_t u = p.K / 4;  // 16-bit units per row of codes
  if (!tensor_map(&a, A, 2, u, p.M, p.batch, u, u * p.M, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tensor_map(&b, B, 2, u, p.N, p.batch, u, u * p.N, 64, NB / 2, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tensor_map(&as, As, 4, 128, kt, p.batch * p.rb_a, 128, 128 * kt, 128, 2,
                  CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !tensor_map4(&bs, Bs, 4, {128, kt, p.batch * p.rb_b, 1},
                   {128, 128 * kt, 128 * kt * p.batch * p.rb_b}, {128, 2, C::SB, 1},
                   CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !tensor_map(&o, O, F32 ? 4 : 2, p.N, p.M, p.batch, p.N, static_cast<int64_t>(p.M) * p.N,
                  F32 ? 32 : 64, 32, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto kern = k_mx4_gemm<NB, OUT>;
  static std::atomic<uint64_t> done{0};
  const LaunchInfo li = launch_info(reinterpret_cast<const void*>(kern), C::SMEM, done);
  if (li.err != cudaSuccess) return li.err;
  int64_t ncl = li.sms / 2;
  if (ncl > tiles) ncl = tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * ncl), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
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

template <int NB>
cudaError_t dispatch_gemm(const uint8_t* A, const uint8_t* As, const uint8_t* B, const uint8_t* Bs,
                          void* O, bool f32, const Mx4Params& p, cudaStream_t st) {
  if (f32) return launch_gemm<NB, PROD_F32>(A, As, B, Bs, O, p, st);
  return p.K > LONG_KB * MK ? launch_gemm<NB, PROD_BF16_CHUNKS>(A, As, B, Bs, O, p, st)
                            : launch_gemm<NB, PROD_BF16>(A, As, B, Bs, O, p, st);
}

}  // namespace

cudaError_t mx4_gemm(const uint8_t* A, const uint8_t* As, const uint8_t* B, const uint8_t* Bs,
                     void* C, bool f32, int M, int N, int K, int64_t batch, cudaStream_t st,
                     const SelfTest& selftest) {
  Mx4Params p;
  memset(&p, 0, sizeof(p));
  p.test = selftest;
  p.M = M;
  p.N = N;
  p.K = K;
  p.batch = batch;
  p.rb_a = static_cast<int>(ceil_div(M, 128));
  p.rb_b = static_cast<int>(ceil_div(N, 128));
  if (batch * p.rb_a > INT32_MAX || batch * p.rb_b > INT32_MAX) return cudaErrorInvalidValue;
  // Tiles of 128 columns where those of 256 leave half of the SM pairs idle: a
  // stage of a tile then takes 173 ns, not 290 (16 x 4096 x 4096 8.4 us, not 9.5;
  // 256 x 8192 x 8192 12.4 us, not 15.7; 36 blocks of 100 x 200 x 512 5.9 us, not
  // 6.5; fp32 results gain more).  With more tiles they need more rounds (40
  // tiles, 1376 columns: 8.8 against 8.9 us; 112 tiles, 4096: 20.1 against 17.3).
  // (So a launch of these has no more tiles than pairs: no pair gets a second one.)
  const LaunchInfo li = device_info();
  if (li.err != cudaSuccess) return li.err;
  const int64_t wide = ceil_div(M, 256) * ceil_div(N, 256) * batch;
  return 2 * wide <= li.sms / 2 ? dispatch_gemm<128>(A, As, B, Bs, C, f32, p, st)
                           : dispatch_gemm<256>(A, As, B, Bs, C, f32, p, st);
}

uint64_t kernel_runs_mx4() {
  unsigned long long v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kernel_runs, sizeof(v)) != cudaSuccess) return 0;
  return v;
}

}  // namespace shp
