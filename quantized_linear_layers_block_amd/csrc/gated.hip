// Gated feed-forward block on blockwise-FP8 weights for gfx950: both projections, the activation
// and the product in one kernel.
//
//   g = x Wg^T,  u = x Wu^T    (E4M3 x E4M3, scales of 1x128 and 128x128 blocks, float32 sums)
//   h = g / (1 + exp(-g)) * u  in float32, then bf16, or E4M3 with a scale for 128 columns
//
// A workgroup computes the same columns of g and of u, so h needs no second pass over either:
// the weight rows of its tile are 64 of the gate and 64 of the up projection for each wave, and a
// lane's accumulators of the two halves belong to the same elements of h.
//
//   more than 64 tokens  tiles of 128 columns (256 weight rows), one segment of the 8-bit output, by 64
//                        to 256 tokens, a kernel for each way of applying scales
//   up to 64 tokens      bound by the weights: 16 to 64 columns a workgroup
#include <type_traits>
#include "common.hpp"
#include "fp8_out.hpp"
#include "gate.hpp"
#include "gemm_common.hpp"
#include "gemv_common.hpp"
#include "launch.hpp"

namespace ql {

namespace {

constexpr int kGCols = 128;      // columns of h per tile: one segment of an 8-bit output
constexpr int kGRows = 256;      // weight rows per tile
constexpr int kGRowBytes = 128;  // one K block of fp8 per LDS row
constexpr int kGPitch = 272;     // output staging: bytes per row of 128 bf16 columns (conflict-free 8-byte writes)
constexpr int kGPitch8 = 144;    // the same for 128 codes (conflict-free 4-byte writes)

__device__ __forceinline__ i32x8 gated_frag(const uint8_t* tile, int row, int g) {
  const uint8_t* p = tile + row * kGRowBytes;
  const i32x4 lo = *(const i32x4*)(p + swz(row, 2 * g) * 16);
  const i32x4 hi = *(const i32x4*)(p + swz(row, 2 * g + 1) * 16);
  return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// A tile's results to memory.  acc[0..3] is g and acc[4..7] u of the wave's 64 columns (16 i + 4 lg + e)
// by 16 MJ tokens (16 j + r); the wave stands at column 64 wn and token mw of the tile.  Everything
// leaves through LDS as whole rows.  `amax`: LDS for [2][TM] words.
template <int THREADS, int TM, int MJ>
__device__ __forceinline__ void gated_store(const Gated& a, f32x4 (&acc)[8][MJ], int split, int64_t m0, int64_t n0, int wn,
                                            int mw, int r, int lg, uint8_t* stage, uint32_t* amax) {
  const int tid = threadIdx.x;
  if (a.split > 1) {   // a part of K: float32 [split][m][2 n], for gated_join_kernel
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      const int64_t row = m0 + mw + 16 * j + r;
      if (row >= a.m) continue;
      float* p = a.scratch + ((int64_t)split * a.m + row) * 2 * a.n + n0 + 64 * wn + 4 * lg;
#pragma unroll
      for (int i = 0; i < 8; ++i) *(f32x4*)(p + (i < 4 ? 16 * i : a.n + 16 * (i - 4))) = acc[i][j];
    }
    return;
  }
  auto rows_out = [&](uint16_t* dst, int64_t stride, int from) {   // bf16(acc[from..from + 3]) -> dst [m][stride]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < MJ; ++j) {
        const f32x4 v = acc[from + i][j];
        *(uint2*)(stage + (mw + 16 * j + r) * kGPitch + (64 * wn + 16 * i + 4 * lg) * 2) =
            make_uint2(pack_bf16x2_rne(v[0], v[1]), pack_bf16x2_rne(v[2], v[3]));
      }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < TM * 16 / THREADS; ++q) {
      const int row = (tid >> 4) + q * (THREADS / 16);
      if (m0 + row < a.m)
        *(i32x4*)(dst + (m0 + row) * stride + n0 + (tid & 15) * 8) = *(const i32x4*)(stage + row * kGPitch + (tid & 15) * 16);
    }
  };
  if (a.gu) {
    rows_out(a.gu, 2 * a.n, 0);
    rows_out(a.gu + a.n, 2 * a.n, 4);
  }
  gate_products(*(f32x4(*)[4][MJ])acc, *(const f32x4(*)[4][MJ])(acc + 4));
  if (a.h) rows_out(a.h, a.n, 0);
  if (!a.hq) return;
  // a token's 128 values are in the four lane groups of the two waves along n
  uint32_t top[MJ];
#pragma unroll
  for (int j = 0; j < MJ; ++j) {
    top[j] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) top[j] = umax(top[j], abs_bits(acc[i][j][e]));
    top[j] = umax(top[j], (uint32_t)__shfl_xor((int)top[j], 16));
    top[j] = umax(top[j], (uint32_t)__shfl_xor((int)top[j], 32));
  }
  __syncthreads();
  if (lg == 0)
#pragma unroll
    for (int j = 0; j < MJ; ++j) amax[wn * TM + mw + 16 * j + r] = top[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < MJ; ++j) {
    const int row = mw + 16 * j + r;
    const uint32_t t = umax(top[j], amax[(wn ^ 1) * TM + row]);
    const Fp8Seg sc = a.pow2 ? fp8_seg_scale<true>(t) : fp8_seg_scale<false>(t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      *(uint32_t*)(stage + row * kGPitch8 + 64 * wn + 16 * i + 4 * lg) = fp8_encode4(f, sc);
    }
    if (lg == 0 && wn == 0 && m0 + row < a.m) {
      const int64_t seg = (m0 + row) * (a.n / 128) + n0 / 128;
      if (a.pow2)
        ((uint8_t*)a.sh)[seg] = (uint8_t)sc.stored;
      else
        ((uint32_t*)a.sh)[seg] = sc.stored;
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < TM * 8 / THREADS; ++q) {
    const int row = (tid >> 3) + q * (THREADS / 8);
    if (m0 + row < a.m)
      *(i32x4*)(a.hq + (m0 + row) * a.n + n0 + (tid & 7) * 16) = *(const i32x4*)(stage + row * kGPitch8 + (tid & 7) * 16);
  }
}

// The workgroup's tile and K blocks, in scalar registers (the copies' base addresses have to be there).
struct GatedWork {
  int64_t tm, tn, kb0, kb1;
  int split;
};
__device__ __forceinline__ GatedWork gated_work(const Gated& a) {
  GatedWork w;
  int64_t tm, tn;
  const int64_t b = a.split > 1 ? blockIdx.x / a.split : gemm_xcd_remap(blockIdx.x, gridDim.x);
  gemm_group_tile(b, a.tiles_m, a.tiles_n, tm, tn);
  w.tm = __builtin_amdgcn_readfirstlane((int)tm);
  w.tn = __builtin_amdgcn_readfirstlane((int)tn);
  w.split = __builtin_amdgcn_readfirstlane(a.split > 1 ? (int)(blockIdx.x % a.split) : 0);
  const int64_t kblocks = a.k / 128;
  w.kb0 = w.split * a.blocks_each;
  w.kb1 = w.kb0 + a.blocks_each < kblocks ? w.kb0 + a.blocks_each : kblocks;
  return w;
}

// Eight E4M3 codes -> eight f16, exactly (the converter's scale is 1).
__device__ __forceinline__ f16x2 e4m3_f16(int w, bool high) {
  return high ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((unsigned)w, 1.0f, true)
              : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((unsigned)w, 1.0f, false);
}
__device__ __forceinline__ f16x8 e4m3_f16x8(int lo, int hi) {
  const f16x2 a = e4m3_f16(lo, false), b = e4m3_f16(lo, true), c = e4m3_f16(hi, false), d = e4m3_f16(hi, true);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// ------------------------------------------------------------------ float32 scales, many tokens
// An output scale is amax / 448 in float32, so the sums behind it have to be right to float32's
// order.  The FP8 matrix instructions align eight products at a time and keep 13 bits below the
// largest (measured: 1.4e-5 of the result on normal data, 5e-5 on codes of every size), f16 ones keep
// float32's 24; and every E4M3 value is an f16.  So the operands stay E4M3 in memory and LDS, the lanes
// turn their fragments into f16 (a lane's 32 bytes are four steps of 8), and each K block's products
// start from zero and are folded into the sums with one FMA by the block's scale.
// Eight waves, 2 along n by 4 along m; a wave's 128 weight rows are 64 of the gate then 64 of the up
// projection, its tokens 16 MJ: with MJ = 3 sums, fragments and two sets of products fit 256 registers.  K blocks are
// copied one ahead, two where LDS has the room (300 x 5120 x 2048 27.5 -> 25.9 us; longer ones 2% or less).  8192 x 14336
// x 4096 1590 us: matrix units 52%, vector units 59% (folding, and each wave's conversions) of the cycles at 1.9 GHz.
constexpr int kGfThreads = 512;
template <int MJ>
constexpr int gf_stages() { return MJ == 3 ? 2 : 3; }
template <int MJ>
constexpr int gf_ring() { return 64 * MJ * 16 + 1024; }   // a slot of the scale ring: 16 bytes a token, then the weights'
template <int MJ>
constexpr size_t gf_lds() {
  constexpr size_t loop = gf_stages<MJ>() * (kGRows + 64 * MJ) * kGRowBytes + 2 * gf_ring<MJ>(), out = 64 * MJ * kGPitch + 2 * 64 * MJ * 4;
  return loop > out ? loop : out;
}

template <int MJ, bool SW4>
__global__ __launch_bounds__(kGfThreads) void gated_f32s_kernel(Gated a) {
  extern __shared__ __align__(16) uint8_t smem[];  // [AHEAD + 1][W 256 x 128 | x TM x 128], scale ring
  constexpr int TM = 64 * MJ, AHEAD = gf_stages<MJ>() - 1;
  constexpr int kStage = (kGRows + TM) * kGRowBytes;
  const GatedWork work = gated_work(a);
  const int64_t tn = work.tn, n0 = tn * kGCols, m0 = work.tm * TM;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int wn = wave & 1, wm = wave >> 1;
  const int r = lane & 15, g = lane >> 4;
  const int64_t kblocks = a.k / 128;

  // Copies of a K block: q < 4 the LDS weight rows 64 q + 8 wave + lane / 8, which are rows
  // 64 (q / 2) + 8 wave + lane / 8 of the gate (q even) or of the up projection; q >= 4 the tokens
  // 64 (q - 4) + 8 wave + lane / 8 (past the last one, the last again).
  uint32_t ow[2], ox[MJ];
  const int64_t m_last = a.m - 1 - m0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 64 * i + 8 * wave + (lane >> 3);   // (its swizzle is that of LDS rows 64 further, too)
    ow[i] = (uint32_t)row * (uint32_t)a.k + (uint32_t)swz(row, lane & 7) * 16;
  }
#pragma unroll
  for (int i = 0; i < MJ; ++i) {
    const int row = 64 * i + 8 * wave + (lane >> 3);
    ox[i] = (uint32_t)(row < m_last ? row : m_last) * (uint32_t)a.k + (uint32_t)swz(row, lane & 7) * 16;
  }
  const uint8_t* gbase = a.wg + n0 * a.k;
  const uint8_t* ubase = a.wu + n0 * a.k;
  const uint8_t* xbase = a.xq + m0 * a.k;
  auto dma = [&](int64_t kb, int buf, int q) {
    const uint32_t lb = lds_addr(smem + buf * kStage) + 8 * wave * kGRowBytes;
    if (q < 4)
      lds_copy16((q & 1 ? ubase : gbase) + kb * 128, ow[q >> 1], lb + 64 * q * kGRowBytes);
    else
      lds_copy16(xbase + kb * 128, ox[q - 4], lb + (kGRows + 64 * (q - 4)) * kGRowBytes);
  };
  // Scales.  SW4 (K a multiple of 512, 16-byte aligned arrays): the four float scales of four blocks of a
  // row are one 16-byte unit, copied to the ring once per four blocks (waves 0 .. MJ - 1 a token a
  // lane, wave 4 the gate's unit in lane 0 and the up projection's in the others).
  const float* sxb = (const float*)a.sx + m0 * kblocks;
  const float* sgb = (const float*)a.sg + tn * kblocks;
  const float* sub = (const float*)a.su + tn * kblocks;
  uint32_t osx[MJ];
#pragma unroll
  for (int j = 0; j < MJ; ++j) {
    const int64_t row = 16 * MJ * wm + 16 * j + r;
    osx[j] = (uint32_t)((row < m_last ? row : m_last) * kblocks);
  }
  constexpr int kRing = gf_stages<MJ>() * kStage;
  const int arow = 64 * (wave & 3) + lane;
  const uint32_t oxu = (uint32_t)((arow < m_last ? arow : m_last) * kblocks * 4);
  auto dma_sc = [&](int64_t grp) {
    const uint32_t lb = lds_addr(smem + kRing) + (uint32_t)(grp & 1) * gf_ring<MJ>();
    if (wave < MJ)
      lds_copy16((const uint8_t*)sxb + 16 * grp, oxu, lb + wave * 1024);
    else if (wave == 4)
      lds_copy16_va((lane == 0 ? sgb : sub) + 4 * grp, lb + TM * 16);
  };
  float sxn[MJ], sgn, sun;
  auto next_sc = [&](int64_t kb) {
    if (SW4) {
      const uint8_t* sl = smem + kRing + (int)((kb >> 2) & 1) * gf_ring<MJ>() + 4 * (int)(kb & 3);
      sgn = *(const float*)(sl + TM * 16);
      sun = *(const float*)(sl + TM * 16 + 16);
#pragma unroll
      for (int j = 0; j < MJ; ++j) sxn[j] = *(const float*)(sl + 16 * (16 * MJ * wm + 16 * j + r));
    } else {
      sgn = sgb[kb];
      sun = sub[kb];
#pragma unroll
      for (int j = 0; j < MJ; ++j) sxn[j] = sxb[osx[j] + kb];
    }
  };

  f32x4 acc[8][MJ];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < MJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int t = 0; t < AHEAD; ++t)
#pragma unroll
    for (int q = 0; q < 4 + MJ; ++q) dma(work.kb0 + t < work.kb1 ? work.kb0 + t : work.kb1 - 1, t, q);
  if (SW4) dma_sc(work.kb0 >> 2);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  next_sc(work.kb0);

  // Software pipeline, fragment by fragment (8 fragments of 16 weight rows against MJ of 16 tokens).
  // Each MFMA stands with one of the FMAs that fold the fragment before and with conversions of the
  // fragment's next step, so that matrix and vector units have work side by side.  The next fragment
  // comes from LDS during a fragment's first step; the next block's copies go out during fragments
  // 0 .. 6, and the barrier sits before fragment 7, which also takes the next block's tokens.
  const f32x4 zero = {0, 0, 0, 0};
  f32x4 p[2][MJ];
  float scg[MJ], scu[MJ], scl[MJ];
  f16x8 xf[MJ][4], wf[2];
  i32x8 wr, wrn;
#pragma unroll
  for (int j = 0; j < MJ; ++j) {
    p[1][j] = zero;
    scu[j] = 0.0f;
    const i32x8 x = gated_frag(smem + kGRows * kGRowBytes, 16 * MJ * wm + 16 * j + r, g);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) xf[j][kk] = e4m3_f16x8(x[2 * kk], x[2 * kk + 1]);
  }
  wr = gated_frag(smem, 128 * wn + r, g);
  wf[0] = e4m3_f16x8(wr[0], wr[1]);
  int buf = 0;
  for (int64_t kb = work.kb0; kb < work.kb1; ++kb) {
    const int64_t kn = kb + 1 < work.kb1 ? kb + 1 : kb;
    const int64_t kc = kb + AHEAD < work.kb1 ? kb + AHEAD : work.kb1 - 1;   // (past the last: into a slot not read again)
    const int bufn = buf == AHEAD ? 0 : buf + 1, bufc = buf == 0 ? AHEAD : buf - 1;
#pragma unroll
    for (int j = 0; j < MJ; ++j) {
      scl[j] = scu[j];
      scg[j] = sxn[j] * sgn;
      scu[j] = sxn[j] * sun;
    }
    // kn's group landed at least a block's barrier ago: a group's copy goes out two blocks before its first
    if (SW4 && ((kb + 2) & 3) == 0 && kb + 2 < work.kb1) dma_sc((kb + 2) >> 2);
    next_sc(kn);
    const uint8_t* As = smem + buf * kStage;
    const uint8_t* An = smem + bufn * kStage;
    i32x8 xr[MJ];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i == 7) {
        // this block's LDS reads are done and the next block's copies have landed
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(AHEAD == 2 ? 4 + MJ : 0) : "memory");
        __syncthreads();
#pragma unroll
        for (int j = 0; j < MJ; ++j) xr[j] = gated_frag(An + kGRows * kGRowBytes, 16 * MJ * wm + 16 * j + r, g);
      }
      f32x4(&pn)[MJ] = p[i & 1];
      const f32x4(&po)[MJ] = p[(i & 1) ^ 1];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
        for (int j = 0; j < MJ; ++j) {
          const int s = kk * MJ + j;
          pn[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wf[kk & 1], xf[j][kk], kk ? pn[j] : zero, 0, 0, 0);
          {  // 4 MJ products of the fragment before, one a step
            const int t = s >> 2, e = s & 3;
            const float sc = i == 0 ? scl[t] : i <= 4 ? scg[t] : scu[t];
            acc[(i + 7) & 7][t][e] += sc * po[t][e];
          }
          if (s == 0) wrn = i < 7 ? gated_frag(As, 128 * wn + 16 * (i + 1) + r, g) : gated_frag(An, 128 * wn + r, g);
          if (j == MJ - 1) wf[(kk & 1) ^ 1] = kk < 3 ? e4m3_f16x8(wr[2 * kk + 2], wr[2 * kk + 3]) : e4m3_f16x8(wrn[0], wrn[1]);
          if (i < 4 + MJ && s == 1) dma(kc, bufc, i);
          if (i == 7) xf[j][kk] = e4m3_f16x8(xr[j][2 * kk], xr[j][2 * kk + 1]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      wr = wrn;
    }
    buf = bufn;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // copies still under way into what gated_store writes
#pragma unroll
  for (int j = 0; j < MJ; ++j) acc[7][j] += scu[j] * p[1][j];
  gated_store<kGfThreads, TM, MJ>(a, acc, work.split, m0, n0, wn, 16 * MJ * wm, r, g, smem, (uint32_t*)(smem + TM * kGPitch));
}

// ------------------------------------------------------------------ powers of two, many tokens
// The MFMA applies E8M0 scales itself and accumulates in place, with the 13 bits named above: a scale, being a power of
// two, is right unless its segment's largest value lies within the sums' error of a border, and f16 products took 1550
// us in place of 885 (8192 x 14336 x 4096, in one tiling).  Eight waves, 2 along n by 4 along m, so that one
// wave's epilogue runs beside the other's of its SIMD (four waves of twice the sums spilled 97 registers there:
// 8192 x 14336 x 512 546 us against 180, x 4096 1073 against 760).  K blocks are copied one ahead, two ahead where
// LDS has the room: a tile of 64 or 128 tokens has less work in a block than a copy takes (n = 16384, K 5120, 128
// tokens a tile: 258 -> 180 us; 64: 226 -> 148).
constexpr int kGpThreads = 512;
template <int TM>
constexpr int gp_stages() { return TM == 256 ? 2 : 3; }
template <int TM>
constexpr int gp_ring() { return TM * 4 + 256; }
template <int TM>
constexpr size_t gp_lds() {
  constexpr size_t loop = gp_stages<TM>() * (kGRows + TM) * kGRowBytes + 2 * gp_ring<TM>(), out = TM * kGPitch + 2 * TM * 4;
  return loop > out ? loop : out;
}

template <int TM, bool SW4>
__global__ __launch_bounds__(kGpThreads) void gated_pow2_kernel(Gated a) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int MJ = TM / 64, NX = TM / 64, AHEAD = gp_stages<TM>() - 1;
  constexpr int kStage = (kGRows + TM) * kGRowBytes;
  const GatedWork work = gated_work(a);
  const int64_t tn = work.tn, n0 = tn * kGCols, m0 = work.tm * TM;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int wn = wave & 1, wm = wave >> 1;
  const int r = lane & 15, g = lane >> 4;
  const int64_t kblocks = a.k / 128;

  // Copies of a K block, each 64 LDS rows: gate, up, gate and up rows, then tokens.
  uint32_t ow[2], ox[NX];
  const int64_t m_last = a.m - 1 - m0;
  const int crow = 8 * wave + (lane >> 3);
  const uint32_t chunk = (uint32_t)swz(crow, lane & 7) * 16;   // (that of any row 64 further, too)
#pragma unroll
  for (int i = 0; i < 2; ++i) ow[i] = (uint32_t)(64 * i + crow) * (uint32_t)a.k + chunk;
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    const int row = 64 * i + crow;
    ox[i] = (uint32_t)(row < m_last ? row : m_last) * (uint32_t)a.k + chunk;
  }
  const uint8_t* gbase = a.wg + n0 * a.k;
  const uint8_t* ubase = a.wu + n0 * a.k;
  const uint8_t* xbase = a.xq + m0 * a.k;
  auto dma = [&](int64_t kb, int buf, int q) {
    const uint32_t lb = lds_addr(smem + buf * kStage) + (64 * q + 8 * wave) * kGRowBytes;
    if (q < 4)
      lds_copy16((q & 1 ? ubase : gbase) + kb * 128, ow[q >> 1], lb);
    else
      lds_copy16(xbase + kb * 128, ox[q - 4], lb);
  };
  const uint8_t* sxb = (const uint8_t*)a.sx + m0 * kblocks;
  const uint8_t* sgb = (const uint8_t*)a.sg + tn * kblocks;
  const uint8_t* sub = (const uint8_t*)a.su + tn * kblocks;
  uint32_t osx[MJ];
#pragma unroll
  for (int j = 0; j < MJ; ++j) {
    const int64_t row = 16 * MJ * wm + 16 * j + r;
    osx[j] = (uint32_t)((row < m_last ? row : m_last) * kblocks);
  }
  // SW4 (K a multiple of 512, 4-byte aligned arrays): the bytes of four blocks are one word, in a ring of two
  constexpr int kRing = gp_stages<TM>() * kStage;
  const int arow = 64 * wave + lane;
  const uint32_t oxw = (uint32_t)((arow < m_last ? arow : m_last) * kblocks);
  auto dma_sc = [&](int64_t grp) {
    const uint32_t lb = lds_addr(smem + kRing) + (uint32_t)(grp & 1) * gp_ring<TM>();
    if (wave < TM / 64) lds_copy4(sxb + 4 * grp, oxw, lb + wave * 256);
    if (wave == 3) lds_copy4_va((lane == 0 ? sgb : sub) + 4 * grp, lb + TM * 4);
  };
  int sgn, sun, sbn[MJ];
  auto next_sc = [&](int64_t kb) {
    if (SW4) {
      const uint8_t* sl = smem + kRing + (int)((kb >> 2) & 1) * gp_ring<TM>() + (int)(kb & 3);
      sgn = sl[TM * 4];
      sun = sl[TM * 4 + 4];
#pragma unroll
      for (int j = 0; j < MJ; ++j) sbn[j] = sl[4 * (16 * MJ * wm + 16 * j + r)];
    } else {
      sgn = sgb[kb];
      sun = sub[kb];
#pragma unroll
      for (int j = 0; j < MJ; ++j) sbn[j] = sxb[osx[j] + kb];
    }
  };

  f32x4 acc[8][MJ];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < MJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int t = 0; t < AHEAD; ++t)
#pragma unroll
    for (int q = 0; q < 4 + NX; ++q) dma(work.kb0 + t < work.kb1 ? work.kb0 + t : work.kb1 - 1, t, q);
  if (SW4) dma_sc(work.kb0 >> 2);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  next_sc(work.kb0);
  int sg = sgn, su = sun, sb[MJ];
#pragma unroll
  for (int j = 0; j < MJ; ++j) sb[j] = sbn[j];
  i32x8 bf[MJ], af, afn;
#pragma unroll
  for (int j = 0; j < MJ; ++j) bf[j] = gated_frag(smem + kGRows * kGRowBytes, 16 * MJ * wm + 16 * j + r, g);
  af = gated_frag(smem, 128 * wn + r, g);
  int buf = 0;
  for (int64_t kb = work.kb0; kb < work.kb1; ++kb) {
    const int64_t kn = kb + 1 < work.kb1 ? kb + 1 : kb;
    const int64_t kc = kb + AHEAD < work.kb1 ? kb + AHEAD : work.kb1 - 1;   // (past the last: into a slot not read again)
    const int bufn = buf == AHEAD ? 0 : buf + 1, bufc = buf == 0 ? AHEAD : buf - 1;
    if (SW4 && ((kb + 2) & 3) == 0 && kb + 2 < work.kb1) dma_sc((kb + 2) >> 2);
    next_sc(kn);
    const uint8_t* As = smem + buf * kStage;
    const uint8_t* An = smem + bufn * kStage;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i == 7) {
        // all but this block's own copies, if those are for the block after the next
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(AHEAD == 2 ? 4 + NX : 0) : "memory");
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < MJ; ++j) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af, bf[j], acc[i][j], 0, 0, 0, i < 4 ? sg : su, 0, sb[j]);
        if (j == 0) afn = i < 7 ? gated_frag(As, 128 * wn + 16 * (i + 1) + r, g) : gated_frag(An, 128 * wn + r, g);
        if (MJ == 4) {
          if (i < 4 && (j == 1 || j == 2)) dma(kc, bufc, 2 * i + j - 1);
        } else if (j == MJ - 1 && i < 4 + NX) {
          dma(kc, bufc, i);
        }
        if (i == 7) bf[j] = gated_frag(An + kGRows * kGRowBytes, 16 * MJ * wm + 16 * j + r, g);
        __builtin_amdgcn_sched_barrier(0);
      }
      af = afn;
    }
    buf = bufn;
    sg = sgn;
    su = sun;
#pragma unroll
    for (int j = 0; j < MJ; ++j) sb[j] = sbn[j];
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // copies still under way into what gated_store writes
  gated_store<kGpThreads, TM, MJ>(a, acc, work.split, m0, n0, wn, 16 * MJ * wm, r, g, smem, (uint32_t*)(smem + TM * kGPitch));
}

// ------------------------------------------------------------------ up to 64 tokens
// Bound by the weights, which are read once.  A workgroup has 16, 32 or 64 columns of h, so an 8-bit output's
// segment of 128 columns comes from several: they leave float32 values in the workspace, and the last to arrive
// (an integer counter, returned to zero) quantizes them.
//   gated_few_kernel   16 columns; eight waves take the K blocks in turn and read weights and tokens straight
//                      into the MFMA's fragments.  For narrow projections, where K has to be split to have waves
//                      enough: 4096 x 4096, one token 11.2 us, 64 tokens 24 (float32 scales; wide: 17.3, 31).
//   gated_wide_kernel  32 or 64 columns, each wave 16 weight rows and all of K, tokens shared through LDS.  Read
//                      into each wave's fragments, 64 tokens cost more than the weights: 14336 x 4096 28.8 us
//                      against 65 (powers of two), 35 against 83 (float32); one token 24 against 28.
constexpr int kFewWaves = 8;

// What follows a workgroup's sums: the outputs of 16 RT columns from n0 on.  part: [copies][2 RT MT pieces][lane],
// the copies' sums to be added, the pieces those of g and then of u; `last` is one word of LDS.
template <int MT, int RT, int COPIES, int WAVES, bool POW2>
__device__ __forceinline__ void few_finish(const Gated& a, int64_t n0, const f32x4* part, int* last) {
  constexpr int kTiles = 2 * RT * MT, kFewThreads = WAVES * kWave;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int r = lane & 15, g = lane >> 4;
  const int64_t nb = n0 / 128;
  __amdgpu_buffer_rsrc_t hs = dev_rsrc(a.scratch);
  for (int t = wave; t < RT * MT; t += WAVES) {   // one 16 x 16 piece of h a wave
    const int i = t / MT, j = t % MT;
    f32x4 gv = {0, 0, 0, 0}, uv = gv;
#pragma unroll
    for (int w = 0; w < COPIES; ++w) {
      gv += part[(w * kTiles + i * MT + j) * kWave + lane];
      uv += part[(w * kTiles + (RT + i) * MT + j) * kWave + lane];
    }
    const f32x4 hv = gate_product4(gv, uv);
    const int64_t row = 16 * j + r, col = n0 + 16 * i + 4 * g;
    if (row >= a.m) continue;
    auto out = [&](uint16_t* p, f32x4 v) {
      *(uint2*)p = make_uint2(pack_bf16x2_rne(v[0], v[1]), pack_bf16x2_rne(v[2], v[3]));
    };
    if (a.gu) {
      out(a.gu + row * 2 * a.n + col, gv);
      out(a.gu + row * 2 * a.n + a.n + col, uv);
    }
    if (a.h) out(a.h + row * a.n + col, hv);
    // the segment's block of the workspace: [n / 128][m][128] float32
    if (a.hq) st_dev4v(hs, (uint32_t)(((nb * a.m + row) * 128 + col % 128) * 4), hv);
  }
  if (!a.hq) return;
  wait_stores();
  __syncthreads();
  constexpr uint32_t kArrive = 128 / (16 * RT);
  if (threadIdx.x == 0) {
    uint32_t* cnt = a.counters + nb;
    const uint32_t old = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *last = old == kArrive - 1;
    if (*last) st_dev_u32(cnt, 0u);
  }
  __syncthreads();
  if (!*last) return;
  // 32 lanes a token, 4 columns each
  const int c4 = threadIdx.x & 31;
  for (int64_t row = threadIdx.x >> 5; row < a.m; row += kFewThreads / 32) {
    const f32x4 v = ld_dev4v(hs, (uint32_t)(((nb * a.m + row) * 128 + 4 * c4) * 4));
    uint32_t top = umax(umax(abs_bits(v[0]), abs_bits(v[1])), umax(abs_bits(v[2]), abs_bits(v[3])));
    top = max_row16(top);
    top = umax(top, (uint32_t)__shfl_xor((int)top, 16));
    const Fp8Seg sc = fp8_seg_scale<POW2>(top);
    const float f[4] = {v[0], v[1], v[2], v[3]};
    *(uint32_t*)(a.hq + row * a.n + nb * 128 + 4 * c4) = fp8_encode4(f, sc);
    if (c4 == 0) {
      const int64_t seg = row * (a.n / 128) + nb;
      if (POW2)
        ((uint8_t*)a.sh)[seg] = (uint8_t)sc.stored;
      else
        ((uint32_t*)a.sh)[seg] = sc.stored;
    }
  }
}

template <int MT, bool POW2>
__global__ __launch_bounds__(kFewWaves * kWave) void gated_few_kernel(Gated a) {
  __shared__ __align__(16) f32x4 part[4 * 2 * MT * kWave];
  __shared__ int last;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t kblocks = a.k / 128;
  const int64_t nb = n0 / 128;
  const uint8_t* gp = a.wg + (n0 + r) * a.k + 16 * g;
  const uint8_t* up = a.wu + (n0 + r) * a.k + 16 * g;
  int64_t xrow[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t row = 16 * j + r;
    xrow[j] = row < a.m ? row : a.m - 1;
  }
  f32x4 acc[2][MT];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[h][j] = f32x4{0, 0, 0, 0};

  // 16 bytes of each half of a block's 128: four lanes have 64 bytes side by side (K's order is alike in both operands)
  auto load32 = [](const uint8_t* p) {
    const i32x4 lo = *(const i32x4*)p, hi = *(const i32x4*)(p + 64);
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  for (int64_t kb = wave; kb < kblocks; kb += kFewWaves) {
    const i32x8 wf[2] = {load32(gp + kb * 128), load32(up + kb * 128)};
    i32x8 xf[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) xf[j] = load32(a.xq + xrow[j] * a.k + kb * 128 + 16 * g);
    if (POW2) {
      const int sw[2] = {((const uint8_t*)a.sg)[nb * kblocks + kb], ((const uint8_t*)a.su)[nb * kblocks + kb]};
      int sx[MT];
#pragma unroll
      for (int j = 0; j < MT; ++j) sx[j] = ((const uint8_t*)a.sx)[xrow[j] * kblocks + kb];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < MT; ++j)
          acc[h][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[h], xf[j], acc[h][j], 0, 0, 0, sw[h], 0, sx[j]);
    } else {
      const float sw[2] = {((const float*)a.sg)[nb * kblocks + kb], ((const float*)a.su)[nb * kblocks + kb]};
      float sx[MT];
#pragma unroll
      for (int j = 0; j < MT; ++j) sx[j] = ((const float*)a.sx)[xrow[j] * kblocks + kb];
      f32x4 p[2][MT];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        f16x8 x16[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) x16[j] = e4m3_f16x8(xf[j][2 * kk], xf[j][2 * kk + 1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f16x8 w16 = e4m3_f16x8(wf[h][2 * kk], wf[h][2 * kk + 1]);
#pragma unroll
          for (int j = 0; j < MT; ++j)
            p[h][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w16, x16[j], kk ? p[h][j] : f32x4{0, 0, 0, 0}, 0, 0, 0);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[h][j] += p[h][j] * (sw[h] * sx[j]);
    }
  }

  // waves 4..7 hand their sums to waves 0..3, then all four to everybody
  auto put = [&](int w) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < MT; ++j) part[((w * 2 + h) * MT + j) * kWave + lane] = acc[h][j];
  };
  if (wave >= 4) put(wave - 4);
  __syncthreads();
  if (wave < 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[h][j] += part[((wave * 2 + h) * MT + j) * kWave + lane];
  }
  __syncthreads();
  if (wave < 4) put(wave);
  __syncthreads();
  few_finish<MT, 1, 4, kFewWaves, POW2>(a, n0, part, &last);
}

// A ring of three K blocks (two under way: 4 to 6 were equal or, with fewer workgroups a CU, slower).  Every
// workgroup begins at another K block: with all of them at one, rows of 4096 bytes lie in the same few channels
// of the memory (14336 x 4096, one token: 28.3 -> 23.8 us; 18944 x 3584: alike).  The order of a sum is a matter
// of n, n0 and k (n chooses a workgroup's width, and n0 its place among them).  Scales come in panels of 16 blocks.
constexpr int kWidePanel = 16, kWideRing = 3;
template <int MT, int WAVES, bool POW2>
constexpr size_t wide_panel() { return kWidePanel * (16 * MT + 2) * (POW2 ? 1 : 4); }
template <int MT, int WAVES, bool POW2>
constexpr size_t wide_lds() { return kWideRing * (16 * WAVES + 16 * MT) * kGRowBytes + wide_panel<MT, WAVES, POW2>() + 64; }

template <int MT, int WAVES, bool POW2>
__global__ __launch_bounds__(WAVES * kWave) void gated_wide_kernel(Gated a) {
  using S = typename std::conditional<POW2, uint8_t, float>::type;
  constexpr int RING = kWideRing, kStage = (16 * WAVES + 16 * MT) * kGRowBytes, kRT = WAVES / 2;
  extern __shared__ __align__(16) uint8_t smem[];
  S* const sxp = (S*)(smem + RING * kStage);
  S* const swp = sxp + kWidePanel * 16 * MT;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int r = lane & 15, g = lane >> 4;
  const bool up = wave >= kRT;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * kRT);
  const int kblocks = (int)(a.k / 128);
  const int first = (int)(blockIdx.x * 5 % kblocks);
  auto at = [&](int t) { return t + first < kblocks ? t + first : t + first - kblocks; };
  const S* sxs = (const S*)a.sx;
  const S* sgs = (const S*)a.sg + n0 / 128 * kblocks;
  const S* sus = (const S*)a.su + n0 / 128 * kblocks;

  const uint8_t* wbase = up ? a.wu + (n0 + 16 * (wave - kRT)) * a.k : a.wg + (n0 + 16 * wave) * a.k;
  constexpr int kX = 2 * MT / WAVES, kOdd = 2 * MT % WAVES;
  uint32_t ow[2], ox[kX + 1];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = 8 * q + (lane >> 3);
    ow[q] = (uint32_t)row * (uint32_t)a.k + (uint32_t)swz(row, lane & 7) * 16;
  }
#pragma unroll
  for (int q = 0; q <= kX; ++q) {
    const int row = 8 * (wave + WAVES * q) + (lane >> 3);
    ox[q] = (uint32_t)(row < a.m ? row : a.m - 1) * (uint32_t)a.k + (uint32_t)swz(row, lane & 7) * 16;
  }
  auto copy = [&](int t, int slot) {
    const int64_t kb = at(t);
    const uint32_t lb = lds_addr(smem + slot * kStage);
#pragma unroll
    for (int q = 0; q < 2; ++q) lds_copy16(wbase + kb * 128, ow[q], lb + (16 * wave + 8 * q) * kGRowBytes);
#pragma unroll
    for (int q = 0; q <= kX; ++q)
      if (q < kX || wave < kOdd) lds_copy16(a.xq + kb * 128, ox[q], lb + (16 * WAVES + 8 * (wave + WAVES * q)) * kGRowBytes);
  };
  f32x4 acc[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) acc[j] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int t = 0; t < RING - 1; ++t)
    if (t < kblocks) copy(t, t);
  int slot = 0;
  for (int t = 0; t < kblocks; ++t) {
    if (t % kWidePanel == 0) {
      if (t) __syncthreads();
      for (int e = threadIdx.x; e < kWidePanel * (16 * MT + 2); e += WAVES * kWave) {
        const int row = e / kWidePanel, b = e % kWidePanel;
        if (t + b >= kblocks) continue;
        const int kb = at(t + b);
        if (row < 16 * MT)
          sxp[b * 16 * MT + row] = sxs[(row < a.m ? row : a.m - 1) * (int64_t)kblocks + kb];
        else
          swp[2 * b + row - 16 * MT] = row == 16 * MT ? sgs[kb] : sus[kb];
      }
    }
    if (t + RING - 2 < kblocks) {
      if (wave < kOdd)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((RING - 2) * (3 + kX)) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((RING - 2) * (2 + kX)) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    __syncthreads();
    if (t + RING - 1 < kblocks) copy(t + RING - 1, slot == 0 ? RING - 1 : slot - 1);
    const uint8_t* As = smem + slot * kStage;
    slot = slot == RING - 1 ? 0 : slot + 1;
    const i32x8 wf = gated_frag(As, 16 * wave + r, g);
    const S* sp = sxp + (t % kWidePanel) * 16 * MT + r;
    const S sw = swp[2 * (t % kWidePanel) + up];
    if constexpr (POW2) {
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const i32x8 xf = gated_frag(As + 16 * WAVES * kGRowBytes, 16 * j + r, g);
        acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf, acc[j], 0, 0, 0, (int)sw, 0, (int)sp[16 * j]);
      }
    } else {
      f16x8 w16[4];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) w16[kk] = e4m3_f16x8(wf[2 * kk], wf[2 * kk + 1]);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const i32x8 xf = gated_frag(As + 16 * WAVES * kGRowBytes, 16 * j + r, g);
        f32x4 p = {0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w16[kk], e4m3_f16x8(xf[2 * kk], xf[2 * kk + 1]), p, 0, 0, 0);
        acc[j] += p * (sw * sp[16 * j]);
      }
    }
  }
  __syncthreads();
  f32x4* part = (f32x4*)smem;   // the ring is free
#pragma unroll
  for (int j = 0; j < MT; ++j) part[(wave * MT + j) * kWave + lane] = acc[j];
  __syncthreads();
  few_finish<MT, kRT, 1, WAVES, POW2>(a, n0, part, (int*)(smem + wide_lds<MT, WAVES, POW2>() - 64));
}

// The parts of K added in their order, and what the tiles' epilogue does: 32 lanes a segment of 128 columns.
__global__ __launch_bounds__(256) void gated_join_kernel(Gated a) {
  const int64_t nb = a.n / 128;
  const int64_t seg = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (seg >= a.m * nb) return;
  const int64_t row = seg / nb, col = (seg % nb) * 128 + 4 * (threadIdx.x & 31);
  const float* p = a.scratch + row * 2 * a.n + col;
  const int64_t each = a.m * 2 * a.n;
  f32x4 g = *(const f32x4*)p, u = *(const f32x4*)(p + a.n);
  for (int s = 1; s < a.split; ++s) {
    g += *(const f32x4*)(p + s * each);
    u += *(const f32x4*)(p + s * each + a.n);
  }
  const f32x4 h4 = gate_product4(g, u);
  const float h[4] = {h4[0], h4[1], h4[2], h4[3]};
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) top = umax(top, abs_bits(h[e]));
  auto out = [](uint16_t* q, float a0, float a1, float a2, float a3) {
    *(uint2*)q = make_uint2(pack_bf16x2_rne(a0, a1), pack_bf16x2_rne(a2, a3));
  };
  if (a.gu) {
    out(a.gu + row * 2 * a.n + col, g[0], g[1], g[2], g[3]);
    out(a.gu + row * 2 * a.n + a.n + col, u[0], u[1], u[2], u[3]);
  }
  if (a.h) out(a.h + row * a.n + col, h[0], h[1], h[2], h[3]);
  if (!a.hq) return;
  top = max_row16(top);
  top = umax(top, (uint32_t)__shfl_xor((int)top, 16));
  const Fp8Seg sc = a.pow2 ? fp8_seg_scale<true>(top) : fp8_seg_scale<false>(top);
  *(uint32_t*)(a.hq + row * a.n + col) = fp8_encode4(h, sc);
  if ((threadIdx.x & 31) == 0) {
    if (a.pow2)
      ((uint8_t*)a.sh)[seg] = (uint8_t)sc.stored;
    else
      ((uint32_t*)a.sh)[seg] = sc.stored;
  }
}

constexpr int64_t kFewM = 64;
constexpr int64_t kGCUs = 256;

// Up to 64 tokens: the wide kernel from 8192 columns on, where each CU has a workgroup, and above 16 tokens from
// 5120 on (5120 x 2048: 16 tokens 11.0 us against the other's 10.9, 64 tokens 15.3 against 19.8; 8192 x 4096:
// one token 18.2 against 17.7, 64 tokens 24 against 36).  Of its two widths the one that leaves the fullest CU
// less; if they do alike, the greater, which reads the tokens half as often (powers of two, 64 tokens: 14336 x 4096
// 28.8 us against 33.4, 28672 x 4096 50 against 64; 48 tokens, 18944 x 3584 38.0 against 36.9).
template <int MT>
hipError_t launch_few(const Gated& a, hipStream_t s) {
  if (a.n < (a.m > 16 ? 20 : 32) * kGCUs) {
    const unsigned grid = (unsigned)(a.n / 16);
    if (a.pow2)
      gated_few_kernel<MT, true><<<grid, kFewWaves * kWave, 0, s>>>(a);
    else
      gated_few_kernel<MT, false><<<grid, kFewWaves * kWave, 0, s>>>(a);
    return hipGetLastError();
  }
  auto go = [&](auto kernel, int waves, size_t lds) {
    hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    kernel<<<(unsigned)(a.n / (8 * waves)), waves * kWave, lds, s>>>(a);
    return hipGetLastError();
  };
  if ((a.n / 32 + kGCUs - 1) / kGCUs < 2 * ((a.n / 64 + kGCUs - 1) / kGCUs))
    return a.pow2 ? go(gated_wide_kernel<MT, 4, true>, 4, wide_lds<MT, 4, true>())
                  : go(gated_wide_kernel<MT, 4, false>, 4, wide_lds<MT, 4, false>());
  return a.pow2 ? go(gated_wide_kernel<MT, 8, true>, 8, wide_lds<MT, 8, true>())
                : go(gated_wide_kernel<MT, 8, false>, 8, wide_lds<MT, 8, false>());
}

// How more than 64 tokens are cut.  Tiles that cannot fill the chip are taken small, and if K is long, cut along
// it: a tile's time then is that of its copies' latency, block by block.  Otherwise the height with the least
// time for all rounds of the chip, a tile's time being its tokens and a share for the weights, which every
// height reads (and, with float32 scales, converts) alike: K 5120, powers of two 64 / 128 / 256 tokens 31 / 41 /
// 68 us a round, share 80; float32 64 / 128 / 192 tokens 60 / 79 / 100 us, share 96.
struct GatedPlan {
  int tm;
  int split;
  int64_t blocks_each;
};
GatedPlan plan_gated(int64_t m, int64_t n, int64_t k, bool pow2) {
  const int64_t nb = n / 128, kb = k / 128;
  const int64_t small = (m + 63) / 64 * nb;
  int64_t sp = small <= kGCUs / 2 ? kGCUs / small : 1;
  if (sp > kb / 4) sp = kb / 4;
  if (sp > 1) {
    const int64_t each = ((kb + sp - 1) / sp + 3) / 4 * 4;   // whole units of four blocks' scales
    return {64, (int)((kb + each - 1) / each), each};
  }
  const int high = pow2 ? 256 : 192, share = pow2 ? 80 : 96;
  int best = 64;
  int64_t least = INT64_MAX;
  for (int tm : {64, 128, high}) {
    const int64_t t = (((m + tm - 1) / tm * nb + kGCUs - 1) / kGCUs) * (tm + share);
    if (t < least) {
      least = t;
      best = tm;
    }
  }
  return {best, 1, kb};
}

// TM tokens a tile; `four`: the scales of four K blocks lie in one aligned unit.
template <int TM>
hipError_t launch_tiles(Gated a, hipStream_t s) {
  a.tiles_m = (a.m + TM - 1) / TM;
  a.tiles_n = a.n / kGCols;
  const unsigned grid = (unsigned)(a.tiles_m * a.tiles_n * a.split);
  const uintptr_t all = (uintptr_t)a.sx | (uintptr_t)a.sg | (uintptr_t)a.su;
  const bool four = (a.k / 128) % 4 == 0 && (all & (a.pow2 ? 3 : 15)) == 0;
  auto go = [&](auto kernel, int threads, size_t lds) {
    hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    kernel<<<grid, threads, lds, s>>>(a);
    if (a.split > 1) gated_join_kernel<<<(unsigned)((a.m * (a.n / 128) + 7) / 8), 256, 0, s>>>(a);
    return hipGetLastError();
  };
  if constexpr (TM <= 192) {
    if (!a.pow2)
      return four ? go(gated_f32s_kernel<TM / 64, true>, kGfThreads, gf_lds<TM / 64>())
                  : go(gated_f32s_kernel<TM / 64, false>, kGfThreads, gf_lds<TM / 64>());
  }
  if constexpr (TM != 192)
    return four ? go(gated_pow2_kernel<TM, true>, kGpThreads, gp_lds<TM>())
                : go(gated_pow2_kernel<TM, false>, kGpThreads, gp_lds<TM>());
  return hipErrorInvalidValue;
}

}  // namespace

bool gated_launchable(int64_t m, int64_t n, int64_t k) {
  if (m <= 0 || n <= 0 || k <= 0 || n % 128 || k % 128 || k >= kFp8MaxK) return false;
  // counters of the few-token kernel, and its 32-bit scratch offsets
  if (m <= kFewM) return n / 128 <= (int64_t)((kWsReserved - kWsCounterOff) / 4) && m * n < (int64_t(1) << 29);
  for (const bool pow2 : {false, true}) {   // fewer than 2^32 threads
    const GatedPlan p = plan_gated(m, n, k, pow2);
    if ((m + p.tm - 1) / p.tm * (n / 128) * p.split >= (int64_t(1) << 32) / 512) return false;
  }
  return true;
}

size_t gated_scratch_bytes(int64_t m, int64_t n, int64_t k) {
  if (m <= kFewM) return (size_t)(m * n) * 4;
  const int split = plan_gated(m, n, k, false).split;   // (the same for both kinds of scales)
  return split > 1 ? (size_t)split * (size_t)m * 2 * n * 4 : 0;
}

hipError_t launch_gated(Gated a, hipStream_t s) {
  if (!gated_launchable(a.m, a.n, a.k)) return hipErrorInvalidValue;
  a.split = 1;
  if (a.m <= 16) return launch_few<1>(a, s);
  if (a.m <= 32) return launch_few<2>(a, s);
  if (a.m <= 48) return launch_few<3>(a, s);
  if (a.m <= kFewM) return launch_few<4>(a, s);
  const GatedPlan p = plan_gated(a.m, a.n, a.k, a.pow2);
  a.split = p.split;
  a.blocks_each = p.blocks_each;
  if (p.tm == 64) return launch_tiles<64>(a, s);
  if (p.tm == 128) return launch_tiles<128>(a, s);
  return a.pow2 ? launch_tiles<256>(a, s) : launch_tiles<192>(a, s);
}

}  // namespace ql
