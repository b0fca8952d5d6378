// Backward pass of the gated feed-forward block on FP8 weights, gfx950 (FP8 forward, BF16 backward:
// rapidrecap.app Jet-RL summary, "Key Points").  With s = 1 / (1 + exp(-g)):
//
//   dg = dh u s (1 + g (1 - s)),  du = dh g s
//   dx = dg Wg + du Wu,   dWg = dg^T x,   dWu = du^T x
//
// First a kernel forms dg and du side by side (D, [m][2 n]) and makes the weights' scales ready, then two
// matrix products follow.  D is formed once in float32 and held twice: as f16 rows scaled by powers of two for dx
// (its rounding, 2^-11, is far below that of a bf16 result; the weights meet it as f16 too, E4M3 values
// times their scales rounded once more), and as bf16 for the weights' gradients, whose sums run over
// tokens of any size, so that a row's factor could not be taken out.
#include <type_traits>

#include "common.hpp"
#include "gate.hpp"
#include "gemm_common.hpp"
#include "launch.hpp"

namespace ql {

namespace {

constexpr int kBCols = 256;                 // columns (k) of an output tile
constexpr int kBStep = 32;                  // depth of a step: one MFMA deep
constexpr int kBThreads = 256;
constexpr int kBPitch = 272;                // output staging: bytes per row of 128 bf16 columns
constexpr int kBPBytes = kBCols * kBStep * 2;      // P of one step, 16 bits an element
constexpr int kBCodeBytes = kBCols * kBStep;
constexpr int kBScaleBytes = 1024;          // one word a thread

__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}

// ---------------------------------------------------------------------- scales of the weights
// For each 128 columns of k the power of two 2^E that puts the largest of the 2 n / 128 scales in
// [32, 64): then every weight is an f16 (448 * 64 < 2^15), normal down to 2^-20 of the largest scale.  tab
// [2 n / 128][k / 128] holds f16(scale * 2^-E) twice in a word, cols [k / 128] E.
struct WeightScales {
  const void* sg;
  const void* su;
  int pow2;
  int64_t nb, kb;       // n / 128, k / 128
  uint32_t* tab;
  int32_t* cols;
};
template <int T>
__device__ __forceinline__ void weight_scales(const WeightScales& a, int64_t c, uint32_t* red) {
  auto scale = [&](int64_t i) {
    const void* s = i < a.nb ? a.sg : a.su;
    const int64_t at = (i < a.nb ? i : i - a.nb) * a.kb + c;
    if (!a.pow2) return ((const float*)s)[at];
    const uint32_t b = ((const uint8_t*)s)[at];
    return b == 255 ? __uint_as_float(0x7FC00000u) : b == 0 ? 0x1p-127f : __uint_as_float(b << 23);
  };
  uint32_t top = 0;
  for (int64_t i = threadIdx.x; i < 2 * a.nb; i += T) top = umax(top, __float_as_uint(scale(i)) & 0x7FFFFFFFu);
  top = max_block<T>(top, red);
  const int e = top >= 0x7F800000u ? 0 : (int)(top >> 23) - 127 - 5;
  for (int64_t i = threadIdx.x; i < 2 * a.nb; i += T) {
    const float s = __builtin_amdgcn_ldexpf(scale(i), -e);
    a.tab[i * a.kb + c] = f16_pair(s, s);
  }
  if (threadIdx.x == 0) a.cols[c] = e;
}

// --------------------------------------------------------------------------------- D
struct GateGrad {
  const uint16_t* dh;   // [m][n]
  const uint16_t* gu;   // [m][2 n]
  int64_t m, n, m_pad;
  uint16_t* d16;        // f16 [2 n / 32][m][32], or null
  int32_t* rs;          // [m]: exponents of the rows' factors, which dx takes off again
  uint16_t* db;         // bf16 [m_pad][2 n], rows past m zero, or null
  const uint16_t* x;    // with db: [m][k], whose last m % 32 rows go to xt [32][k], the others there zero
  uint16_t* xt;
  int64_t k;
  WeightScales ws;      // with d16: its kb workgroups come first
};

// T threads a row, NV units of 8 columns each in registers (NV 0: any n, read twice, the second
// time from the caches: 8192 x 18944 461 us, 2.2 GB at 4.7 TB/s).  Bound by memory:
// 6 bytes read, 4 or 8 written a column of h; eight waves a SIMD, so that two workgroups of 1024 threads share a CU.
template <int T, int NV>
__global__ __launch_bounds__(T, 8) void gate_grad_kernel(GateGrad a) {
  __shared__ uint32_t red[T / kWave];
  const int64_t scales = a.d16 ? a.ws.kb : 0;
  if (blockIdx.x < scales) {
    weight_scales<T>(a.ws, blockIdx.x, red);
    return;
  }
  // Neighbouring rows share lines of d16: they go to one XCD, whose cache puts the lines together (8192 x 14336: 351
  // us, 1.73 GB at 4.9 TB/s; 386 with the rows dealt out one by one).
  const int64_t b = blockIdx.x - scales, rows = gridDim.x - scales, whole = rows / 8 * 8;
  const int64_t row = b < whole ? gemm_xcd_remap(b, whole) : b;
  const int64_t units = a.n / 8;
  const int t = threadIdx.x;
  if (a.db && a.m_pad != a.m && row >= a.m_pad - kBStep) {   // the last step of the weights' gradients is not full
    uint16_t* p = a.xt + (row - (a.m_pad - kBStep)) * a.k;
    for (int64_t u = t; u < a.k / 8; u += T)
      *(uint4*)(p + u * 8) = row < a.m ? *(const uint4*)(a.x + row * a.k + u * 8) : make_uint4(0, 0, 0, 0);
    if (row >= a.m) {
      for (int64_t u = t; u < 2 * units; u += T) *(uint4*)(a.db + row * 2 * a.n + u * 8) = make_uint4(0, 0, 0, 0);
      return;
    }
  }
  const uint16_t* ph = a.dh + row * a.n;
  const uint16_t* pg = a.gu + row * 2 * a.n;
  auto highest = [](const float (&dg)[8], const float (&du)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      top = umax(top, umax(__float_as_uint(dg[e]) & 0x7FFFFFFFu, __float_as_uint(du[e]) & 0x7FFFFFFFu));
    return top;
  };
  auto store = [&](int64_t u, const float (&dg)[8], const float (&du)[8], int e) {
    if (a.db) {
      uint16_t* p = a.db + row * 2 * a.n + u * 8;
      *(uint4*)p = make_uint4(pack_bf16x2_rne(dg[0], dg[1]), pack_bf16x2_rne(dg[2], dg[3]),
                              pack_bf16x2_rne(dg[4], dg[5]), pack_bf16x2_rne(dg[6], dg[7]));
      *(uint4*)(p + a.n) = make_uint4(pack_bf16x2_rne(du[0], du[1]), pack_bf16x2_rne(du[2], du[3]),
                                      pack_bf16x2_rne(du[4], du[5]), pack_bf16x2_rne(du[6], du[7]));
    }
    if (a.d16) {
      uint16_t* p = a.d16 + ((u >> 2) * a.m + row) * 32 + (u & 3) * 8;
      auto pair = [&](const float (&d)[8], int i) {
        return f16_pair(__builtin_amdgcn_ldexpf(d[i], e), __builtin_amdgcn_ldexpf(d[i + 1], e));
      };
      *(uint4*)p = make_uint4(pair(dg, 0), pair(dg, 2), pair(dg, 4), pair(dg, 6));
      *(uint4*)(p + a.n * a.m) = make_uint4(pair(du, 0), pair(du, 2), pair(du, 4), pair(du, 6));
    }
  };
  // the exponent of the power of two that puts the row's largest value in [2^14, 2^15)
  auto factor = [&](uint32_t top) {
    top = max_block<T>(top, red);
    const int e = top == 0 || top >= 0x7F800000u ? 0 : 14 - ((int)(top >> 23) - 127);
    if (t == 0 && a.rs) a.rs[row] = -e;
    return e;
  };
  if constexpr (NV > 0) {
    float dg[NV][8], du[NV][8];
    uint4 g[NV], u[NV], h[NV];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)i * T + t;
      const bool in = c < units;
      g[i] = in ? *(const uint4*)(pg + c * 8) : make_uint4(0, 0, 0, 0);
      u[i] = in ? *(const uint4*)(pg + a.n + c * 8) : make_uint4(0, 0, 0, 0);
      h[i] = in ? *(const uint4*)(ph + c * 8) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      gate_grad8(g[i], u[i], h[i], dg[i], du[i]);
      top = umax(top, highest(dg[i], du[i]));
    }
    const int e = factor(top);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)i * T + t;
      if (c < units) store(c, dg[i], du[i], e);
    }
  } else {
    uint32_t top = 0;
    float dg[8], du[8];
    for (int64_t c = t; c < units; c += T) {
      gate_grad8(*(const uint4*)(pg + c * 8), *(const uint4*)(pg + a.n + c * 8), *(const uint4*)(ph + c * 8), dg, du);
      top = umax(top, highest(dg, du));
    }
    const int e = factor(top);
    for (int64_t c = t; c < units; c += T) {
      gate_grad8(*(const uint4*)(pg + c * 8), *(const uint4*)(pg + a.n + c * 8), *(const uint4*)(ph + c * 8), dg, du);
      store(c, dg, du, e);
    }
  }
}

// ------------------------------------------------------------------------------ weights, turned
// For many tokens: both weights as f16 [2 n / 32][k][32], times their scales from tab.  A workgroup takes 128 x 128 codes; a
// thread 8 rows by 4 columns, whose bytes v_perm_b32 turns into 4 columns of 8.  Bound by memory (1 byte read, 2
// written a weight): 103 us for 2 x 14336 x 4096, which the product gains back from about 2800 tokens on.
__global__ __launch_bounds__(256) void gated_weights_kernel(const uint8_t* __restrict__ wg, const uint8_t* __restrict__ wu,
                                                            const uint32_t* __restrict__ tab, int64_t n, int64_t k,
                                                            uint16_t* __restrict__ w16) {
  const int64_t z0 = (int64_t)blockIdx.y * 128, k0 = (int64_t)blockIdx.x * 128;
  const uint8_t* w = z0 < n ? wg + z0 * k : wu + (z0 - n) * k;
  const f16x2 sc = __builtin_bit_cast(f16x2, tab[(z0 / 128) * (k / 128) + k0 / 128]);
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int z = 64 * (wave & 1) + 8 * (lane & 7), c = 32 * (2 * q + (wave >> 1)) + 4 * (lane >> 3);
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = *(const uint32_t*)(w + (int64_t)(z + e) * k + k0 + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) {   // column c + e: byte e of the eight rows
      const uint32_t pick = 0x0C0C0400u + (uint32_t)e * 0x0101u;   // (byte e of the second operand, then of the first)
      uint32_t out[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint32_t two = __builtin_amdgcn_perm(v[2 * h + 1], v[2 * h], pick);
        out[h] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(two, 1.0f, false) * sc);
      }
      *(uint4*)(w16 + ((z0 + z) / 32 * k + k0 + c + e) * 32 + z % 32) = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
}

// ------------------------------------------------------------------------------ products
// out[row][k] = 2^(rs[row] + cols[k / 128]) * sum over z of P[z][k] Q[z][row]   (kDw: without the factor)
//   kDx:  rows are tokens, z the 2 n weight rows: P the weights (E4M3 in memory, f16 from there), Q = D16 in steps,
//         [z / 32][row][32], so that what a step reads of 256 rows is one piece of whole lines
//   kDxT: the same with P = the weights as f16 [z / 32][k][32], turned by gated_weights_kernel beforehand
//   kDw:  rows are the 2 n weight rows, z tokens: P = x [z][k], Q = Db [z][row], bf16
// Tiles of 256 k x 256 rows by four waves (2 x 2) of 128 x 128 each: 64 MFMAs of 16x16x32 for 16 fragments
// a step, which leaves half of LDS's read rate free.  P is the MFMA's A operand, so a lane's four results
// lie side by side along k.  Operands whose z is not contiguous in memory are kept in LDS as they come
// ([z][256], 512-byte rows) and read with the transposing read (four z of a lane's column each).
// A step is four quarters of 16 MFMAs (4 fragments of each operand): P low Q low, P high Q low, P high Q high,
// P low Q high.  Each quarter reads the four fragments that are new in a later one, over those that no
// MFMA needs any more, so LDS, which the four waves' fragments keep busy for half of a step's time and the
// copies for a quarter, is read evenly.  The barrier stands in the middle: there every fragment of step s is read
// and step s + 1 has landed, so that from there to the next middle the copies of s + RING go into the place of s.
// kDx: the codes of s + 2 have landed too, and each lane turns those that it copied itself into f16 from this
// middle to the next.
// A wave alone on its SIMD issues an instruction in about five cycles (measured: MFMAs of 16x16x32, 16
// cycles, keep their rate beside one other instruction each and lose a quarter beside two): so every
// other instruction has a place behind an MFMA, and there are few of them -- copies by four with one base, the
// ring's places constants of an unrolled loop.  (32x32x16 MFMAs leave more room and took a fifth fewer cycles, but
// move their sums twice as often for the same work: the card's power lowered the clock from 1.9 to 1.5 GHz and the
// time rose by a tenth.)
// NJ: Q fragments of a wave.  8 (tiles of 256 rows, one wave a SIMD) for depth; 4 (128 rows) has half the sums
// -- two halves of 16 MFMAs a step, P low and P high -- for few tokens (kDx), or so that two workgroups share a CU
// and one's start and end, most of the time of a few steps, run beside the other's products (kDw).
enum Kind { kDw, kDx, kDxT };
struct GatedProduct {
  const uint8_t* codes[2];   // kDx: gate and up, E4M3 [n][k]
  const uint32_t* tab;       // kDx: [2 n / 128][k / 128] f16 scale twice
  const uint16_t* p;         // kDw: x [z][k]; kDxT: the weights, f16 [z / 32][k][32]
  const uint16_t* xt;        // kDw: x's last step, rows past the last token zero, where z is no multiple of 32
  const uint16_t* q;         // D16 [z / 32][rows][32], or Db [z padded][rows]
  const int32_t* rs;         // kDx, kDxT: [rows]
  const int32_t* cols;       // the same: [k / 128]
  int64_t rows, z, n, k;     // z: 2 n, or tokens; n: rows of one weight
  uint16_t* out[2];          // kDx, kDxT: dx twice; else the gate's and the up projection's gradient
  int64_t tiles_r, tiles_c, full;
  int32_t split;
  int32_t tile_rows;         // 32 NJ
  float* part;               // [split workgroup][tile_rows][256 k]
};

// 16-byte slot of logical slot s in LDS row z (32 slots of 512 bytes).  A transposing read of 32 lanes
// covers eight rows (z & 3 and bit 3 vary) by 32 bytes, which slot bits 1..3 spread over the banks; a write
// of even slots of one row and the row two below takes odd ones in the second half and in the lower row.
__device__ __forceinline__ int zslot(int z, int s) { return s ^ (((s >> 4) ^ (z >> 1)) & 1) ^ (2 * ((z & 3) | ((z >> 1) & 4))); }

// The same for rows of 256 bytes (16 slots).
__device__ __forceinline__ int qslot(int z, int s) { return s ^ (2 * ((z & 3) | ((z >> 1) & 4))); }
// The 16-byte slot of a 64-byte row of D that holds slot 0, by bits 2 and 3 of the row: 16-byte reads of one slot of
// 16 rows go over LDS as rows 0..3 and 12..15 of one slot with 4..11 of the next, which these four keep apart.
__device__ __forceinline__ int dslot(int q) { return ((q << 1) ^ (q & 2 ? 3 : 0)) & 3; }

// At most N of the copies under way are left.
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Workgroup b of a product's: whole tiles first, then the parts of the split ones.
__device__ __forceinline__ GemmWork product_work(const GatedProduct& a, int64_t b) {
  GemmWork w;
  int64_t t;
  if (b < a.full) {
    t = gemm_xcd_remap(b, a.full);
    w.slot = -1;
    w.split = 0;
    w.nsplit = 1;
  } else {
    const int64_t tail = a.tiles_r * a.tiles_c - a.full, at = b - a.full;
    if (a.split % 8 == 0) {   // workgroups go to the eight XCDs in turn: an XCD takes a part of z of every tile
      w.split = (int)(at % 8 + 8 * (at / 8 / tail));
      t = at / 8 % tail;
    } else {
      w.split = (int)(at % a.split);
      t = at / a.split;
    }
    w.slot = t * a.split + w.split;
    t += a.full;
    w.nsplit = a.split;
  }
  gemm_group_tile(t, a.tiles_r, a.tiles_c, w.tm, w.tn);
  return w;
}

// LDS of a kind: slots of P and Q together; kDx: ring of Q, ring of codes, two steps of weights in f16, ring of scale
// words.  The output's staging takes the same place.
template <Kind KIND, int NJ>
struct Lds {
  static constexpr int kRing = KIND == kDw && NJ == 4 ? 3 : 4;
  static constexpr int kQBytes = 32 * NJ * kBStep * 2;
  static constexpr int kQOff = KIND == kDx ? 0 : kBPBytes;
  static constexpr int kSlot = KIND == kDx ? kQBytes : kBPBytes + kQBytes;
  static constexpr int kCodeOff = kRing * kSlot, kWOff = kCodeOff + kRing * kBCodeBytes, kScaleOff = kWOff + 2 * kBPBytes;
  static constexpr int kStage = 16 * NJ * kBPitch;   // of a wave's output
  static constexpr int kLoop = KIND == kDx ? kScaleOff + kRing * kBScaleBytes : kRing * kSlot;
  static constexpr int kBytes = kLoop > 4 * kStage ? kLoop : 4 * kStage;
};

template <Kind KIND, int NJ>
__device__ __forceinline__ void gated_product(const GatedProduct& a, int64_t b, uint8_t* smem) {
  using L = Lds<KIND, NJ>;
  constexpr bool FUSED = KIND == kDx, TURNED = KIND == kDxT, DW = KIND == kDw;
  constexpr int kRows = 32 * NJ, kWRows = 16 * NJ;      // rows of a tile, of a wave
  const GemmWork work = product_work(a, b);
  const int64_t c0 = (int64_t)__builtin_amdgcn_readfirstlane((int)work.tn) * kBCols;
  const int64_t r0 = (int64_t)__builtin_amdgcn_readfirstlane((int)work.tm) * kRows;
  const int part_no = __builtin_amdgcn_readfirstlane(work.split);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int wk = wave & 1, wr = wave >> 1;
  const int r = lane & 15, g = lane >> 4;
  const int steps = (int)((a.z + kBStep - 1) / kBStep);
  const int nsplit = __builtin_amdgcn_readfirstlane(work.nsplit);
  const int per = (steps + nsplit - 1) / nsplit;
  const int st0 = part_no * per;
  const int st1 = st0 + per < steps ? st0 + per : steps;
  const int64_t c_room = a.k - c0;         // at least 128
  const int64_t r_last = a.rows - 1 - r0;
  auto clamp_st = [&](int st) { return st < st1 ? st : st1 - 1; };
  const uint32_t lds0 = lds_addr(smem);

  // ---- copies of a step, the same by every wave, from uniform addresses with a lane's 32-bit offsets
  //   P  kDx: weight rows 8 wave + 4 c + lane / 16 (two copies, 16 codes a lane), and a scale word for a lane's codes
  //      kDxT: columns of k 64 wave + 16 c + lane / 4, 16-byte slot lane % 4
  //      kDw: x rows (z) 8 wave + 2 c + lane / 32, slot lane % 32
  //   Q  kDx, kDxT: D rows 8 NJ wave + 16 c + lane / 4, slot lane % 4; kDw: D rows (z) of 2 kRows bytes
  constexpr int kQCopies = NJ / 2;
  constexpr int kCopies = (FUSED ? 3 : 4) + kQCopies;
  constexpr uint32_t kUp = 3 * 1024;     // see lds_copy16x4
  uint32_t op[4], od[4], osc = 0;
  {
    // columns past k: the 128 before
    const int col = 16 * (lane & 15) < c_room ? 16 * (lane & 15) : 16 * (lane & 15) - 128;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (DW) {
        const int z = 8 * wave + 2 * c + (lane >> 5), s = zslot(z, lane & 31);     // (its own inverse)
        op[c] = (uint32_t)(z * a.k * 2 + (8 * s < c_room ? 8 * s : 8 * s - 128) * 2) + kUp - 1024 * c;
        const int zq = NJ == 8 ? z : 8 * wave + 4 * (c & 1) + (lane >> 4);
        od[c] = (uint32_t)(zq * a.rows * 2 + (NJ == 8 ? s : qslot(zq, lane & 15)) * 16) + kUp - 1024 * (NJ == 8 ? c : c & 1);
      } else {
        const int in = ((lane & 3) ^ dslot(lane >> 4)) * 16;
        const int prow = 64 * wave + 16 * c + (lane >> 2), qrow = 8 * NJ * wave + 16 * c + (lane >> 2);
        op[c] = TURNED ? (uint32_t)((prow < c_room ? prow : prow - 128) * 64 + in) + kUp - 1024 * c
                       : (uint32_t)((8 * wave + 4 * (c & 1) + (lane >> 4)) * a.k + col) + kUp - 1024 * (c & 1);
        od[c] = (uint32_t)((qrow < r_last ? qrow : r_last) * 64 + in) + kUp - 1024 * c;
      }
    }
    osc = (uint32_t)(col / 128 * 4);
  }
  const int whole = DW ? (int)(a.z / kBStep) : steps;   // steps of whole rows of x
  // (sizes in 32 bits: a 64-bit product is two scalar instructions then, not seven)
  const uint32_t k32 = (uint32_t)a.k, rows32 = (uint32_t)a.rows, n32 = (uint32_t)a.n;
  auto from_p = [&](int st) {
    const uint32_t z0 = (uint32_t)st * kBStep;
    if (FUSED) {
      const bool up = z0 >= n32;
      return (up ? a.codes[1] : a.codes[0]) + (uint64_t)(up ? z0 - n32 : z0) * k32 + c0 - kUp;
    }
    if (TURNED) return (const uint8_t*)(a.p + ((uint64_t)(uint32_t)st * k32 + c0) * kBStep) - kUp;
    return (const uint8_t*)((st < whole ? a.p + (uint64_t)z0 * k32 : a.xt) + c0) - kUp;
  };
  auto from_d = [&](int st) {
    return (const uint8_t*)(a.q + (DW ? (uint64_t)((uint32_t)st * kBStep) * rows32 + r0 : ((uint64_t)(uint32_t)st * rows32 + r0) * kBStep)) - kUp;
  };
  auto copy_p = [&](const uint8_t* src, int slot) {
    if (FUSED)
      lds_copy16x2(src, op[0], op[1], lds0 + L::kCodeOff + slot * kBCodeBytes + wave * 2048);
    else
      lds_copy16x4(src, op[0], op[1], op[2], op[3], lds0 + slot * L::kSlot + wave * 4096);
  };
  auto copy_sc = [&](int st, int slot) {
    lds_copy4((const uint8_t*)(a.tab + ((uint32_t)st / (128 / kBStep)) * (k32 / 128) + c0 / 128), osc,
              lds0 + L::kScaleOff + slot * kBScaleBytes + wave * 256);
  };
  auto copy_d = [&](const uint8_t* src, int slot) {
    const uint32_t dst = lds0 + L::kQOff + slot * L::kSlot + wave * 512 * NJ;
    if (NJ == 8)
      lds_copy16x4(src, od[0], od[1], od[2], od[3], dst);
    else
      lds_copy16x2(src, od[0], od[1], dst);
  };

  // ---- kDx: the step's weights from codes to f16, 32 a thread, those that the thread itself copied
  auto read_codes = [&](int slot, int c) {
    return *(const i32x4*)(smem + L::kCodeOff + slot * kBCodeBytes + (8 * wave + 4 * c + (lane >> 4)) * 256 + 16 * (lane & 15));
  };
  auto read_scale = [&](int slot) {
    return __builtin_bit_cast(f16x2, *(const uint32_t*)(smem + L::kScaleOff + slot * kBScaleBytes + wave * 256 + 4 * lane));
  };
  f16x2 wv[4];
  int wo[2][2];   // where a thread's pieces of 8 go
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int z = 8 * wave + 4 * c + (lane >> 4);
      wo[c][h] = z * 512 + zslot(z, 2 * (lane & 15) + h) * 16;
    }
  auto dequant = [&](const i32x4& w, const f16x2& sc, int buf, int c, int q) {   // piece q of ten of one 16-code unit
    const int h = q / 5, e = q % 5;
    if (e < 4) {
      wv[e] = (e & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((unsigned)w[2 * h + (e >> 1)], 1.0f, true)
                     : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((unsigned)w[2 * h + (e >> 1)], 1.0f, false)) * sc;
      return;
    }
    *(f16x8*)(smem + wo[c][h] + L::kWOff + buf * kBPBytes) =
        f16x8{wv[0][0], wv[0][1], wv[1][0], wv[1][1], wv[2][0], wv[2][1], wv[3][0], wv[3][1]};
  };

  // ---- fragments: lane (r, g) has z 8 g .. 8 g + 7 of column (or row) r.  Transposing reads: lanes 4 e + b name row
  // 8 g + 4 q + e, columns 4 b .. 4 b + 3, and receive rows 8 g + 4 q + (0 .. 3) of column r.
  const int te = r >> 2, tb = r & 3, tz = 8 * g + te;
  int ta[8], tq[NJ];   // fragment i flips bits 5 .. 7 of fragment 0's place
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int in = 16 * i * 64 + r * 64 + (g ^ dslot(r >> 2)) * 16;
    ta[i] = TURNED ? 128 * wk * 64 + in : (tz * 512 + zslot(tz, 16 * wk + (tb >> 1)) * 16 + (tb & 1) * 8) ^ (i << 5);
    if (i < NJ) {
      const int z0 = NJ == 8 ? tz * 512 + zslot(tz, 16 * wr + (tb >> 1)) * 16 : tz * 256 + qslot(tz, 8 * wr + (tb >> 1)) * 16;
      tq[i < NJ ? i : 0] = L::kQOff + (DW ? (z0 + (tb & 1) * 8) ^ (i << 5) : kWRows * wr * 64 + in);
    }
  }
  auto read_tr = [&](const uint8_t* p, int four) {   // four: bytes of four rows
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + four));
    return __builtin_bit_cast(i32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto read_p = [&](int s, int i) {
    if (TURNED) return *(const i32x4*)(smem + ta[i] + s % L::kRing * L::kSlot);
    return read_tr(smem + ta[i] + (FUSED ? L::kWOff + (s & 1) * kBPBytes : s % L::kRing * L::kSlot), 2048);
  };
  auto read_q = [&](int s, int j) {
    if (!DW) return *(const i32x4*)(smem + tq[j] + s % L::kRing * L::kSlot);
    return read_tr(smem + tq[j] + s % L::kRing * L::kSlot, 8 * kRows);
  };
  auto mfma = [](const i32x4& x, const i32x4& y, const f32x4& c) {
    if (!DW) return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
  };

  f32x4 acc[8][NJ];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  i32x4 pf[8], qf[NJ], cw = {0, 0, 0, 0};
  f16x2 sc = {0, 0};
  // Copies that may be under way at a step's middle: those of the steps behind the next (kDx: but for the codes and scale
  // of the first of them, three copies).
  constexpr int kAhead = (L::kRing - 2) * kCopies - (FUSED ? 3 : 0);
  if (st1 > st0) {
#pragma unroll
    for (int s = 0; s < L::kRing; ++s) {
      copy_p(from_p(clamp_st(st0 + s)), s);
      if (FUSED) copy_sc(clamp_st(st0 + s), s);
      copy_d(from_d(clamp_st(st0 + s)), s);
    }
    // step 0 (kDx: and step 1's codes and scales)
    __builtin_amdgcn_sched_barrier(0);
    wait_copies<kAhead + kCopies>();
    if (FUSED) {
#pragma unroll
      for (int u = 0; u < 3; ++u) {   // all of step 0, half of step 1
        sc = read_scale(u >> 1);
        cw = read_codes(u >> 1, u & 1);
#pragma unroll
        for (int q = 0; q < 10; ++q) dequant(cw, sc, u >> 1, u & 1, q);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < 3 || NJ == 4) pf[i] = read_p(0, i);
      if (i < 3 || NJ == 8) qf[i] = read_q(0, i);
    }
  }
  // One step, the U-th of each turn of the ring (its places are then constants); true if it was the last.  For kDx the
  // turn is even, so that the two places of the weights are constants as well.
  auto step = [&](auto U, int st) {
    constexpr int s = decltype(U)::value;
    const int ahead = clamp_st(st + L::kRing);
    constexpr int kParts = NJ / 2;     // quarters or halves
    const uint8_t* src = nullptr;
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
      const bool late = h >= kParts / 2;
      if (h == kParts / 2) {
        wait_copies<kAhead>();
        __syncthreads();
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        if (NJ == 8) {
          const int i = (h == 1 || h == 2 ? 4 : 0) + x / 4, j = (h >= 2 ? 4 : 0) + x % 4;
          acc[i][j] = mfma(pf[i], qf[j], acc[i][j]);
          if (h == 0) {
            if (x == 0) pf[3] = read_p(s, 3);
            if (x == 2 || x == 5 || x == 8 || x == 11) pf[4 + x / 3] = read_p(s, 4 + x / 3);
          }
          if (h == 1 && x % 3 == 0 && x < 12) qf[4 + x / 3] = read_q(s, 4 + x / 3);
          if (h == 2 && x % 3 == 0 && x < 12) qf[x / 3] = read_q(s + 1, x / 3);
          if (h == 3 && x % 4 == 0 && x > 0) pf[x / 4 - 1] = read_p(s + 1, x / 4 - 1);
        } else {
          const int i = 4 * h + x % 4, j = x / 4;
          acc[i][j] = mfma(pf[i], qf[j], acc[i][j]);
          if (h == 0) {
            if (x == 0) qf[3] = read_q(s, 3);
            if (x == 2 || x == 5 || x == 8 || x == 11) pf[4 + x / 3] = read_p(s, 4 + x / 3);
          } else {
            if (x == 1 || x == 3 || x == 5 || x == 7) pf[x / 2] = read_p(s + 1, x / 2);
            if (x == 4 || x == 8 || x == 12) qf[x / 4 - 1] = read_q(s + 1, x / 4 - 1);
          }
        }
        // the copies of step s + kRing, their addresses a few places before
        if (NJ == 8 ? h == 2 && x == 1 : late && x == 0) src = from_p(ahead);
        if (NJ == 8 ? h == 2 && x == 5 : late && x == 2) copy_p(src, s % L::kRing);
        if (FUSED && (NJ == 8 ? h == 2 && x == 14 : late && x == 5)) copy_sc(ahead, s % L::kRing);
        if (NJ == 8 ? h == 3 && x == 2 : late && x == 9) src = from_d(ahead);
        if (NJ == 8 ? h == 3 && x == 7 : late && x == 11) copy_d(src, s % L::kRing);
        if (FUSED) {   // a unit of ten pieces in two quarters, or in a half
          const int d = late ? s + 2 : s + 1;
          if (h % (kParts / 2) == 0 && x == 1) {
            sc = read_scale(d % L::kRing);
            cw = read_codes(d % L::kRing, !late);
          }
          const int q = NJ == 4 ? (x >= 6 ? x - 6 : -1) : x == 9 ? 0 : x == 10 ? 1 : x == 12 ? 2 : x == 13 ? 3 : x == 15 ? 4 : -1;
          if (q >= 0) dequant(cw, sc, d & 1, !late, NJ == 4 ? q : q + 5 * (h & 1));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    return st + 1 >= st1;
  };
  for (int st = st0; st < st1; st += L::kRing) {
    if (step(std::integral_constant<int, 0>(), st) || step(std::integral_constant<int, 1>(), st + 1) ||
        step(std::integral_constant<int, 2>(), st + 2))
      break;
    if (L::kRing == 4 && step(std::integral_constant<int, 3>(), st + 3)) break;
  }
  wait_copies<0>();

  // lane: k = c0 + 128 wk + 16 i + 4 g + (0 .. 3), row r0 + kWRows wr + 16 j + r
  if (!DW) {
    // both exponents at once: the row's factor alone may leave float32's range where the result does not
    const int ce = a.cols[(128 * wk < c_room ? c0 + 128 * wk : c0) / 128];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int64_t row = r0 + kWRows * wr + 16 * j + r;
      const int e = a.rs[row < a.rows ? row : a.rows - 1] + ce;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_amdgcn_ldexpf(acc[i][j][q], e);
    }
  }
  if (work.slot >= 0) {   // a part of a tile's depth, added by gated_join_kernel
    float* pt = a.part + work.slot * (kRows * kBCols);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int row = kWRows * wr + 16 * j + r;
      if (r0 + row >= a.rows) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) *(f32x4*)(pt + row * kBCols + 128 * wk + 16 * i + 4 * g) = acc[i][j];
    }
    return;
  }
  __syncthreads();   // every wave is done with the operands
  uint8_t* stage = smem + wave * L::kStage;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const f32x4 v = acc[i][j];
      *(uint2*)(stage + (16 * j + r) * kBPitch + (16 * i + 4 * g) * 2) =
          make_uint2(pack_bf16x2_rne(v[0], v[1]), pack_bf16x2_rne(v[2], v[3]));
    }
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's LDS writes are done
  if (128 * wk >= c_room) return;
  // the wave's rows lie in one of the two outputs (n is a multiple of 128)
  const int64_t row0 = r0 + kWRows * wr;
  const int second = DW && row0 >= a.n;
  uint16_t* base = (second ? a.out[1] : a.out[0]) + (second ? row0 - a.n : row0) * a.k + c0 + 128 * wk + (lane & 15) * 8;
#pragma unroll
  for (int q = 0; q < 4 * NJ; ++q) {
    const int row = 4 * q + (lane >> 4);
    if (row0 + row >= a.rows) continue;
    const i32x4 v = *(const i32x4*)(stage + row * kBPitch + (lane & 15) * 16);
    // the weights' gradients, which nothing here reads again, past the caches (200 x 18944 x 3584: 92 -> 78 us, and the
    // parts of dx are still there when they are added, 14 -> 9)
    if (DW)
      __builtin_nontemporal_store(v, (i32x4*)(base + row * a.k));
    else
      *(i32x4*)(base + row * a.k) = v;
  }
}

template <Kind KIND, int NJ>
__global__ __launch_bounds__(kBThreads, KIND == kDw && NJ == 4 ? 2 : 1) void gated_product_kernel(GatedProduct a) {
  extern __shared__ __align__(16) uint8_t smem[];
  gated_product<KIND, NJ>(a, blockIdx.x, smem);
}
// dx and the weights' gradients side by side, where neither has enough tiles to fill the chip: a workgroup of a
// few steps takes some 12 us, most of it its start and end.
template <int NJ>
__global__ __launch_bounds__(kBThreads) void gated_both_kernel(GatedProduct dx, GatedProduct dw, unsigned first) {
  extern __shared__ __align__(16) uint8_t smem[];
  if (blockIdx.x < first)
    gated_product<kDx, NJ>(dx, blockIdx.x, smem);
  else
    gated_product<kDw, 8>(dw, blockIdx.x - first, smem);
}

// The parts of split tiles added in their order: 4 rows of a tile a workgroup, 4 columns a thread.
__device__ __forceinline__ void gated_join(const GatedProduct& a, int64_t b) {
  const int64_t per = a.tile_rows / 4, tail = b / per;
  const int row = (int)(b % per) * 4 + (int)(threadIdx.x >> 6);
  const int col = (int)(threadIdx.x & 63) * 4;
  int64_t tr, tc;
  gemm_group_tile(a.full + tail, a.tiles_r, a.tiles_c, tr, tc);
  const int64_t rr = tr * a.tile_rows + row, c = tc * kBCols + col;
  if (rr >= a.rows || c >= a.k) return;
  const int64_t each = (int64_t)a.tile_rows * kBCols;
  const float* p = a.part + tail * a.split * each + row * kBCols + col;
  f32x4 v = *(const f32x4*)p;
  for (int sp = 1; sp < a.split; ++sp) v += *(const f32x4*)(p + sp * each);
  const int second = rr >= a.n && a.out[1] != a.out[0];
  store4((second ? a.out[1] : a.out[0]) - (second ? a.n * a.k : 0), 0, a.k, rr, c, v, a.k);
}
__global__ __launch_bounds__(256) void gated_join_kernel(GatedProduct dx, GatedProduct dw, unsigned first) {
  if (blockIdx.x < first)
    gated_join(dx, blockIdx.x);
  else
    gated_join(dw, blockIdx.x - first);
}

// Tiles and how the ones behind the last full round of the chip are split along z.  More than eight parts come in
// eights, a part of every tile on one XCD.
struct ProductPlan {
  int64_t tiles_r = 0, tiles_c = 0, full = 0;
  int32_t split = 1, tile_rows = 256;
  int64_t tail() const { return split > 1 ? tiles_r * tiles_c - full : 0; }
  unsigned grid() const { return (unsigned)(full + tail() * split); }
  unsigned joins() const { return (unsigned)(tail() * (tile_rows / 4)); }
  size_t part_bytes() const { return (size_t)tail() * (size_t)split * (size_t)tile_rows * kBCols * 4; }
};
constexpr int64_t kBCUs = 256;
ProductPlan plan_product(int64_t rows, int64_t z, int64_t k, int tile_rows) {
  ProductPlan p;
  p.tile_rows = tile_rows;
  p.tiles_r = (rows + tile_rows - 1) / tile_rows;
  p.tiles_c = (k + kBCols - 1) / kBCols;
  const int64_t tiles = p.tiles_r * p.tiles_c, rem = tiles % kBCUs;
  const int64_t steps = (z + kBStep - 1) / kBStep;
  int64_t sp = rem > 0 && rem <= kBCUs / 2 ? kBCUs / rem : 1;
  if (sp > 32) sp = 32;
  if (sp > steps / 8) sp = steps / 8;
  if (sp > 8) sp = sp / 8 * 8;
  p.split = (int32_t)(sp > 1 ? sp : 1);
  p.full = p.split > 1 ? tiles - rem : tiles;
  return p;
}
// dx: tiles of 128 rows for up to 128 tokens (14336 x 4096, 64 tokens 52 us against 70 with half-empty ones of 256; 256
// tokens 88 against 82).
ProductPlan plan_dx(int64_t m, int64_t n, int64_t k) { return plan_product(m, 2 * n, k, m <= 128 ? 128 : 256); }
// The weights' gradients: few steps a tile and more than a round of tiles go two workgroups a CU, whose starts and
// ends then run beside one another (14336 x 4096, the whole call: 64 tokens 119 -> 109 us, 512 283 -> 266, 768 374 ->
// 372, 1024 455 -> 462).
constexpr int64_t kShallow = 512;
ProductPlan plan_dw(int64_t m, int64_t n, int64_t k) {
  const ProductPlan p = plan_product(2 * n, m, k, 256);
  if (m > kShallow || p.tiles_r * p.tiles_c <= kBCUs) return p;
  ProductPlan q = p;
  q.tile_rows = 128;
  q.tiles_r = 2 * n / 128;
  q.full = q.tiles_r * q.tiles_c;
  q.split = 1;
  return q;
}

constexpr size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Both products.  If all their tiles fit one round of the chip they may run side by side, each cut along its depth so
// that together they fill the round: the slower is cut further (by more than eight in eights) while there is room and
// a part has eight steps or more.  Against each filling the chip by itself, one behind the other, that halves the
// parts to be added (8192 x 1024 x 512 108 -> 74 us, 8192 x 2048 x 1024 195 -> 171) but may leave the longer one alone in
// the end (6614 x 2816 x 640 190 -> 198), so the two are compared: a step of the weights' gradients is 0.6 us, one of dx
// 0.9, a part written and read 0.1.  The plan is that of both gradients whatever is asked for, so that the bits do not
// depend on it.
// Otherwise, from many tokens on, dx reads the weights turned to f16 beforehand (14336 x 4096, the whole call: 1024 tokens
// 458 us without, 535 with; 2048 842 and 888; 4096 1614 and 1543).
struct BackwardPlan {
  ProductPlan dx, dw;
  bool turned, side;   // side: one launch for both
};
constexpr int64_t kTurned = 2816;
BackwardPlan plan_backward(int64_t m, int64_t n, int64_t k) {
  BackwardPlan b;
  b.dx = plan_dx(m, n, k);
  b.dw = plan_dw(m, n, k);
  const int64_t tiles[2] = {b.dx.tiles_r * b.dx.tiles_c, b.dw.tiles_r * b.dw.tiles_c};
  bool round = tiles[0] + tiles[1] <= kBCUs;
  if (round) {
    const int64_t steps[2] = {2 * n / kBStep, (m + kBStep - 1) / kBStep};
    int64_t sp[2] = {1, 1};
    auto time = [&](int i, int64_t split) { return (steps[i] + split - 1) / split * (i == 0 ? 9 : 6); };   // tenths of a us
    auto parts = [&](int i, int64_t split) { return split > 1 ? tiles[i] * split : 0; };
    for (;;) {
      const int i = time(0, sp[0]) >= time(1, sp[1]) ? 0 : 1;
      const int64_t next = sp[i] < 8 ? sp[i] + 1 : sp[i] + 8;
      if (next > 32 || next > steps[i] / 8 || tiles[i] * next + tiles[1 - i] * sp[1 - i] > kBCUs) break;
      sp[i] = next;
    }
    const int64_t t0 = time(0, sp[0]), t1 = time(1, sp[1]);
    const int64_t together = (t0 > t1 ? t0 : t1) + parts(0, sp[0]) + parts(1, sp[1]);
    const int64_t apart = time(0, b.dx.split) + time(1, b.dw.split) + parts(0, b.dx.split) + parts(1, b.dw.split);
    round = together < apart;
    ProductPlan* p[2] = {&b.dx, &b.dw};
    for (int i = 0; round && i < 2; ++i) {
      p[i]->split = (int32_t)sp[i];
      p[i]->full = sp[i] > 1 ? 0 : tiles[i];
    }
  }
  b.turned = m >= kTurned && !round;
  b.side = !b.turned && b.dw.tile_rows == 256;
  return b;
}

int grad_threads(int64_t n) { return n <= 4096 ? 256 : n <= 8192 ? 512 : 1024; }   // a row of D
int64_t pad_tokens(int64_t m) { return (m + kBStep - 1) / kBStep * kBStep; }
constexpr int64_t kGridThreads = int64_t(1) << 32;   // a launch's threads stay below

// last rows of x | cols | scale table | row factors | D16 | Db | turned weights | parts of dx | of the weights' gradients
struct BwdWs {
  uint16_t* xt;
  int32_t* cols;
  uint32_t* tab;
  int32_t* rs;
  uint16_t* d16;
  uint16_t* db;
  uint16_t* w16;
  float* part[2];
  size_t bytes;
};
BwdWs bwd_ws(void* ws, int64_t m, int64_t n, int64_t k) {
  BwdWs w;
  char* p = (char*)ws;
  size_t at = 0;
  auto take = [&](size_t b) {
    char* q = p + at;
    at += up256(b);
    return q;
  };
  w.xt = (uint16_t*)take((size_t)kBStep * (size_t)k * 2);
  w.cols = (int32_t*)take((size_t)(k / 128) * 4);
  w.tab = (uint32_t*)take((size_t)(2 * n / 128) * (size_t)(k / 128) * 4);
  w.rs = (int32_t*)take((size_t)m * 4);
  w.d16 = (uint16_t*)take((size_t)m * 2 * n * 2);
  w.db = (uint16_t*)take((size_t)pad_tokens(m) * 2 * n * 2);
  const BackwardPlan plan = plan_backward(m, n, k);
  w.w16 = (uint16_t*)take(plan.turned ? (size_t)k * 2 * n * 2 : 0);
  w.part[0] = (float*)take(plan.dx.part_bytes());
  w.part[1] = (float*)take(plan.dw.part_bytes());
  w.bytes = at;
  return w;
}

}  // namespace

// 32-bit offsets of a tile's rows, and grids
bool gated_backward_launchable(int64_t m, int64_t n, int64_t k) {
  if (m <= 0 || n <= 0 || k <= 0 || n % 128 || k % 128 || n >= (int64_t(1) << 22) || k >= (int64_t(1) << 22)) return false;
  const int64_t rt = (m + 255) / 256, jt = 2 * n / 128, ct = (k + 255) / 256;
  return rt * ct < kGridThreads / kBThreads && jt * ct < kGridThreads / kBThreads &&
         pad_tokens(m) + k / 128 < kGridThreads / grad_threads(n);
}

size_t gated_backward_bytes(int64_t m, int64_t n, int64_t k) { return bwd_ws(nullptr, m, n, k).bytes; }

hipError_t launch_gated_backward(const GatedBackward& a, hipStream_t s) {
  if (!gated_backward_launchable(a.m, a.n, a.k)) return hipErrorInvalidValue;
  const BwdWs w = bwd_ws(a.scratch, a.m, a.n, a.k);
  GateGrad d;
  d.dh = a.dh;
  d.gu = a.gu;
  d.m = a.m;
  d.n = a.n;
  d.m_pad = pad_tokens(a.m);
  d.d16 = a.dx ? w.d16 : nullptr;
  d.rs = w.rs;
  d.db = a.dgate ? w.db : nullptr;
  d.x = a.x;
  d.xt = w.xt;
  d.k = a.k;
  d.ws.sg = a.sg;
  d.ws.su = a.su;
  d.ws.pow2 = a.pow2;
  d.ws.nb = a.n / 128;
  d.ws.kb = a.k / 128;
  d.ws.tab = w.tab;
  d.ws.cols = w.cols;
  const unsigned grid = (unsigned)((a.dgate ? d.m_pad : a.m) + (a.dx ? d.ws.kb : 0));
  if (a.n <= 2048) gate_grad_kernel<256, 1><<<grid, 256, 0, s>>>(d);
  else if (a.n <= 4096) gate_grad_kernel<256, 2><<<grid, 256, 0, s>>>(d);
  else if (a.n <= 8192) gate_grad_kernel<512, 2><<<grid, 512, 0, s>>>(d);
  else if (a.n <= 16384) gate_grad_kernel<1024, 2><<<grid, 1024, 0, s>>>(d);
  else gate_grad_kernel<1024, 0><<<grid, 1024, 0, s>>>(d);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;

  GatedProduct dx = {}, dw = {};
  const BackwardPlan plan = plan_backward(a.m, a.n, a.k);
  ProductPlan px = {}, pw = {};
  auto planned = [&](GatedProduct& p, const ProductPlan& plan, float* part) {
    p.n = a.n;
    p.k = a.k;
    p.tiles_r = plan.tiles_r;
    p.tiles_c = plan.tiles_c;
    p.full = plan.full;
    p.split = plan.split;
    p.tile_rows = plan.tile_rows;
    p.part = part;
  };
  if (a.dx) {
    px = plan.dx;
    planned(dx, px, w.part[0]);
    dx.codes[0] = a.wg;
    dx.codes[1] = a.wu;
    dx.tab = w.tab;
    dx.p = w.w16;
    dx.q = w.d16;
    dx.rs = w.rs;
    dx.cols = w.cols;
    dx.rows = a.m;
    dx.z = 2 * a.n;
    dx.out[0] = dx.out[1] = a.dx;
  }
  if (a.dgate) {
    pw = plan.dw;
    planned(dw, pw, w.part[1]);
    dw.p = a.x;
    dw.xt = w.xt;
    dw.q = w.db;
    dw.rows = 2 * a.n;
    dw.z = a.m;
    dw.out[0] = a.dgate;
    dw.out[1] = a.dup;
  }
  auto go = [&](auto kernel, int lds, unsigned grid, auto... args) {
    e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return false;
    kernel<<<grid, kBThreads, lds, s>>>(args...);
    return true;
  };
  constexpr auto most = [](int x, int y) { return x > y ? x : y; };
  const bool small_dx = px.tile_rows == 128;
  bool ok = true;
  if (plan.side && a.dx && a.dgate) {
    constexpr int dw8 = Lds<kDw, 8>::kBytes;
    if (small_dx)
      ok = go(gated_both_kernel<4>, most(Lds<kDx, 4>::kBytes, dw8), px.grid() + pw.grid(), dx, dw, px.grid());
    else
      ok = go(gated_both_kernel<8>, most(Lds<kDx, 8>::kBytes, dw8), px.grid() + pw.grid(), dx, dw, px.grid());
  } else {
    if (a.dx && plan.turned) {
      gated_weights_kernel<<<dim3((unsigned)(a.k / 128), (unsigned)(2 * a.n / 128)), 256, 0, s>>>(a.wg, a.wu, w.tab, a.n, a.k, w.w16);
      ok = go(gated_product_kernel<kDxT, 8>, Lds<kDxT, 8>::kBytes, px.grid(), dx);
    } else if (a.dx && small_dx) {
      ok = go(gated_product_kernel<kDx, 4>, Lds<kDx, 4>::kBytes, px.grid(), dx);
    } else if (a.dx) {
      ok = go(gated_product_kernel<kDx, 8>, Lds<kDx, 8>::kBytes, px.grid(), dx);
    }
    if (ok && a.dgate)
      ok = pw.tile_rows == 128 ? go(gated_product_kernel<kDw, 4>, Lds<kDw, 4>::kBytes, pw.grid(), dw)
                               : go(gated_product_kernel<kDw, 8>, Lds<kDw, 8>::kBytes, pw.grid(), dw);
  }
  if (!ok) return e;
  const unsigned join = px.joins() + pw.joins();
  if (join) gated_join_kernel<<<join, 256, 0, s>>>(dx, dw, px.joins());
  return hipGetLastError();
}

}  // namespace ql
