// Attention over the NVFP4 KV cache for gfx950 (layout: kv4_common.hpp).
//
//   o = sum_t softmax_t(scale q . k_t) v_t,   k_t = khat_t 2^ek_t,  v_t = vhat_t 2^ev_t
//
// with khat, vhat = E2M1 * E4M3, which are exact in f16 (at most 6 significant bits, between
// 2^-10 and 2688).  q is brought to f16 by one power of two a row (exact but for magnitudes
// below 2^-29 of the row's largest), so q . khat is a product of exact f16 operands summed in
// float32.  The value row's exponent joins the logit:
//
//   w_t = scale log2(e) q.k_t + ev_t,  p_t = 2^(w_t - m + 9),  l = sum p_t 2^(-9 - ev_t),
//   o = 2^-9 (sum p_t vhat_t) / l
//
// with m near the largest w so far, so that p (rounded to f16 for the second product, 2^-11
// relative) and the sum of p vhat need no second scale.  m is only moved when some w passes
// it by 6, i.e. when p would pass 2^15; below, f16 holds p down to 2^-34 of the largest.
//
// l is rebuilt from p, and p is 0 below 2^-126: with ev far below the ev that set m, a token's whole
// weight would be lost.  What is lost is at most 2^(spread of ev - 135) of l a token.  So this
// holds while every ev lies in a window of 64 (values whose rows' largest are between 2^-35 and 2^28); from the
// first step that has another one (a zero row is one), l is summed by itself, relative to the
// largest logit (`apart`).
//
// The products are taken transposed: S^T = K Q^T and O^T = V^T P^T with the 16x16x32 MFMA, so
// that a lane holds one query row's logits for four consecutive tokens -- the four a lane
// takes of V^T -- and P goes from one product to the next in registers.
#include "../../include/qlinear.h"
#include "gemv_common.hpp"
#include "kv4_common.hpp"
#include "launch.hpp"

namespace ql {

constexpr int kAttnWaves = 4;
constexpr float kNoMax = -3.0e38f;  // m before any token was seen; exp2(-inf - kNoMax) = 0

// The window of ev that l and the sums of values share one maximum in (exponent bytes).
constexpr uint32_t kEvLow = 81, kEvSpan = 64;

// A logit is acc * (scale 2^e) * 2^ek, e the query row's exponent.  The factors meet in float32 where
// |scale 2^e| is in [kRowLow, kRowHigh]; the waves with a row outside of it form scale 2^(e + ek) in
// one step, no larger than float32 holds: acc is 0 for a key at right angles to the row, whatever their sizes.
constexpr float kRowLow = 0x1p-110f, kRowHigh = 0x1p9f;
__device__ __forceinline__ bool row_at_ends(float factor) {
  const float f = __builtin_fabsf(factor);
  return f < kRowLow || f > kRowHigh;
}
__device__ __forceinline__ float far_factor(float scale, int e, float key_power) {
  const int ek = (int)(__float_as_uint(key_power) >> 23) - 127;
  return __builtin_amdgcn_fmed3f(__builtin_ldexpf(scale, e + ek), -3.4e38f, 3.4e38f);
}

// 2^(d / 2) for d <= 0: l is multiplied by it twice, since 2^d alone may be 0 where l 2^d counts.
__device__ __forceinline__ float half_power(float d) { return __builtin_amdgcn_exp2f(0.5f * d); }

// Brings a row's maxima m (of logits with ev) and ml (of logits, which l is relative to) to one, so that l is
// between 2^-80 and 2^110 (2^30 tokens); the factor for the sums of values.
__device__ __forceinline__ float one_maximum(float& m, float ml, float& l) {
  const float to = __builtin_fminf(__builtin_fmaxf(m, ml - 80.0f), ml + 80.0f);
  const float by = __builtin_amdgcn_exp2f(m - to);
  l *= __builtin_amdgcn_exp2f(ml - to);
  m = to;
  return by;
}

struct AttnRange {
  int nq, n;        // query rows (tokens) and cached tokens of the sequence
  int64_t q0;       // first query token
  bool bad;
};

// The sequence's extents, cut to what the tables and tensors hold.
__device__ __forceinline__ AttnRange attn_range(const Attn4& a, int b) {
  AttnRange r;
  r.bad = false;
  int64_t n = a.kv_lens[b];
  const int64_t room = a.table_pages << a.page_shift;
  if (n < 0 || n > room) {
    r.bad = true;
    n = n < 0 ? 0 : room;
  }
  r.n = (int)n;
  if (a.q_starts) {
    const int64_t s = a.q_starts[b], e = a.q_starts[b + 1];
    r.q0 = s;
    r.nq = (int)(e - s);
    if (s < 0 || e < s || e > a.total_q || e - s > a.max_q) {
      r.bad = true;
      r.q0 = 0;
      r.nq = 0;
    }
  } else {
    r.q0 = (int64_t)b * a.max_q;
    r.nq = a.max_q;
  }
  return r;
}

__device__ __forceinline__ uint64_t uniform(uint64_t v) {
  return ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
         (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
}
// The same for a sequence that the whole wave asks for, in scalar registers.
__device__ __forceinline__ AttnRange attn_range_uniform(const Attn4& a, int b) {
  AttnRange r = attn_range(a, b);
  r.nq = __builtin_amdgcn_readfirstlane(r.nq);
  r.n = __builtin_amdgcn_readfirstlane(r.n);
  r.q0 = (int64_t)uniform((uint64_t)r.q0);
  return r;
}

// Registers of 16 tokens of one head as one lane takes them.
template <int D>
struct Keys4 {
  uint32_t k[D / 32];   // token lane % 16, elements (lane / 16) D / 4 on
  uint32_t ks;          // their D / 64 scales, at bit 8 (lane / 16) D / 64 % 32
  uint32_t e;           // at byte lane % 4 the exponent byte of token lane % 16: the key row's, or (few-row
                        // kernel) in lanes past 15 the value row's
};
template <int D>
struct Values4 {
  uint32_t v[D / 32];   // pair 16 j + lane % 16 of tokens 4 (lane / 16) + 0..3
  uint32_t vs[D / 32];  // their scales in block 2 j + (lane % 16) / 8
};

// N dwords of a group at a lane's offset.  The group is a buffer of its own (its address in
// scalar registers, its size the bound), so that a load takes one vector register of address.
template <int D>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t group_rsrc(const uint8_t* grp) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(grp), (short)0, kv4_group_bytes(D), 0x00020000);
}
template <int N>
__device__ __forceinline__ void load_words(uint32_t* dst, __amdgpu_buffer_rsrc_t grp, uint32_t off) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const i32x4 x = __builtin_amdgcn_raw_buffer_load_b128(grp, (int)(off + 16 * i), 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[4 * i + j] = (uint32_t)x[j];
    }
  } else if constexpr (N == 2) {
    const auto x = __builtin_amdgcn_raw_buffer_load_b64(grp, (int)off, 0, 0);
    dst[0] = (uint32_t)x[0];
    dst[1] = (uint32_t)x[1];
  } else {
    dst[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(grp, (int)off, 0, 0);
  }
}

// Offsets of a lane's loads within a group (the group's own address is the wave's).
template <int D>
struct Lane4 {
  uint32_t k, ks, e, v, vs;
  __device__ __forceinline__ explicit Lane4(int lane) {
    const uint32_t m = lane & 15, g = lane >> 4;
    k = m * (D / 2) + g * (D / 8);
    // whole dwords: the compiler's widening copies of shorter loads would wait for them at once
    ks = kv4_k_scales(D) + ((m * (D / 16) + g * (D / 64)) & ~3u);
    e = (g ? kv4_v_exps(D) : kv4_k_exps(D)) + (m & ~3u);
    v = kv4_v_codes(D) + lane * (D / 8);
    vs = kv4_v_scales(D) + g * (D / 4) + (m >> 3) * (D / 8);
  }
};
template <int D>
__device__ __forceinline__ void load_keys(Keys4<D>& f, const uint8_t* grp, const Lane4<D>& at) {
  const __amdgpu_buffer_rsrc_t rs = group_rsrc<D>(grp);
  load_words<D / 32>(f.k, rs, at.k);
  load_words<1>(&f.ks, rs, at.ks);
  load_words<1>(&f.e, rs, at.e);
}
template <int D>
__device__ __forceinline__ void load_values(Values4<D>& f, const uint8_t* grp, const Lane4<D>& at) {
  const __amdgpu_buffer_rsrc_t rs = group_rsrc<D>(grp);
  load_words<D / 32>(f.v, rs, at.v);
  load_words<D / 32>(f.vs, rs, at.vs);
}

// Two E4M3 scales (bytes 0 and 1 of w, or 2 and 3) as f16, exactly; 0x7F and 0xFF are NaN.
template <bool HI>
__device__ __forceinline__ f16x2 scales2(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, HI);
}

// Eight elements of one dword of codes times a scale; the products are exact.
__device__ __forceinline__ f16x8 scaled8(uint32_t codes, f16x2 s0, f16x2 s1, f16x2 s2, f16x2 s3) {
  const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0) * s0;
  const f16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1) * s1;
  const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2) * s2;
  const f16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3) * s3;
  return f16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}
__device__ __forceinline__ f16x2 both(_Float16 s) { return f16x2{s, s}; }

// The call's work is cut on the device from the lengths that are there when it runs (so that a
// captured call follows them).  A unit is R query rows of one sequence and KV head, as many
// chunks of 128 tokens long as the sequence needs (one at least); the units in the order
// (sequence, row tile, head) make one line of chunks, of which each workgroup takes the same
// length.  One round of workgroups fills the chip and all end together, whatever the lengths;
// a unit that lies in more than one workgroup's part is joined from partial results.
//
// Decoding is bound by the cache's bytes: 256 sequences of up to 4096 tokens, 64/8 heads of 128, take
// 132 us for 620 MB (4.7 TB/s; a large copy moves 5.2), where the same kernel with its loads alone
// takes 129; 64 of them 54 us, 53 with the loads alone.  Pages in the order of memory in place of
// scattered ones would give 116 and 45.  One sequence of 613 tokens, 8.9 us, is the latency of the
// chain: cut, page, codes, joins in the workgroup and between workgroups.
constexpr int kAttnStep = 32;                        // tokens of one wave's step
constexpr int kAttnChunk = kAttnWaves * kAttnStep;   // of the workgroup's
// Workgroups that fit the chip: 256 CUs and the waves a SIMD holds by the kernel's registers.
constexpr int attn_wgs_per_cu(int d) { return d == 256 ? 2 : d == 64 ? 4 : 3; }
constexpr int attn_wgs(int d) { return 256 * attn_wgs_per_cu(d); }

// Positions on the line fit 32 bits unless a call could be enormous (a.wide, set from its bounds on
// the host); the narrow form has the wave's scan in DPP steps and short divisions.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_add(uint32_t v) {
  return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {  // inclusive
  v = dpp_add<0x111, 0xF>(v);  // row_shr:1, 2, 4, 8
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);  // the last of rows 0 and 2 to rows 1 and 3
  return dpp_add<0x143, 0xC>(v);  // the last of row 1 to rows 2 and 3
}
__device__ __forceinline__ uint64_t wave_scan(uint64_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t lo = (uint32_t)__shfl_up((int)(uint32_t)v, o), hi = (uint32_t)__shfl_up((int)(v >> 32), o);
    if (lane >= o) v += ((uint64_t)hi << 32) | lo;
  }
  return v;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {  // of all in the last lane
  v = dpp_max<0x111, 0xF>(v);
  v = dpp_max<0x112, 0xF>(v);
  v = dpp_max<0x114, 0xF>(v);
  v = dpp_max<0x118, 0xF>(v);
  v = dpp_max<0x142, 0xA>(v);
  return dpp_max<0x143, 0xC>(v);
}
__device__ __forceinline__ uint32_t of_lane(uint32_t v, int j) { return (uint32_t)__builtin_amdgcn_readlane((int)v, j); }
__device__ __forceinline__ uint64_t of_lane(uint64_t v, int j) {
  return ((uint64_t)of_lane((uint32_t)(v >> 32), j) << 32) | of_lane((uint32_t)v, j);
}

// The first token that some row of the sequence sees, down to a step.
__device__ __forceinline__ int attn_lo(const Attn4& a, int nq, int n) {
  return a.window ? max(n - nq + 1 - a.window, 0) & ~(kAttnStep - 1) : 0;
}

// How the line is cut.  A unit's start in a workgroup (its query rows, the first loads, the joins at
// its end) takes as long as two or three chunks.  So, where that makes the shares hardly longer,
// each unit gets whole workgroups: its stretch is filled up to a multiple of the share (16 sequences of
// 4096 tokens, 28/4 heads: 18.6 us, 22.7 without).  Else, where the shares are long, a unit's stretch
// begins with `cost` places without a chunk (256 of up to 4096, 64/8 heads: 137 us, 148 without).
struct AttnCut {
  uint64_t each;   // chunks a workgroup
  uint64_t end;    // of the line
  uint32_t cost;
  bool whole;
  template <typename T>
  __device__ __forceinline__ T stretch(uint32_t chunks) const {
    if (!whole || each <= 1) return (T)chunks + cost;
    return (T)((chunks + (uint32_t)each - 1) / (uint32_t)each) * (T)each;
  }
};
// kWholeMore: chunks that a share may grow by for whole workgroups.  kUnitCost is taken in full from
// kUnitCost * kCostShare chunks a workgroup on; charged to shorter shares it costs more than it evens
// out (32 sequences of 2000 tokens at D = 64: 19.3 us, 16.6 without).
constexpr uint32_t kUnitCost = 2, kCostShare = 3, kWholeMore = 2;

// A workgroup's place on the line.
struct AttnPlace {
  uint64_t pos, stop;   // chunks of the line
  int b, tile, head, k; // unit and its first chunk here
  AttnCut cut;
  int done, turn;       // chunks behind it; when the waves' priority is lowered next
};

// Of the workgroups that share a CU the oldest is served first at every turn: equal shares ended
// after 90 to 146 us.  So a wave that is ahead gives way: its priority falls at a half, three
// quarters and seven eighths of its share (256 sequences of up to 4096 tokens: 149 us, 158 without).
__device__ __forceinline__ void attn_give_way(AttnPlace& pl, int each) {
  if (pl.turn < each / 2 + each / 4) {
    __builtin_amdgcn_s_setprio(2);
    pl.turn = each / 2 + each / 4;
  } else if (pl.turn < each - each / 8) {
    __builtin_amdgcn_s_setprio(1);
    pl.turn = each - each / 8;
  } else {
    __builtin_amdgcn_s_setprio(0);
    pl.turn = INT32_MAX;
  }
}

// A sequence's chunks, and its units (all tiles and heads).
__device__ __forceinline__ uint32_t attn_chunks(const Attn4& a, const AttnRange& r) {
  return max((max(r.n - attn_lo(a, r.nq, r.n), 0) + kAttnChunk - 1) / kAttnChunk, 1);
}
template <int R>
__device__ __forceinline__ uint32_t attn_units(const Attn4& a, const AttnRange& r) {
  return (r.nq * a.group > a.few ? 0u : (uint32_t)(r.nq * a.group + R - 1) / R) * (uint32_t)a.heads;
}

// units, chunks: a lane's sequence of the first 64; sum, sum_u: the chunks and units of all
template <int R, int WGS, typename T>
__device__ __forceinline__ AttnCut attn_cut(const Attn4& a, uint32_t units, uint32_t chunks, T sum, T sum_u) {
  AttnCut c{(uint64_t)((sum + WGS - 1) / WGS), (uint64_t)sum, 0, sum <= WGS};
  if (c.whole) return c;
  if (sum_u <= WGS) {
    const uint32_t each = (uint32_t)c.each;   // < 2^24: a unit's chunks are
    for (uint32_t e = each; e <= each + kWholeMore; ++e) {
      uint32_t n = units * ((chunks + e - 1) / e);
      for (int b = 64 + (threadIdx.x & 63); b < a.batch; b += 64) {
        const AttnRange r = attn_range(a, b);
        n += attn_units<R>(a, r) * ((attn_chunks(a, r) + e - 1) / e);
      }
      n = of_lane(wave_scan(n), 63);
      if (n <= WGS) return AttnCut{e, (uint64_t)n * e, 0, true};
    }
  }
  c.cost = (uint32_t)min((T)kUnitCost, sum / (WGS * kCostShare));
  c.end = (uint64_t)(sum + sum_u * c.cost);
  c.each = (c.end + WGS - 1) / WGS;
  return c;
}

// Every wave works this out for itself, 64 sequences at a time.
template <int R, int WGS, typename T>
__device__ __forceinline__ bool attn_place(const Attn4& a, AttnPlace& pl, AttnRange& rg) {
  const int lane = threadIdx.x & 63;
  const auto range = [&](int b) { return b < a.batch ? attn_range(a, b) : AttnRange{0, 0, 0, false}; };
  AttnRange r = range(lane);
  bool bad = r.bad;
  const uint32_t units = attn_units<R>(a, r), chunks = attn_chunks(a, r);
  T sum_u = units, sum = (T)units * chunks;
  for (int b0 = 64; b0 < a.batch; b0 += 64) {
    const AttnRange x = range(b0 + lane);
    bad |= x.bad;
    const uint32_t u = attn_units<R>(a, x);
    sum_u += u;
    sum += (T)u * attn_chunks(a, x);
  }
  if (blockIdx.x == 0 && threadIdx.x < 64 && __any(bad) && lane == 0) atomicOr(a.status, (int32_t)kStatusBadItem);
  sum_u = of_lane(wave_scan(sum_u), 63);
  sum = of_lane(wave_scan(sum), 63);
  const AttnCut cut = attn_cut<R, WGS, T>(a, units, chunks, sum, sum_u);
  T mine = (T)units * cut.stretch<T>(chunks), upto = wave_scan(mine);
  const T each = (T)cut.each, pos = (T)blockIdx.x * each, end = (T)cut.end;
  if (pos >= end) return false;
  pl.cut = cut;
  pl.stop = min(pos + each, end);
  T before = 0;
  for (int b0 = 0;;) {
    const uint64_t past = __ballot(before + upto > pos);
    if (past) {
      const int j = __builtin_ctzll(past);
      pl.b = b0 + j;
      rg.nq = __builtin_amdgcn_readlane(r.nq, j);
      rg.n = __builtin_amdgcn_readlane(r.n, j);
      rg.q0 = (int64_t)of_lane((uint64_t)r.q0, j);
      // place within the sequence: its units and their length
      const T at = pos - before - of_lane((T)(upto - mine), j);
      const T len = cut.stretch<T>(attn_chunks(a, rg));
      const uint32_t unit = (uint32_t)(at / len);
      const int k = __builtin_amdgcn_readfirstlane((int)(at - (T)unit * len)) - (int)cut.cost;
      pl.k = max(k, 0);
      pl.pos = pos + (uint32_t)(pl.k - k);
      pl.tile = __builtin_amdgcn_readfirstlane((int)(unit / (uint32_t)a.heads));
      pl.head = __builtin_amdgcn_readfirstlane((int)(unit - (uint32_t)pl.tile * (uint32_t)a.heads));
      return pl.pos < pl.stop;
    }
    before += of_lane(upto, 63);
    b0 += 64;
    if (b0 >= a.batch) return false;
    r = range(b0 + lane);
    mine = (T)attn_units<R>(a, r) * cut.stretch<T>(attn_chunks(a, r));
    upto = wave_scan(mine);
  }
}

// The workgroups that a unit of `chunks` from u0 on the line lies in: the first, and how many.
__device__ __forceinline__ int attn_parts(const Attn4& a, uint64_t u0, uint32_t chunks, uint64_t each, int& w0) {
  if (a.wide) {
    w0 = (int)(u0 / each);
    return (int)((u0 + chunks - 1) / each) - w0 + 1;
  }
  const uint32_t e = (uint32_t)each;
  w0 = (int)((uint32_t)u0 / e);
  return (int)(((uint32_t)u0 + chunks - 1) / e) - w0 + 1;
}

// Partial results of a split: R rows of D float32 sums, then m and l of the rows.
template <int D, int R>
__host__ __device__ constexpr uint32_t attn_part_bytes() {
  return R * (D + 2) * 4;
}

// x / d for 0 <= x < d + 16.
__device__ __forceinline__ int small_div(int x, int d) {
  return d >= 16 ? x >= d : (int)(((float)x + 0.5f) * __builtin_amdgcn_rcpf((float)d));
}

template <int D, int R>
struct AttnShared {
  float o[kAttnWaves][R][D + 4];
  float m[kAttnWaves][R], l[kAttnWaves][R];
  __attribute__((aligned(16))) float x[kAttnWaves][2][64];
  int last;
};

// The waves take alternate 32-token steps of a unit and their sums are joined through shared
// memory.  Of a unit in several workgroups' parts, the one that arrives last joins the results,
// in their order.
//
// A lane's dword of V holds an even and an odd element of four tokens, and the conversion
// gives them as pairs.  The pairs stay together as neighbours along the product's depth,
// with P beside zeros: [p 0] takes the even elements and [0 p] the odd ones.  That doubles the
// matrix instructions of the second product, which have room, and saves the vector
// instructions that would part the pairs, which have none.  With R = 8 rows the two are the
// two halves of the 16 columns of one product, with R = 16 two products.
template <int D, int R>
__device__ __forceinline__ void attn4_unit(const Attn4& a, AttnPlace& pl, const AttnRange& rg, int lo, int stop,
                                           int chunks, AttnShared<D, R>& sh) {
  constexpr int KW = D / 32, P = R / 8;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  const int rn = R == 16 ? n16 : n16 & 7;                 // this lane's query row of the tile
  const int odd_shift = R == 16 ? 16 : (n16 >> 3) << 4;   // where p goes beside its zero
  const int h = pl.head;
  const int rows = rg.nq * a.group;
  const int r0 = pl.tile * R;
  const int live = min(rows - r0, R);   // rows of the tile; lanes past them repeat the last

  // the query tokens of the tile, this lane's, and the tokens [from, to) that it sees
  const int qa = r0 / a.group, ra = r0 - qa * a.group;
  const int qb = qa + small_div(ra + live - 1, a.group);
  const int mine_r = min(rn, live - 1);
  const int dq = small_div(ra + mine_r, a.group);
  const int head = h * a.group + ra + mine_r - dq * a.group;
  const int to = a.causal ? rg.n - rg.nq + qa + dq + 1 : rg.n;
  const int from = a.window ? to - a.window : 0;
  const int end = a.causal ? rg.n - rg.nq + qb + 1 : rg.n;         // some row sees [begin, end)
  const int all_to = a.causal ? rg.n - rg.nq + qa + 1 : rg.n;      // every row sees [all_from, all_to)
  const int begin = a.window ? max(all_to - a.window, 0) : 0;
  const int all_from = a.window ? end - a.window : 0;
  const int hi = min(end, stop);

  f32x4 o[P][KW];
#pragma unroll
  for (int y = 0; y < P; ++y)
#pragma unroll
    for (int j = 0; j < KW; ++j) o[y][j] = f32x4{0, 0, 0, 0};
  float m = kNoMax, l = 0.0f;
  uint32_t apart = 0;   // 1: l is relative to ml, the largest logit
  float ml = kNoMax;
  const int32_t* table = a.table + (int64_t)pl.b * a.table_stride;
  const int per = 1 << (a.page_shift - 4);
  bool bad_page = false;

  // The wave's groups of 16 tokens are numbered x = 0, 1, ..: group x is at lo + 32 wave +
  // 128 (x / 2) + 16 (x % 2).  Lane x % 64 looks up the page of group x for all: -1 where it is
  // outside the cache, and where no row of the tile sees the group.
  int pages = 0;
  const auto look_up = [&](int x0) {
    const int x = x0 + lane;
    const int t = lo + wave * 32 + (x >> 1) * (kAttnWaves * 32) + (x & 1) * 16;
    pages = -1;
    if (t < hi && t + 16 > begin) {
      pages = table[t >> a.page_shift];
      if (pages < 0 || pages >= a.pages) {
        pages = -1;
        bad_page = true;
      }
    }
  };
  const auto group_at = [&](int x, int t) {
    const int pg = max(__builtin_amdgcn_readlane(pages, x & 63), 0);
    const int64_t gi = (((int64_t)pg * a.heads + h) << (a.page_shift - 4)) + ((t >> 4) & (per - 1));
    return a.data + uniform((uint64_t)gi * kv4_group_bytes(D));
  };

  const Lane4<D> lane_at(lane);
  const uint32_t sel_k = g == 0 ? ~0u : 0u, sel_v = g == 1 ? ~0u : 0u;
  Keys4<D> f[2];
  Values4<D> fv[2];
  const uint8_t* grp[2];
  bool ok[2] = {false, false};
  int x = 0;
  const bool any = lo + wave * 32 < hi;
  // the first loads in the order in which they are waited for: pages, the query row, codes
  look_up(0);
  uint4 qx[KW];
  {
    const uint16_t* qp = a.q + (rg.q0 + qa + dq) * a.q_stride + (int64_t)head * D + g * (D / 4);
#pragma unroll
    for (int s = 0; s < KW; ++s) qx[s] = *(const uint4*)(qp + 8 * s);
  }
  if (any) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      ok[u] = __builtin_amdgcn_readlane(pages, u) >= 0;
      grp[u] = group_at(u, lo + wave * 32 + 16 * u);
      load_keys<D>(f[u], grp[u], lane_at);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) load_values<D>(fv[u], grp[u], lane_at);
  }

  // the query row as f16 with its largest magnitude in [2^14, 2^15)
  f16x8 q[KW];
  float kc;
  uint32_t at_ends;
  {
    uint32_t amax = 0;
#pragma unroll
    for (int s = 0; s < KW; ++s) {
      u16x2 t = max_u16x2(max_u16x2(abs_bits2(qx[s].x), abs_bits2(qx[s].y)),
                          max_u16x2(abs_bits2(qx[s].z), abs_bits2(qx[s].w)));
      amax = umax(amax, hmax_u16x2(t));
    }
    amax = umax(amax, (uint32_t)__shfl_xor((int)amax, 16));
    amax = umax(amax, (uint32_t)__shfl_xor((int)amax, 32));
    const int e = amax ? (int)(amax >> 7) - 127 - 14 : 0;   // subnormal rows: -141, still exact
    kc = __builtin_ldexpf(a.scale_log2e, e);
    at_ends = __any(row_at_ends(kc) && a.scale_log2e != 0.0f && amax < kBf16InfBits);
    if (__builtin_expect(at_ends, 0)) {
      sh.l[wave][rn] = __int_as_float(e);   // (not in use before the waves' sums are joined)
      kc = 1.0f;
    }
    if (amax >= kBf16InfBits) kc = __builtin_nanf("");
#pragma unroll
    for (int s = 0; s < KW; ++s) {
      const uint32_t w[4] = {qx[s].x, qx[s].y, qx[s].z, qx[s].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[s][2 * i] = (_Float16)__builtin_ldexpf(bf16_lo(w[i]), -e);
        q[s][2 * i + 1] = (_Float16)__builtin_ldexpf(bf16_hi(w[i]), -e);
      }
    }
  }

  const int each = (int)min(pl.cut.each, (uint64_t)(1 << 30));
  int done = pl.done;
  for (int t0 = lo + wave * 32; t0 < hi; t0 += kAttnWaves * 32) {
    if (++done > pl.turn) attn_give_way(pl, each);
    // what depends on the token alone is worked out by one lane a token and shared: 2^ek, ev + 127
    // and 2^(-9 - ev) at 0, 16 and 32 of x
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t eb = (f[u].e >> (8 * (lane & 3))) & 0xFFu, b23 = eb << 23;
      // (selected by masks: written as a choice, the compiler branches)
      const uint32_t ve = __float_as_uint((float)eb), lf = (245u - min(eb, 244u)) << 23;
      sh.x[wave][u][lane] = __uint_as_float((b23 & sel_k) | (ve & sel_v) | (lf & ~(sel_k | sel_v)));
    }
    __builtin_amdgcn_wave_barrier();
    f32x4 c[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t ks = f[u].ks >> ((8 * (D / 64) * g) & 31);
      const f16x2 s01 = scales2<false>(ks), s23 = scales2<true>(ks);
      c[u] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KW; ++s) {
        const f16x2 sp = both((s >> 1) < 2 ? s01[(s >> 1) & 1] : s23[(s >> 1) & 1]);
        c[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(scaled8(f[u].k[s], sp, sp, sp, sp), q[s], c[u], 0, 0, 0);
      }
    }
    if (__builtin_expect(at_ends, 0)) {   // the sums become logits here
      const int e = __float_as_int(sh.l[wave][rn]);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[u][i] *= far_factor(a.scale_log2e, e, sh.x[wave][u][4 * g + i]);
      __builtin_amdgcn_wave_barrier();
      if (g == 0) sh.x[wave][0][n16] = sh.x[wave][1][n16] = 1.0f;
      __builtin_amdgcn_wave_barrier();
    }
    // which of its 8 tokens this lane's row sees
    uint32_t seen = 0xFFu, off[2];   // off: of ev from the window, in the lanes past 15, which hold value rows' exponents
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = t0 + 16 * u;
      off[u] = ((f[u].e >> (8 * (lane & 3))) & 0xFFu) - kEvLow;
      if (!ok[u] || t < all_from || t + 16 > all_to) {
        const int t4 = t + 4 * g;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(ok[u] && t4 + i >= from && t4 + i < to)) seen &= ~(1u << (4 * u + i));
        // tokens that no row sees may be memory that was never written: no NaN from their scales
        const int skip = min(max(begin - t4, 0), 4), keep = ok[u] ? min(max(rg.n - t4, 0), 4) : 0;
        const uint32_t mask = (uint32_t)(((uint64_t)1 << (8 * keep)) - 1) & ~(uint32_t)(((uint64_t)1 << (8 * skip)) - 1);
#pragma unroll
        for (int j = 0; j < KW; ++j) fv[u].vs[j] &= mask;
        if (!(ok[u] && t + n16 >= begin && t + n16 < end)) off[u] = 0;   // a token that no row sees
      }
    }
    if ((__ballot(umax(off[0], off[1]) >= kEvSpan) >> 16) != 0 && !apart) {
      apart = 1;
      ml = m;
    }
    const bool edge = !ok[0] || !ok[1] || t0 < all_from || t0 + 32 > all_to;
    // The next step's keys are on their way from here, its values from when this step's are
    // used.  After the last step the same groups are fetched again: with a branch around the
    // loads the compiler would wait for all that are in flight.
    {
      const bool more = t0 + kAttnWaves * 32 < hi;
      x += more ? 2 : 0;
      const int tn = t0 + (more ? kAttnWaves * 32 : 0);
      if (more && (x & 63) == 0) look_up(x);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        ok[u] = __builtin_amdgcn_readlane(pages, (x + u) & 63) >= 0;
        grp[u] = group_at(x + u, tn + 16 * u);
        load_keys<D>(f[u], grp[u], lane_at);
      }
    }
    // w - add of the step's tokens, -inf where the row does not see them
    float p[2][4];
    const auto weigh = [&](float add) {
      float top = -__builtin_inff();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f32x4 kf = *(const f32x4*)&sh.x[wave][u][4 * g] * kc;
        const f32x4 ve = *(const f32x4*)&sh.x[wave][u][16 + 4 * g];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[u][i] = __builtin_fmaf(c[u][i], kf[i], ve[i] + add);
      }
      if (edge) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!(seen >> (4 * u + i) & 1)) p[u][i] = -__builtin_inff();
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = __builtin_fmaxf(top, p[u][i]);
      return top;
    };
    if (__builtin_expect(apart, 0)) {
      float w[2][4], top = -__builtin_inff();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f32x4 kf = *(const f32x4*)&sh.x[wave][u][4 * g] * kc;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[u][i] = seen >> (4 * u + i) & 1 ? c[u][i] * kf[i] : -__builtin_inff();
          top = __builtin_fmaxf(top, w[u][i]);
        }
      }
      top = __builtin_fmaxf(top, __shfl_xor(top, 16));
      top = __builtin_fmaxf(top, __shfl_xor(top, 32));
      top = __builtin_fmaxf(top, ml);
      l *= __builtin_amdgcn_exp2f(ml - top);
      ml = top;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) l += __builtin_amdgcn_exp2f(w[u][i] - top);
    }
    if (__any(weigh(9.0f - 127.0f - m) > 15.0f)) {   // x holds ev + 127
      // the maximum moves: w again in full, the sums to the new one
      float w = weigh(-127.0f);
      w = __builtin_fmaxf(w, __shfl_xor(w, 16));
      w = __builtin_fmaxf(w, __shfl_xor(w, 32));
      const float mn = __builtin_fmaxf(m, w), shrink = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= apart ? 1.0f : shrink;
#pragma unroll
      for (int y = 0; y < P; ++y)
#pragma unroll
        for (int j = 0; j < KW; ++j) o[y][j] *= shrink;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[u][i] = p[u][i] - m + 9.0f;
    }
    const float l_apart = l;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
      u32x4 pe, po;
      const f32x4 lf = *(const f32x4*)&sh.x[wave][u][32 + 4 * g];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = __builtin_amdgcn_exp2f(p[u][i]);
        l = __builtin_fmaf(e, lf[i], l);
        const uint32_t hbits = __builtin_bit_cast(uint16_t, (_Float16)e);
        pe[i] = hbits;
        po[i] = hbits << odd_shift;
      }
#pragma unroll
      for (int j = 0; j < KW; ++j) {
        const f16x2 s01 = scales2<false>(fv[u].vs[j]), s23 = scales2<true>(fv[u].vs[j]);
        const f16x8 v = scaled8(fv[u].v[j], both(s01[0]), both(s01[1]), both(s23[0]), both(s23[1]));
        o[0][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, __builtin_bit_cast(f16x8, R == 16 ? pe : po), o[0][j], 0, 0, 0);
        if constexpr (R == 16)
          o[P - 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, __builtin_bit_cast(f16x8, po), o[P - 1][j], 0, 0, 0);
      }
    }
    if (apart) l = l_apart;
#pragma unroll
    for (int u = 0; u < 2; ++u) load_values<D>(fv[u], grp[u], lane_at);
  }
  if (__any(bad_page) && lane == 0) atomicOr(a.status, (int32_t)kStatusBadItem);

  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (apart) {
    const float by = one_maximum(m, ml, l);
#pragma unroll
    for (int y = 0; y < P; ++y)
#pragma unroll
      for (int j = 0; j < KW; ++j) o[y][j] *= by;
  }
#pragma unroll
  for (int y = 0; y < P; ++y)
#pragma unroll
    for (int j = 0; j < KW; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sh.o[wave][rn][32 * j + 8 * g + 2 * i + (R == 16 ? y : n16 >> 3)] = o[y][j][i];
  if (g == 0 && n16 < R) {
    sh.m[wave][rn] = m;
    sh.l[wave][rn] = l;
  }
  __syncthreads();
  // E elements of a row a thread
  constexpr int E = R * D / (kAttnWaves * 64) < 4 ? 4 : R * D / (kAttnWaves * 64), kPer = D / E;
  constexpr int kJoin = 32 / E < 4 ? 4 : 32 / E;  // splits joined at a time
  const int orow = threadIdx.x / kPer, part = threadIdx.x % kPer;
  const bool mine = orow < live;
  const int src = mine ? orow : 0;
  float top = sh.m[0][src];
#pragma unroll
  for (int w = 1; w < kAttnWaves; ++w) top = __builtin_fmaxf(top, sh.m[w][src]);
  float acc[E], lsum = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll
  for (int w = 0; w < kAttnWaves; ++w) {
    const float r = half_power(sh.m[w][src] - top), s = r * r;
    lsum += sh.l[w][src] * r * r;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += s * sh.o[w][src][part * E + e];
  }
  const uint64_t u0 = pl.pos - (uint64_t)pl.k;   // the unit on the line, and the workgroups it lies in
  int w0;
  const int splits = attn_parts(a, u0, (uint32_t)chunks, pl.cut.each, w0);
  if (splits > 1) {
    // a workgroup has two places for partial results: for the unit that goes on in the next
    // workgroup (1) and for the one that came from the one before (0)
    constexpr uint32_t kBytes = attn_part_bytes<D, R>();
    const __amdgpu_buffer_rsrc_t rs = dev_rsrc(a.parts);
    const int split = (int)blockIdx.x - w0;
    const uint32_t at = (uint32_t)(2 * blockIdx.x + (split == 0)) * kBytes;
    const uint32_t mine_at = (uint32_t)(src * D + part * E) * 4;
    if (mine) {
#pragma unroll
      for (int e = 0; e < E; e += 4)
        st_dev4v(rs, at + mine_at + 4 * e, f32x4{acc[e], acc[e + 1], acc[e + 2], acc[e + 3]});
      if (part == 0) {
        st_dev_u32((uint32_t*)(a.parts + at + R * D * 4) + src, __float_as_uint(top));
        st_dev_u32((uint32_t*)(a.parts + at + R * D * 4) + R + src, __float_as_uint(lsum));
      }
    }
    if (a.join) return;   // by the kernel that follows
    wait_stores();
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t* c = a.counters + w0;   // no two units go on from the same workgroup
      const uint32_t old = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      sh.last = old == (uint32_t)splits - 1;
      if (sh.last) st_dev_u32(c, 0u);
    }
    __syncthreads();
    if (!sh.last || !mine) return;
    const uint32_t first = (uint32_t)(2 * w0 + 1) * kBytes;   // split s at w0 + s: (2 w0 + 1) or 2 (w0 + s)
    const auto place = [&](int s) { return s == 0 ? first : first + (uint32_t)(2 * s - 1) * kBytes; };
    const uint32_t ml = R * D * 4 + (uint32_t)src * 4;
    const auto ld = [&](uint32_t off) { return __uint_as_float(ld_dev_u32((const uint32_t*)(a.parts + off))); };
    // the running maximum is moved once for kJoin splits, so that their loads
    // are in flight together (a load from another XCD takes over a microsecond)
    top = kNoMax;
    lsum = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll 1
    for (int s0 = 0; s0 < splits; s0 += kJoin) {
      float mx[kJoin], lx[kJoin];
      f32x4 v[kJoin][E / 4];
#pragma unroll
      for (int i = 0; i < kJoin; ++i) {
        const uint32_t from_s = place(min(s0 + i, splits - 1));
        mx[i] = ld(from_s + ml);
        lx[i] = ld(from_s + ml + R * 4);
#pragma unroll
        for (int e = 0; e < E / 4; ++e) v[i][e] = ld_dev4v(rs, from_s + mine_at + 16 * e);
      }
      float mn = top;
#pragma unroll
      for (int i = 0; i < kJoin; ++i) mn = __builtin_fmaxf(mn, mx[i]);
      const float back = half_power(top - mn), shrink = back * back;
      lsum = lsum * back * back;
      top = mn;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= shrink;
#pragma unroll
      for (int i = 0; i < kJoin; ++i) {
        const float r = s0 + i < splits ? half_power(mx[i] - top) : 0.0f, w = r * r;
        lsum = __builtin_fmaf(lx[i] * r, r, lsum);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = __builtin_fmaf(w, v[i][e / 4][e & 3], acc[e]);
      }
    }
  }
  if (!mine) return;
  const int oq = qa + small_div(ra + src, a.group), oh = h * a.group + (r0 + src) - oq * a.group;
  const float inv = lsum == 0.0f ? 0.0f : 0.001953125f / lsum;  // a row that sees nothing: zeros
  uint16_t* op = a.out + (rg.q0 + oq) * a.out_stride + (int64_t)oh * D + part * E;
#pragma unroll
  for (int e = 0; e < E; e += 4)
    *(uint2*)(op + e) = make_uint2(pack_bf16x2_rne(acc[e] * inv, acc[e + 1] * inv),
                                   pack_bf16x2_rne(acc[e + 2] * inv, acc[e + 3] * inv));
  if (a.lse && part == 0)
    a.lse[(rg.q0 + oq) * a.q_heads + oh] =
        lsum == 0.0f ? -__builtin_inff() : (__builtin_log2f(lsum) + top) * 0.6931471805599453f;
}

template <int D, int R>
__global__ __launch_bounds__(kAttnWaves * 64, attn_wgs_per_cu(D)) void attn4_kernel(Attn4 a) {
  __shared__ AttnShared<D, R> sh;
  AttnPlace pl;
  AttnRange rg;
  if (!(a.wide ? attn_place<R, attn_wgs(D), uint64_t>(a, pl, rg) : attn_place<R, attn_wgs(D), uint32_t>(a, pl, rg))) return;
  pl.done = 0;
  pl.turn = (int)min(pl.cut.each, (uint64_t)(1 << 30)) / 2;
  __builtin_amdgcn_s_setprio(3);
  for (;;) {
    const int lo_b = attn_lo(a, rg.nq, rg.n);
    const int chunks = (int)attn_chunks(a, rg);
    const int k1 = (int)min((uint64_t)chunks, pl.k + (pl.stop - pl.pos));
    attn4_unit<D, R>(a, pl, rg, lo_b + pl.k * kAttnChunk, k1 == chunks ? rg.n : lo_b + k1 * kAttnChunk, chunks, sh);
    pl.pos += k1 - pl.k;
    pl.done += k1 - pl.k;
    if (k1 == chunks) pl.pos += pl.cut.cost;
    if (pl.cut.whole || pl.pos >= pl.stop) break;
    pl.k = 0;
    if (++pl.head == a.heads) {
      pl.head = 0;
      if (++pl.tile * R >= rg.nq * a.group) {
        pl.tile = 0;
        do rg = attn_range_uniform(a, ++pl.b); while (rg.nq == 0 || rg.nq * a.group > a.few);   // pos < stop: another unit is there
      }
    }
    __syncthreads();   // the shared memory of the unit before is read
  }
}
// Where few units are cut into many parts, the one workgroup that joins a unit would take longer
// (230 KB for 64 parts of 7 rows at D = 128, 13 us) than a launch: this kernel joins each row of
// each unit by a workgroup.
template <int D, int R>
__global__ __launch_bounds__(256) void attn4_join_kernel(Attn4 a, int tiles) {
  constexpr int WGS = attn_wgs(D), kPer = D / 4, kSide = 256 / kPer;   // threads a part, parts side by side
  constexpr uint32_t kBytes = attn_part_bytes<D, R>();
  __shared__ float sm[WGS], sl[WGS], red[kSide][D], smax[4], ssum[kSide];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = blockIdx.x % R, unit = blockIdx.x / R;
  const int head = unit % a.heads, tile = unit / a.heads % tiles, b = unit / a.heads / tiles;
  const AttnRange rg = attn_range_uniform(a, b);
  if (tile * R + row >= rg.nq * a.group || rg.nq * a.group > a.few) return;
  // (of no more than 64 sequences: launch_r)
  const AttnRange at = lane < a.batch ? attn_range(a, lane) : AttnRange{0, 0, 0, false};
  const uint32_t chunks = attn_chunks(a, rg), units = attn_units<R>(a, at), of_lanes = attn_chunks(a, at);
  const AttnCut cut = attn_cut<R, WGS, uint64_t>(a, units, of_lanes, of_lane(wave_scan((uint64_t)units * of_lanes), 63),
                                              of_lane(wave_scan((uint64_t)units), 63));
  const uint64_t before = lane < b ? units * cut.stretch<uint64_t>(of_lanes) : 0;
  const uint64_t u0 = of_lane(wave_scan(before), 63) +
                      (uint64_t)(tile * a.heads + head) * cut.stretch<uint64_t>(chunks) + cut.cost;
  int w0;
  const int splits = attn_parts(a, u0, chunks, cut.each, w0);
  if (splits < 2) return;
  const uint32_t first = (uint32_t)(2 * w0 + 1) * kBytes;   // as the parts are placed by attn4_unit
  const auto place = [&](int s) { return s == 0 ? first : first + (uint32_t)(2 * s - 1) * kBytes; };
  const int part = threadIdx.x % kPer, side = threadIdx.x / kPer;
  constexpr int kFly = 8;
  f32x4 v[kFly];
  const auto fetch = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kFly; ++i)
      v[i] = *(const f32x4*)(a.parts + place(min(s0 + i * kSide + side, splits - 1)) + (uint32_t)(row * D + part * 4) * 4);
  };
  fetch(0);
  float top = kNoMax;
  for (int s = threadIdx.x; s < splits; s += 256) {
    const float* ml = (const float*)(a.parts + place(s) + R * D * 4) + row;
    sm[s] = ml[0];
    sl[s] = ml[R];
    top = __builtin_fmaxf(top, ml[0]);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o));
  if (lane == 0) smax[wave] = top;
  __syncthreads();
  top = __builtin_fmaxf(__builtin_fmaxf(smax[0], smax[1]), __builtin_fmaxf(smax[2], smax[3]));
  f32x4 acc{0, 0, 0, 0};
  float l = 0.0f;
  for (int s0 = 0; s0 < splits; s0 += kFly * kSide) {
    if (s0 > 0) fetch(s0);
#pragma unroll
    for (int i = 0; i < kFly; ++i) {
      const int s = s0 + i * kSide + side;
      const float r = s < splits ? half_power(sm[min(s, splits - 1)] - top) : 0.0f, w = r * r;
      l = __builtin_fmaf(sl[min(s, splits - 1)] * r, r, l);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(w, v[i][e], acc[e]);
    }
  }
  *(f32x4*)&red[side][part * 4] = acc;
  if (part == 0) ssum[side] = l;
  __syncthreads();
  if (side > 0) return;
  l = 0.0f;
  acc = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int y = 0; y < kSide; ++y) {
    l += ssum[y];
    acc += *(const f32x4*)&red[y][part * 4];
  }
  const int r = tile * R + row, oq = r / a.group, oh = head * a.group + r - oq * a.group;
  const float inv = l == 0.0f ? 0.0f : 0.001953125f / l;
  *(uint2*)(a.out + (rg.q0 + oq) * a.out_stride + (int64_t)oh * D + part * 4) =
      make_uint2(pack_bf16x2_rne(acc[0] * inv, acc[1] * inv), pack_bf16x2_rne(acc[2] * inv, acc[3] * inv));
  if (a.lse && part == 0)
    a.lse[(rg.q0 + oq) * a.q_heads + oh] =
        l == 0.0f ? -__builtin_inff() : (__builtin_log2f(l) + top) * 0.6931471805599453f;
}

// ------------------------------------------------------------------ many query rows
//
// Prompts and prompt pieces: waves of 32 query rows share the keys and values of 64 tokens at
// a time, which they bring to f16 in shared memory in the order in which the 32x32x16 MFMA takes
// them (one 16-byte slot a lane), two tiles in turn, so that one barrier a tile is enough.  The
// codes of the tile after are on their way in registers meanwhile.
//
// The rows' exponents go into the f16 values here, relative to the largest of each 16 tokens,
// E for keys and F for values: khat 2^(ek - E + 4), vhat 2^(ev - F + 4), at most 43008 and exact for
// rows down to 2^-18 of the largest.  A logit then takes one fused multiply-add with factors of its
// group, w = (acc kc 2^(E - 4)) + F, where a factor a token would cost two more of some nine vector
// instructions a logit, and the vector instructions (the exponential takes four of them) weigh as
// much as the matrix products.  Sixteen tokens with rows further apart (2^18 for keys, 2^5 for
// values) are held relative to their own exponents (E = ek, F = ev for each), and the tiles that have
// some take the longer way with factors a token: tokens that a query does not see are among the 16,
// and must not cost it the ones that it sees.
//
// At D = 128 a prompt of 8192 tokens, 28/4 heads, takes 505 us (952 TFLOP/s of the products that are
// seen; a library product reaches 1390), with the matrix units busy for 39% of the cycles and the
// vector units for 45%: little of the two overlaps.  Three ways to overlap more took more cycles than they
// saved (4 x 512 tokens behind 16384, against 1005 TFLOP/s in the same runs; matrix and vector units busy
// and clock on the prompt of 8192, against 41%, 45% and 1.94 GHz): products and exponentials of two tiles
// interleaved in a wave 907 (34%, 41%, 2.07), waves in two halves half a tile apart 912 (34%, 40%, 2.05),
// 64 rows a wave 699 (25%, 39%, 2.25).  Tiles of 128 tokens gave 976 against 990.
// The longer way costs nothing where few tiles take it (508 us with four small value rows at the start
// of the 8192) and 1.6 times the time where all do (values spread over 2^10 in every 16 tokens: 836).
constexpr int kPrTok = 64, kPrGroups = kPrTok / 16;
// Waves of a workgroup, and workgroups of a CU: at D = 128 eight waves, two a SIMD; at D = 64 three
// workgroups of four (40 sequences of up to 333 tokens in a window of 1024: 71 us against 88 with
// eight); at D = 256, where the sums of 32 rows take 128 registers, four with a SIMD each.
constexpr int prompt_waves(int d) { return d == 128 ? 8 : 4; }
constexpr int prompt_wgs_per_cu(int d) { return d == 64 ? 3 : 1; }
constexpr int prompt_rows(int d) { return 32 * prompt_waves(d); }
// Where the units leave CUs idle they are cut along the tokens (PromptCut), into as many parts as two
// rounds of workgroups hold at most; a kernel of its own joins them.  28/4 heads at D = 128, 512
// queries behind 2048 tokens: 44 us, 74 uncut; behind 4096: 61.  Not worth its launch where no
// sequence can have kPrCutFrom tokens.
constexpr int kPrPartTiles = 4, kPrCutFrom = 768, kPrJoinRows = 4;
int64_t prompt_units(int64_t total_q, int64_t batch, int64_t group, int64_t heads, int d) {
  return (total_q * group / prompt_rows(d) + batch) * heads;   // at most one tile a sequence more
}
int prompt_parts(int64_t units, int d) {
  const int64_t room = 2 * 256 * prompt_wgs_per_cu(d) / units;
  return room < 1 ? 1 : room > 64 ? 64 : (int)room;
}
__host__ __device__ constexpr size_t prompt_part_bytes(int d) { return (size_t)prompt_rows(d) * (d + 2) * 4; }

// What keeps a tile from the short way: a group that is left out; an ev outside the window that l may
// share; rows further apart than the gaps.  Keys are exact to 2^18.  F joins the logits, so m
// follows it: where the row that sets F is one that a query does not see, or that has no weight, all its other
// weights would lose F - ev of the bits below f16's smallest normal.  With 2^5 that is 2^-28 of the largest
// weighted value a token at most.
constexpr uint32_t kOddOut = 1, kOddFar = 2, kOddWide = 4;
constexpr uint32_t kPrKeyGap = 18, kPrValueGap = 5;

template <int D>
struct PromptShared {
  uint4 k[2][kPrTok / 32][D / 16][64];   // [tile][32 tokens][16 elements][lane]
  uint4 v[2][kPrGroups][D / 32][64];     // [tile][16 tokens][32 elements][lane]
  float ke[2][kPrGroups];                // 2^(E - 4), 0 for a group that is left out
  float2 vf[2][kPrGroups];               // F and 2^(-9 - F)
  __attribute__((aligned(8))) uint8_t odd[2][2][kPrGroups];   // kOdd.. of the groups' keys and values
  __attribute__((aligned(16))) float tke[2][kPrTok], tf[2][kPrTok];   // ke and F of each token (kOddWide)
  __attribute__((aligned(8))) _Float16 by[8][16];   // a wave's 2^(ev - F + 4) of 16 tokens
};

// 2^e as f16 for e <= 15 (0 below the format).
__device__ __forceinline__ _Float16 pow2_f16(int e) {
  return (_Float16)__uint_as_float((uint32_t)max(e + 127, 0) << 23);
}

// Keys of a group to f16 slots; the group's factor.  A token outside [0, valid) counts for nothing.
template <int D>
__device__ __forceinline__ void prompt_keys(PromptShared<D>& sh, int buf, int grp, const Keys4<D>& f, int lane,
                                            uint32_t valid) {
  constexpr int KW = D / 32;
  const int n16 = lane & 15, g = lane >> 4;
  const uint32_t e = (f.e >> (8 * (n16 & 3))) & 0xFFu;
  const uint32_t top = max_row16((valid >> n16 & 1) ? min(e, 244u) : 0u);
  const bool wide = (__ballot(e + kPrKeyGap < top) & valid) != 0;
  int off = (int)e - (int)top;
  if (__builtin_expect(wide, 0)) {
    off = 0;
    if (g == 0) sh.tke[buf][grp * 16 + n16] = __uint_as_float((uint32_t)max((int)e - 4, 0) << 23);
  }
  const f16x2 by = both(pow2_f16(off + 4));
  const uint32_t ks = f.ks >> ((8 * (D / 64) * g) & 31);
  const f16x2 s01 = scales2<false>(ks) * by, s23 = scales2<true>(ks) * by;
#pragma unroll
  for (int i = 0; i < KW; ++i) {
    const f16x2 sp = both((i >> 1) < 2 ? s01[(i >> 1) & 1] : s23[(i >> 1) & 1]);
    const int w = g * KW + i;   // elements 8 w ..
    sh.k[buf][grp >> 1][w >> 1][(w & 1) * 32 + (grp & 1) * 16 + n16] =
        __builtin_bit_cast(uint4, scaled8(f.k[i], sp, sp, sp, sp));
  }
  if (lane == 0) {
    sh.ke[buf][grp] = valid ? __uint_as_float((uint32_t)max((int)top - 4, 0) << 23) : 0.0f;
    sh.odd[buf][0][grp] = valid ? wide ? kOddWide : 0 : kOddOut;
  }
}

template <int D>
__device__ __forceinline__ void prompt_values(PromptShared<D>& sh, int buf, int grp, Values4<D>& f, uint32_t e4, int wave,
                                              int lane, uint32_t valid) {
  constexpr int KW = D / 32;
  const int m = lane & 15, g = lane >> 4;
  // lane % 16 works out its token's factor; a lane takes those of its four tokens
  const uint32_t e = (valid >> m & 1) ? min((e4 >> (8 * (m & 3))) & 0xFFu, 244u) : 0u;
  const uint32_t top = max_row16(e);
  const bool wide = (__ballot(e + kPrValueGap < top) & valid) != 0, far = (__ballot(e - kEvLow >= kEvSpan) & valid) != 0;
  int off = (int)e - (int)top;
  if (__builtin_expect(wide, 0)) {
    off = 0;
    if (g == 0) sh.tf[buf][grp * 16 + m] = (float)(int)e - 127.0f;
  }
  sh.by[wave][m] = pow2_f16(off + 4);
  __builtin_amdgcn_wave_barrier();
  if (valid != 0xFFFFu) {   // memory that was never written: no NaN from its scales
    const uint32_t mine = valid >> (4 * g) & 15u;
    const uint32_t mask = (mine & 1 ? 0xFFu : 0) | (mine & 2 ? 0xFF00u : 0) | (mine & 4 ? 0xFF0000u : 0) |
                          (mine & 8 ? 0xFF000000u : 0);
#pragma unroll
    for (int j = 0; j < KW; ++j) f.vs[j] &= mask;
  }
  const f16x2 by01 = *(const f16x2*)&sh.by[wave][4 * g], by23 = *(const f16x2*)&sh.by[wave][4 * g + 2];
#pragma unroll
  for (int j = 0; j < KW; ++j) {
    const f16x2 s01 = scales2<false>(f.vs[j]) * by01, s23 = scales2<true>(f.vs[j]) * by23;
    // nibbles of the even (low) and odd (high) elements of tokens (0, 1) to byte 0, (2, 3) to byte 2
    const uint32_t low = 0x000F000Fu, w = f.v[j], w4 = w >> 4, w8 = w >> 8;
    const uint32_t even = (w & low) | (w4 & ~low), odd = (w4 & low) | (w8 & ~low);
    const f16x2 e0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(even, 1.0f, 0) * s01;
    const f16x2 e1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(even, 1.0f, 2) * s23;
    const f16x2 o0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(odd, 1.0f, 0) * s01;
    const f16x2 o1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(odd, 1.0f, 2) * s23;
    uint2* at = (uint2*)&sh.v[buf][grp][j][(g & 1) * 32 + m] + (g >> 1);
    at[0] = make_uint2(__builtin_bit_cast(uint32_t, e0), __builtin_bit_cast(uint32_t, e1));
    at[32] = make_uint2(__builtin_bit_cast(uint32_t, o0), __builtin_bit_cast(uint32_t, o1));
  }
  if (lane == 0) {
    sh.vf[buf][grp] = make_float2((float)(int)top - 127.0f, __uint_as_float((245u - top) << 23));
    sh.odd[buf][1][grp] = (far ? kOddFar : 0) | (wide ? kOddWide : 0);
  }
}

// Unit `id`: (sequence, row tile, head), those that see the most tokens first, so that the last
// to start are the shortest (4 x 1024 causal, 32/8 heads: 64 us, 78 in the order of the sequences).  A
// tile's key is its sequence's context in row tiles less the tiles behind it: each wave finds the
// key T with fewer than `id` units above it by bisection, 64 sequences at a time.
template <int D>
__device__ __forceinline__ bool prompt_unit(const Attn4& a, uint32_t id, int& b, int& tile, int& h) {
  const int lane = threadIdx.x & 63;
  const uint32_t heads = (uint32_t)a.heads;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    AttnRange r{0, 0, 0, false};
    if (b0 + lane < a.batch) r = attn_range(a, b0 + lane);
    const int rows = r.nq * a.group;
    const int tiles = rows > a.few ? (rows + prompt_rows(D) - 1) / prompt_rows(D) : 0;
    // (of q_starts that do not rise the sums may pass 32 bits: what is found then is checked below)
    const uint32_t all = of_lane(wave_scan((uint32_t)tiles * heads), 63);
    if (id >= all) {
      id -= all;
      continue;
    }
    const int key = max((int)min((int64_t)r.n * a.group / prompt_rows(D), (int64_t)1 << 30), tiles);   // of the last tile; >= 1 of the first
    const uint64_t with = __ballot(tiles > 0);
    if ((with & (with - 1)) == 0) {   // one sequence
      const int j = __builtin_ctzll(with);
      b = b0 + j;
      tile = __builtin_amdgcn_readlane(tiles, j) - 1 - (int)(id / heads);
      h = (int)(id % heads);
      return true;
    }
    const auto above = [&](int t) { return of_lane(wave_scan((uint32_t)min(max(key - t, 0), tiles) * heads), 63); };
    int lo = 0, hi = (int)of_lane(wave_max((uint32_t)(tiles ? key : 0)), 63);   // above(hi) = 0 <= id < above(lo)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      (above(mid) > id ? lo : hi) = mid;
    }
    id -= above(hi);
    uint64_t at = __ballot(key - hi >= 0 && key - hi < tiles);   // sequences with a tile of the key hi
    for (uint32_t skip = id / heads; skip && at; --skip) at &= at - 1;
    if (!at) return false;
    const int j = __builtin_ctzll(at);
    b = b0 + j;
    tile = __builtin_amdgcn_readlane(tiles, j) - 1 - (__builtin_amdgcn_readlane(key, j) - hi);
    h = (int)(id % heads);
    return true;
  }
  return false;
}

// Tiles of 64 tokens that some row of the unit sees, from `first` on.
struct PromptTiles {
  int begin, stop, first, tiles;
};
template <int D>
__device__ __forceinline__ PromptTiles prompt_tiles(const Attn4& a, const AttnRange& rg, int tile) {
  const int r0 = tile * prompt_rows(D), live = min(rg.nq * a.group - r0, prompt_rows(D));
  const int qa = r0 / a.group, qz = (r0 + live - 1) / a.group;
  PromptTiles t;
  t.stop = a.causal ? rg.n - rg.nq + qz + 1 : rg.n;
  t.begin = a.window ? max(rg.n - rg.nq + qa + 1 - a.window, 0) : 0;
  t.first = t.begin & ~(kPrTok - 1);
  t.tiles = t.stop > t.first ? (t.stop - t.first + kPrTok - 1) / kPrTok : 0;
  return t;
}

// How the units are cut: their number, and the tiles of a part.  Parts of `each` tiles are to fit one
// round of workgroups or two: of units all alike as many each as fit, of others no more than
// sum / each + units together.  The cut is taken that ends first, where a workgroup's start takes
// the time of two or three tiles and the joining that of two; or none.
// (a.parts_each > 1 only for few units, which fit one round uncut: the sums stay in 32 bits.)
struct PromptCut {
  uint32_t units, each;
  __device__ __forceinline__ int parts(const Attn4& a, int tiles) const {
    return min(max((int)(((uint32_t)tiles + each - 1) / each), 1), a.parts_each);
  }
};
template <int D>
__device__ __forceinline__ PromptCut prompt_cut(const Attn4& a) {
  const int lane = threadIdx.x & 63;
  uint32_t sum = 0, units = 0, most = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    if (b0 + lane >= a.batch) continue;
    const AttnRange r = attn_range(a, b0 + lane);
    const int rows = r.nq * a.group;
    if (rows <= a.few || rows == 0) continue;
    const int n = (rows + prompt_rows(D) - 1) / prompt_rows(D);
    const uint32_t t0 = min(prompt_tiles<D>(a, r, 0).tiles, 1 << 20), t1 = min(prompt_tiles<D>(a, r, n - 1).tiles, 1 << 20);
    most = umax(most, umax(t0, t1));
    units += (uint32_t)n * (uint32_t)a.heads;
    sum += (t0 + t1) * (uint32_t)n * (uint32_t)a.heads;   // twice the tiles, about
  }
  constexpr uint32_t kSlots = 256 * prompt_wgs_per_cu(D);
  sum = of_lane(wave_scan(sum), 63) / 2;
  most = of_lane(wave_max(most), 63);
  PromptCut c;
  c.units = min(max(of_lane(wave_scan(units), 63), 1u), (uint32_t)a.most_units);   // (q_starts may not rise)
  c.each = max(most, 1u);
  uint32_t best = c.each;   // the time in tiles beyond one start
#pragma unroll
  for (uint32_t k = 1; k <= 2; ++k) {
    const uint32_t slots = k * kSlots;
    if (c.units > slots) continue;
    const uint32_t alike = slots / c.units;
    uint32_t each = (most + alike - 1) / alike;
    if (c.units < slots) each = min(each, sum / (slots - c.units) + 1);
    each = max(each, (uint32_t)kPrPartTiles);
    const uint32_t time = k * each + (5 * k - 5) / 2 + 2;
    if (time < best) {
      best = time;
      c.each = each;
    }
  }
  c.each = (uint32_t)__builtin_amdgcn_readfirstlane((int)c.each);
  return c;
}

template <int D>
__global__ __launch_bounds__(prompt_waves(D) * 64, prompt_waves(D) * prompt_wgs_per_cu(D) / 4) void attn4_prompt_kernel(Attn4 a) {
  constexpr int KS = D / 16, DT = D / 32, W = prompt_waves(D), kPrRows = prompt_rows(D), kAhead = 4;
  extern __shared__ __attribute__((aligned(16))) uint8_t raw[];
  PromptShared<D>& sh = *(PromptShared<D>*)raw;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n32 = lane & 31, half = lane >> 5;

  int b, tile, h;
  // the units' first parts, their second ones, ..: workgroups without work come last (between the
  // others, some CUs got two of those while some got none)
  PromptCut cut{1, 1};
  uint32_t unit = blockIdx.x, part = 0;
  if (a.parts_each > 1) {
    cut = prompt_cut<D>(a);
    part = (uint32_t)__builtin_amdgcn_readfirstlane((int)(unit / cut.units));
    unit -= part * cut.units;
    if (part >= (uint32_t)a.parts_each) return;
  }
  if (!prompt_unit<D>(a, unit, b, tile, h)) return;
  const AttnRange rg = attn_range_uniform(a, b);
  if (rg.bad && h == 0 && threadIdx.x == 0) atomicOr(a.status, (int32_t)kStatusBadItem);
  const int rows = rg.nq * a.group;
  const int r0 = tile * kPrRows;
  const int tile_live = min(rows - r0, kPrRows);
  const int qa = r0 / a.group, ra = r0 - qa * a.group;
  // this part's tiles and the tokens in them that some row of the workgroup sees
  const PromptTiles pt = prompt_tiles<D>(a, rg, tile);
  const int parts = __builtin_amdgcn_readfirstlane(cut.parts(a, pt.tiles));
  if ((int)part >= parts) return;
  const int x0 = __builtin_amdgcn_readfirstlane((int)((int64_t)pt.tiles * part / parts));
  const int tiles = __builtin_amdgcn_readfirstlane((int)((int64_t)pt.tiles * (part + 1) / parts)) - x0;
  const int first = pt.first + x0 * kPrTok;
  const int begin = max(pt.begin, first), stop = min(pt.stop, first + tiles * kPrTok);

  // this wave's rows and this lane's
  const int wr = wave * 32;
  const bool busy = wr < tile_live;
  const int row = min(ra + wr + n32, ra + tile_live - 1);
  const int dq = (int)((uint32_t)row / (uint32_t)a.group);
  const int head = h * a.group + row - dq * a.group;
  const int qrow = qa + dq;
  const int to = a.causal ? rg.n - rg.nq + qrow + 1 : rg.n;
  const int from = a.window ? to - a.window : 0;
  const int wq0 = qa + (ra + min(wr, tile_live - 1)) / a.group, wq1 = qa + (ra + min(wr + 31, tile_live - 1)) / a.group;
  const int end_w = a.causal ? rg.n - rg.nq + wq1 + 1 : rg.n;      // some row of the wave sees [begin_w, end_w)
  const int all_to = a.causal ? rg.n - rg.nq + wq0 + 1 : rg.n;     // every row sees [all_from, all_to)
  const int begin_w = a.window ? max(all_to - a.window, 0) : 0;
  const int all_from = a.window ? end_w - a.window : 0;

  // the tiles' codes: of 8 waves 2 x and 2 x + 1 take the keys and the values of group x, of 4 each both
  const int grp = W == 8 ? wave >> 1 : wave;
  const bool takes_keys = W == 4 || (wave & 1) == 0, takes_values = W == 4 || (wave & 1) != 0;
  const int32_t* table = a.table + (int64_t)b * a.table_stride;
  int pages = 0;   // lane x % 64: the page of this wave's group in tile x, -1 if there is none to read
  bool bad_page = false;
  const auto look_up = [&](int x0) {
    const int t = first + (x0 + lane) * kPrTok + grp * 16;
    pages = -1;
    if (t < stop && t + 16 > begin) {
      pages = table[t >> a.page_shift];
      if (pages < 0 || pages >= a.pages) {
        pages = -1;
        bad_page = true;
      }
    }
  };
  Lane4<D> lane_at(lane);
  lane_at.e = kv4_k_exps(D) + (lane & 12);   // the key rows' exponents in every lane
  Keys4<D> fk;
  Values4<D> fv;
  uint32_t fe = 0, valid = 0;
  const auto fetch = [&](int x) {
    const int t = first + x * kPrTok + grp * 16;
    const int pg = __builtin_amdgcn_readlane(pages, x & 63);
    const int64_t gi = (((int64_t)max(pg, 0) * a.heads + h) << (a.page_shift - 4)) +
                       ((t >> 4) & ((1 << (a.page_shift - 4)) - 1));
    const uint8_t* at = a.data + uniform((uint64_t)gi * kv4_group_bytes(D));
    // tokens of the group that may be read
    const int hi = pg < 0 ? 0 : min(max(stop - t, 0), 16), lo = min(max(begin - t, 0), 16);
    valid = ((1u << hi) - 1) & ~((1u << lo) - 1);
    if (takes_keys) load_keys<D>(fk, at, lane_at);
    if (takes_values) {
      load_values<D>(fv, at, lane_at);
      load_words<1>(&fe, group_rsrc<D>(at), kv4_v_exps(D) + (lane & 12));
    }
  };
  const auto put = [&](int buf) {
    if (takes_keys) prompt_keys<D>(sh, buf, grp, fk, lane, valid);
    if (takes_values) prompt_values<D>(sh, buf, grp, fv, fe, wave, lane, valid);
  };

  // the query rows as f16 with their largest magnitude in [2^14, 2^15) and the scale's sign, so that
  // kc > 0 and a logit of -inf stays -inf; a row with Inf or NaN is NaN throughout
  f16x8 q[KS];
  float kc, ke2;
  {
    const uint16_t* qp = a.q + (rg.q0 + qrow) * a.q_stride + (int64_t)head * D + half * 8;
    uint32_t amax = 0;
    uint4 x[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      x[s] = *(const uint4*)(qp + 16 * s);
      amax = umax(amax, hmax_u16x2(max_u16x2(max_u16x2(abs_bits2(x[s].x), abs_bits2(x[s].y)),
                                             max_u16x2(abs_bits2(x[s].z), abs_bits2(x[s].w)))));
    }
    amax = umax(amax, (uint32_t)__shfl_xor((int)amax, 32));
    const int e = amax ? (int)(amax >> 7) - 127 - 14 : 0;
    // scale 2^e in two factors, each with half the exponent: neither product with 2^(E - 4) leaves
    // float32 on the way to a number inside it
    const int x2 = e + __builtin_amdgcn_frexp_expf(a.scale_log2e);
    kc = a.scale_log2e == 0.0f ? 1.0f : __builtin_ldexpf(__builtin_fabsf(__builtin_amdgcn_frexp_mantf(a.scale_log2e)), x2 - (x2 >> 1));
    ke2 = __builtin_ldexpf(1.0f, x2 >> 1);
    const float sign = amax >= kBf16InfBits ? __builtin_nanf("") : a.scale_log2e > 0.0f ? 1.0f : a.scale_log2e < 0.0f ? -1.0f : 0.0f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint32_t w[4] = {x[s].x, x[s].y, x[s].z, x[s].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[s][2 * i] = (_Float16)(__builtin_ldexpf(bf16_lo(w[i]), -e) * sign);
        q[s][2 * i + 1] = (_Float16)(__builtin_ldexpf(bf16_hi(w[i]), -e) * sign);
      }
    }
  }

  f32x16 o[DT];
#pragma unroll
  for (int j = 0; j < DT; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;
  float m = 0.0f, l = 0.0f;
  float limit = kNoMax;   // m moves when w - m + 9 passes it: 15 once the row has seen a token
  uint32_t apart = 0;     // l is relative to ml, the largest logit
  float ml = kNoMax;

  if (tiles > 0) {
    look_up(0);
    fetch(0);
    put(0);
    if (tiles > 1) fetch(1);
  }
  __syncthreads();
  for (int x = 0; x < tiles; ++x) {
    const int buf = x & 1, t0 = first + x * kPrTok;
    if (x + 1 < tiles) {
      put(buf ^ 1);
      if (x + 2 < tiles) {
        if (((x + 2) & 63) == 0) look_up(x + 2);
        fetch(x + 2);
      }
    }
    if (busy && t0 < end_w && t0 + kPrTok > begin_w) {
      const uint2 odd2 = *(const uint2*)sh.odd[buf];   // (under way during the products)
      __builtin_amdgcn_sched_barrier(0);
      f32x16 c[2];
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) c[tt][i] = 0.0f;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
          c[tt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, sh.k[buf][tt][s][lane]), q[s], c[tt],
                                                         0, 0, 0);
      // the reads of the key fragments kAhead products ahead (the compiler puts each right before its use)
      __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
      for (int i = 0; i < 2 * KS - kAhead; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
      __builtin_amdgcn_sched_barrier(0);
      float w[2][16];   // (numbers of their own: as vectors they would be copied around the branches)
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) w[tt][i] = c[tt][i];
      // below 1e-37 a logit is 0; at most what float32 holds, for a key at right angles to the row (acc 0)
      const auto factor = [&](float ke) { return __builtin_amdgcn_fmed3f(ke * ke2 * kc, 1e-37f, 3.4e38f); };
      float kf[kPrGroups], vf[kPrGroups], lf[kPrGroups];
#pragma unroll
      for (int gr = 0; gr < kPrGroups; ++gr) {
        const float ke = sh.ke[buf][gr];
        kf[gr] = factor(ke);
        const float2 vv = sh.vf[buf][gr];
        vf[gr] = vv.x + (9.0f - m);
        lf[gr] = vv.y;
      }
      const uint32_t odd_k = (uint32_t)__builtin_amdgcn_readfirstlane((int)odd2.x);
      const uint32_t odd_v = (uint32_t)__builtin_amdgcn_readfirstlane((int)odd2.y);
      uint32_t back = 0;   // l is relative to ml in this tile alone
      if (__builtin_expect((odd_k | odd_v) != 0 || apart || t0 < all_from || t0 + kPrTok > all_to, 0)) {
        if ((odd_k & 0x01010101u * kOddOut) || t0 < all_from || t0 + kPrTok > all_to) {
          // a logit that the row does not see becomes -inf
#pragma unroll
          for (int tt = 0; tt < 2; ++tt)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int t = t0 + 32 * tt + 8 * (i >> 2) + 4 * half + (i & 3);
              if (!(t >= from && t < to && sh.ke[buf][2 * tt + (i >> 3)] != 0.0f)) w[tt][i] = -__builtin_inff();
            }
        }
        const bool wide = ((odd_k | odd_v) & 0x01010101u * kOddWide) != 0;
        if (wide) {
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const f32x4 ke = *(const f32x4*)&sh.tke[buf][8 * y + 4 * half];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[y >> 2][4 * (y & 3) + i] *=
                  odd_k >> (8 * (y >> 1)) & kOddWide ? factor(ke[i]) : kf[y >> 1];
          }
#pragma unroll
          for (int gr = 0; gr < kPrGroups; ++gr) kf[gr] = 1.0f;
        }
        if (apart || (odd_v & 0x01010101u * (kOddFar | kOddWide))) {
          if (!apart) ml = limit == 15.0f ? m : kNoMax;
          apart |= odd_v & 0x01010101u * kOddFar;
          back = apart == 0;
          float top = ml;
#pragma unroll
          for (int tt = 0; tt < 2; ++tt)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, w[tt][i] * kf[2 * tt + (i >> 3)]);
          top = __builtin_fmaxf(top, __shfl_xor(top, 32));
          l *= __builtin_amdgcn_exp2f(ml - top);
          ml = top;
#pragma unroll
          for (int tt = 0; tt < 2; ++tt)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              l += __builtin_amdgcn_exp2f(__builtin_fmaf(w[tt][i], kf[2 * tt + (i >> 3)], -top));
#pragma unroll
          for (int gr = 0; gr < kPrGroups; ++gr) lf[gr] = 0.0f;
        }
        if (wide) {
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const f32x4 f = *(const f32x4*)&sh.tf[buf][8 * y + 4 * half];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[y >> 2][4 * (y & 3) + i] += odd_v >> (8 * (y >> 1)) & kOddWide ? f[i] + (9.0f - m) : vf[y >> 1];
          }
#pragma unroll
          for (int gr = 0; gr < kPrGroups; ++gr) vf[gr] = 0.0f;
        }
      }
      float top = -__builtin_inff();
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int gr = 2 * tt + (i >> 3);
          w[tt][i] = __builtin_fmaf(w[tt][i], kf[gr], vf[gr]);
          top = __builtin_fmaxf(top, w[tt][i]);
        }
      if (__any(top > limit)) {   // the maximum moves
        top = __builtin_fmaxf(top, __shfl_xor(top, 32));
        const bool fresh = limit != 15.0f, any = top > kNoMax;
        const float up = any ? fresh ? top - 9.0f : __builtin_fmaxf(top - 9.0f, 0.0f) : 0.0f;
        const float shrink = fresh ? 0.0f : __builtin_amdgcn_exp2f(-up);
        m += up;
        limit = any ? 15.0f : limit;
        if (!apart && !back) l *= shrink;
#pragma unroll
        for (int j = 0; j < DT; ++j) o[j] *= shrink;
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
          for (int i = 0; i < 16; ++i) w[tt][i] -= up;
      }
      if (__builtin_expect(back != 0, 0)) l *= __builtin_amdgcn_exp2f(ml - (limit == 15.0f ? m : kNoMax));
#pragma unroll
      for (int gr = 0; gr < kPrGroups; ++gr) {
        f16x8 p;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = __builtin_amdgcn_exp2f(w[gr >> 1][8 * (gr & 1) + i]);
          sum += e;
          p[i] = (_Float16)e;
        }
        l = __builtin_fmaf(sum, lf[gr], l);
#pragma unroll
        for (int j = 0; j < DT; ++j)
          o[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, sh.v[buf][gr][j][lane]), p, o[j], 0,
                                                        0, 0);
      }
      // the value fragments kAhead products ahead, and the next group's exponentials beside the products
      __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 1);
      __builtin_amdgcn_sched_group_barrier(0x400, 8, 1);
      __builtin_amdgcn_sched_group_barrier(0x002, 13, 1);
#pragma unroll
      for (int i = 0; i < kPrGroups * DT; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 1);
        if (i < kPrGroups * DT - kAhead) __builtin_amdgcn_sched_group_barrier(0x100, 1, 1);
        if (i < 3 * DT) {
          __builtin_amdgcn_sched_group_barrier(0x400, 8 / DT, 1);
          __builtin_amdgcn_sched_group_barrier(0x002, 13 / DT, 1);
        }
      }
    }
    __syncthreads();
  }
  if (__any(bad_page) && lane == 0) atomicOr(a.status, (int32_t)kStatusBadItem);

  l += __shfl_xor(l, 32);
  if (apart && limit == 15.0f) {
    const float by = one_maximum(m, ml, l);
#pragma unroll
    for (int j = 0; j < DT; ++j) o[j] *= by;
  }
  if (wr + n32 >= tile_live) return;
  if (parts > 1) {   // this part's sums and their maximum, for the joining kernel
    float* to_part = (float*)(a.parts + ((size_t)unit * a.parts_each + part) * prompt_part_bytes(D));
    const int r = wr + n32;
#pragma unroll
    for (int j = 0; j < DT; ++j)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float* at = to_part + r * D + 32 * j + 16 * y + 8 * half;
        *(f32x4*)at = f32x4{o[j][4 * y], o[j][8 + 4 * y], o[j][4 * y + 1], o[j][8 + 4 * y + 1]};
        *(f32x4*)(at + 4) = f32x4{o[j][4 * y + 2], o[j][8 + 4 * y + 2], o[j][4 * y + 3], o[j][8 + 4 * y + 3]};
      }
    if (half == 0) {
      to_part[kPrRows * D + r] = limit == 15.0f ? m : kNoMax;
      to_part[kPrRows * D + kPrRows + r] = l;
    }
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.220703125e-4f / l;   // 2^-13; a row that sees nothing: zeros
  uint16_t* op = a.out + (rg.q0 + qrow) * a.out_stride + (int64_t)head * D + 8 * half;
#pragma unroll
  for (int j = 0; j < DT; ++j)
#pragma unroll
    for (int y = 0; y < 2; ++y) {  // elements 32 j + 16 y + 8 half ..
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2_rne(o[j][4 * y + i] * inv, o[j][8 + 4 * y + i] * inv);
      *(uint4*)(op + 32 * j + 16 * y) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  if (a.lse && half == 0)
    a.lse[(rg.q0 + qrow) * a.q_heads + head] =
        l == 0.0f ? -__builtin_inff() : (__builtin_log2f(l) + m) * 0.6931471805599453f;
}

// Joins the parts of the prompt kernel's units: D / 4 threads a row, four rows each (finding the
// unit takes as long as a row: 16 x 96 rows in two parts, 8 heads: 37 us, 46 with a row each).
template <int D>
__global__ __launch_bounds__(256) void attn4_prompt_join_kernel(Attn4 a) {
  constexpr int kPer = D / 4, kSide = 256 / kPer, ROWS = prompt_rows(D), kWgs = ROWS / (kPrJoinRows * kSide);
  int b, tile, h;
  const int unit = (int)blockIdx.x / kWgs;
  if (!prompt_unit<D>(a, unit, b, tile, h)) return;
  const AttnRange rg = attn_range_uniform(a, b);
  const int parts = prompt_cut<D>(a).parts(a, prompt_tiles<D>(a, rg, tile).tiles);
  const int live = rg.nq * a.group - tile * ROWS;
  const int r0 = (int)blockIdx.x % kWgs * (kPrJoinRows * kSide) + (int)threadIdx.x / kPer, part = (int)threadIdx.x % kPer;
  if (parts < 2 || r0 >= live) return;
  const float* from = (const float*)(a.parts + (size_t)unit * a.parts_each * prompt_part_bytes(D));
  constexpr size_t kStep = prompt_part_bytes(D) / 4;
  float top[kPrJoinRows], l[kPrJoinRows];
  f32x4 acc[kPrJoinRows];
  int r[kPrJoinRows];
#pragma unroll
  for (int i = 0; i < kPrJoinRows; ++i) {
    r[i] = r0 + i * kSide < live ? r0 + i * kSide : r0;
    top[i] = kNoMax;
    l[i] = 0.0f;
    acc[i] = f32x4{0, 0, 0, 0};
  }
#pragma unroll 2
  for (int s = 0; s < parts; ++s)
#pragma unroll
    for (int i = 0; i < kPrJoinRows; ++i) top[i] = __builtin_fmaxf(top[i], from[s * kStep + ROWS * D + r[i]]);
#pragma unroll 2
  for (int s = 0; s < parts; ++s)
#pragma unroll
    for (int i = 0; i < kPrJoinRows; ++i) {
      const float f = half_power(from[s * kStep + ROWS * D + r[i]] - top[i]), w = f * f;
      l[i] = __builtin_fmaf(from[s * kStep + ROWS * D + ROWS + r[i]] * f, f, l[i]);
      const f32x4 v = *(const f32x4*)(from + s * kStep + r[i] * D + part * 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = __builtin_fmaf(w, v[e], acc[i][e]);
    }
#pragma unroll
  for (int i = 0; i < kPrJoinRows; ++i) {
    if (r0 + i * kSide >= live) return;
    const int row = tile * ROWS + r[i], oq = row / a.group, oh = h * a.group + row - oq * a.group;
    const float inv = l[i] == 0.0f ? 0.0f : 1.220703125e-4f / l[i];
    *(uint2*)(a.out + (rg.q0 + oq) * a.out_stride + (int64_t)oh * D + part * 4) =
        make_uint2(pack_bf16x2_rne(acc[i][0] * inv, acc[i][1] * inv), pack_bf16x2_rne(acc[i][2] * inv, acc[i][3] * inv));
    if (a.lse && part == 0)
      a.lse[(rg.q0 + oq) * a.q_heads + oh] =
          l[i] == 0.0f ? -__builtin_inff() : (__builtin_log2f(l[i]) + top[i]) * 0.6931471805599453f;
  }
}

static_assert(attn_wgs(64) * 4 + kWsCounterOff <= kWsReserved, "one counter a workgroup");

// Sequences of more query rows a KV head than kFewRows take the prompt kernel, the others the
// few-row one; where the lengths are on the device both are launched, and each leaves the other's
// sequences out.  (32 sequences of 3000 tokens, 64/8 heads: 64 rows 50 us against 65 in the prompt kernel
// at D = 64, 82 against 79 at D = 128, 127 against 210 at D = 256; 128 rows 92 against 67, 148 against 84,
// 253 against 225.)  Up to twice the rows take the few-row kernel if the units are few enough: two
// sequences of 1000 tokens and 128 rows, 16 us against 27 at D = 64, 17 against 31 at D = 128, 28 against
// 73 at D = 256; eight of 8000 67 against 54, 101 against 105, 151 against 174.
constexpr int kFewRows = 64;
constexpr int few_units(int d) { return d == 256 ? 1024 : 384; }

// The prompt kernel's grid: 2^22 units of up to 512 threads.
bool attn4_launchable(int64_t batch, int64_t total_q, int64_t group, int64_t heads, int head_dim, int64_t max_q) {
  return max_q * group <= kFewRows || prompt_units(total_q, batch, group, heads, head_dim) <= (int64_t)1 << 22;
}

size_t attn4_scratch_bytes(int64_t batch, int64_t total_q, int64_t group, int64_t heads, int head_dim, int64_t max_q) {
  const size_t few = (size_t)2 * attn_wgs(head_dim) * 16 * (head_dim + 2) * 4;
  if (max_q * group <= kFewRows) return few;
  const int64_t units = prompt_units(total_q, batch, group, heads, head_dim);
  const int parts = prompt_parts(units, head_dim);
  const size_t many = parts > 1 ? (size_t)units * parts * prompt_part_bytes(head_dim) : 0;
  return many > few ? many : few;
}

// A second launch pays where units are cut into many parts: few units, and sequences that may be
// long enough.  28/4 heads: 1 x 8192 tokens (64 parts) 12.7 us against 15.9, 1 x 131072 (192) 29 against
// 47; 8 x 4096 (24) 15.6 against 14.0; 2 x 8192 of 64/8 heads (48) 15.7 against 16.0.
constexpr int kJoinParts = 48;

template <int D, int R>
static hipError_t launch_r(const Attn4& call, hipStream_t s) {
  Attn4 a = call;
  const int64_t rows = min((int64_t)a.max_q * a.group, (int64_t)a.few);   // of a sequence here
  const int64_t tiles = (rows + R - 1) / R, units = tiles * a.heads * a.batch;
  a.join = units * kJoinParts <= attn_wgs(D) && (a.table_pages << a.page_shift) >= kJoinParts * kAttnChunk;
  const int64_t chunks = (a.table_pages << a.page_shift) / kAttnChunk + 1 + kUnitCost;   // < 2^25
  a.wide = units > (int64_t)INT32_MAX / chunks;
  attn4_kernel<D, R><<<attn_wgs(D), kAttnWaves * 64, 0, s>>>(a);
  if (a.join) attn4_join_kernel<D, R><<<(unsigned)(units * R), 256, 0, s>>>(a, (int)tiles);
  return hipGetLastError();
}

template <int D>
static hipError_t launch_prompt(const Attn4& call, hipStream_t s) {
  Attn4 a = call;
  const int64_t units = prompt_units(a.total_q, a.batch, a.group, a.heads, D);
  // (no more than the longest sequence that the table holds can have)
  const int64_t room = a.table_pages << a.page_shift;
  a.most_units = (int)units;
  a.parts_each = room < kPrCutFrom ? 1 : (int)min((int64_t)prompt_parts(units, D), room / (kPrTok * kPrPartTiles));
  const size_t lds = sizeof(PromptShared<D>);
  const hipError_t e = hipFuncSetAttribute((const void*)attn4_prompt_kernel<D>,
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  attn4_prompt_kernel<D><<<(unsigned)(units * a.parts_each), prompt_waves(D) * 64, lds, s>>>(a);
  if (a.parts_each > 1)
    attn4_prompt_join_kernel<D><<<(unsigned)(units * (prompt_rows(D) * (D / 4) / (256 * kPrJoinRows))), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int D>
static hipError_t launch_d(const Attn4& call, hipStream_t s) {
  Attn4 a = call;
  const int64_t most = (int64_t)a.max_q * a.group;
  a.few = INT32_MAX;
  if (most <= 8) return launch_r<D, 8>(a, s);
  if (most <= kFewRows || (most <= 2 * kFewRows && (most + 15) / 16 * a.heads * a.batch <= few_units(D)))
    return launch_r<D, 16>(a, s);
  a.few = a.q_starts ? kFewRows : 0;
  const hipError_t e = launch_prompt<D>(a, s);
  if (e != hipSuccess || !a.q_starts) return e;
  return a.group <= 8 ? launch_r<D, 8>(a, s) : launch_r<D, 16>(a, s);
}

hipError_t launch_attn4(const Attn4& a, int head_dim, hipStream_t s) {
  if (head_dim == 64) return launch_d<64>(a, s);
  if (head_dim == 128) return launch_d<128>(a, s);
  return launch_d<256>(a, s);
}

}  // namespace ql
