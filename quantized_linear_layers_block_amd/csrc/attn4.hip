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
  const int64_t room = a.table_stride << a.page_shift;
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

// Registers of 16 tokens of one head as one lane takes them.
template <int D>
struct Keys4 {
  uint32_t k[D / 32];   // token lane % 16, elements (lane / 16) D / 4 on
  uint32_t ks;          // their D / 64 scales
  uint32_t e;           // an exponent byte: lanes 0..15 the key row's, the others the value row's of token lane % 16
};
template <int D>
struct Values4 {
  uint32_t v[D / 32];   // pair 16 j + lane % 16 of tokens 4 (lane / 16) + 0..3
  uint32_t vs[D / 32];  // their scales in block 2 j + (lane % 16) / 8
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t* dst, const uint8_t* p) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 x = *(const uint4*)(p + 16 * i);
      dst[4 * i] = x.x;
      dst[4 * i + 1] = x.y;
      dst[4 * i + 2] = x.z;
      dst[4 * i + 3] = x.w;
    }
  } else {
    const uint2 x = *(const uint2*)p;
    dst[0] = x.x;
    dst[1] = x.y;
  }
}

template <int D>
__device__ __forceinline__ void load_keys(Keys4<D>& f, const uint8_t* grp, int lane) {
  const int m = lane & 15, g = lane >> 4;
  load_words<D / 32>(f.k, grp + m * (D / 2) + g * (D / 8));
  const uint8_t* ks = grp + kv4_k_scales(D) + m * (D / 16) + g * (D / 64);
  if constexpr (D == 64) f.ks = *ks;
  if constexpr (D == 128) f.ks = *(const uint16_t*)ks;
  if constexpr (D == 256) f.ks = *(const uint32_t*)ks;
  f.e = grp[(g ? kv4_v_exps(D) : kv4_k_exps(D)) + m];
}
template <int D>
__device__ __forceinline__ void load_values(Values4<D>& f, const uint8_t* grp, int lane) {
  const int m = lane & 15, g = lane >> 4;
  load_words<D / 32>(f.v, grp + kv4_v_codes(D) + lane * (D / 8));
  load_words<D / 32>(f.vs, grp + kv4_v_scales(D) + g * (D / 4) + (m >> 3) * (D / 8));
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

// The call's work, cut on the device from the lengths that are there when it runs (so that a
// captured call follows them): an item is R query rows of one sequence and KV head against
// `span` of its tokens, `span` the same for every sequence and such that there are about
// kAttnItems of them; a sequence of at most `span` tokens is one item.  Items go (sequence,
// row tile, head, split).  Every wave works the cut out for itself, 64 sequences at a time.
constexpr int kAttnItems = 1024;  // four workgroups a CU
constexpr int kAttnStep = 32;     // tokens of one wave's step
struct AttnItem {
  int nq, n;
  int64_t q0;
  int b, tile, head, split, splits;
  int lo, span;  // first token of the sequence's range, tokens of a split
  int part;      // first of the splits' partial results, when there are more than one
};

__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
  for (int o = 32; o >= 1; o >>= 1) {
    const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, o), hi = (uint32_t)__shfl_xor((int)(v >> 32), o);
    v += ((uint64_t)hi << 32) | lo;
  }
  return v;
}

__device__ __forceinline__ int attn_lo(const Attn4& a, const AttnRange& r) {
  return a.window ? max(r.n - r.nq + 1 - a.window, 0) & ~(kAttnStep - 1) : 0;
}

template <int R>
__device__ __forceinline__ bool attn_item(const Attn4& a, int id, AttnItem& it) {
  const int lane = threadIdx.x & 63;
  const auto cost = [&](const AttnRange& r, int& tiles, int& tok) {
    tiles = (r.nq * a.group + R - 1) / R;
    tok = max(r.n - attn_lo(a, r), 0);
  };
  AttnRange first{0, 0, 0, false};
  uint64_t sum = 0;
  bool bad = false;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    if (b0 + lane >= a.batch) continue;
    const AttnRange r = attn_range(a, b0 + lane);
    if (b0 == 0) first = r;
    int tiles, tok;
    cost(r, tiles, tok);
    sum += (uint64_t)tiles * (uint64_t)tok;
    bad |= r.bad;
  }
  if (blockIdx.x == 0 && threadIdx.x < 64 && __any(bad) && lane == 0) atomicOr(a.status, (int32_t)kStatusBadItem);
  sum = wave_sum_u64(sum) * (uint64_t)a.heads;
  constexpr int kWgStep = kAttnWaves * kAttnStep;
  const uint64_t want = (sum + kAttnItems - 1) / kAttnItems;
  const int span = want <= kWgStep ? kWgStep : (int)min((want + kWgStep - 1) / kWgStep * kWgStep, (uint64_t)1 << 30);
  int items = 0, parts = 0;  // of the sequences before b0
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    AttnRange r{0, 0, 0, false};
    int tiles = 0, tok = 0;
    if (b0 + lane < a.batch) {
      r = b0 == 0 ? first : attn_range(a, b0 + lane);
      cost(r, tiles, tok);
    }
    const int splits = tok > span ? (int)((uint32_t)(tok + span - 1) / (uint32_t)span) : 1;
    const int mine = tiles * a.heads * splits, pmine = splits > 1 ? mine : 0;
    int upto = mine, pupto = pmine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(upto, o), y = __shfl_up(pupto, o);
      if (lane >= o) {
        upto += x;
        pupto += y;
      }
    }
    const uint64_t past = __ballot(items + upto > id);
    if (past) {
      const int j = __builtin_ctzll(past);
      const int local = id - items - __builtin_amdgcn_readlane(upto - mine, j);
      it.splits = __builtin_amdgcn_readlane(splits, j);
      it.split = local % it.splits;
      const int th = local / it.splits;
      it.tile = th / a.heads;
      it.head = th - it.tile * a.heads;
      it.part = parts + __builtin_amdgcn_readlane(pupto - pmine, j) + th * it.splits;
      it.b = b0 + j;
      it.nq = __builtin_amdgcn_readlane(r.nq, j);
      it.n = __builtin_amdgcn_readlane(r.n, j);
      it.q0 = ((int64_t)__builtin_amdgcn_readlane((int)(r.q0 >> 32), j) << 32) |
              (uint32_t)__builtin_amdgcn_readlane((int)r.q0, j);
      it.span = span;
      it.lo = a.window ? max(it.n - it.nq + 1 - a.window, 0) & ~(kAttnStep - 1) : 0;
      return true;
    }
    items += __builtin_amdgcn_readlane(upto, 63);
    parts += __builtin_amdgcn_readlane(pupto, 63);
  }
  return false;
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

// One workgroup an item; the waves take alternate 32-token steps and their sums are joined
// through shared memory.  Of a split sequence, the workgroup that arrives last joins the
// splits' results, in their order.
//
// A lane's dword of V holds an even and an odd element of four tokens, and the conversion
// gives them as pairs.  The pairs stay together as neighbours along the product's depth,
// with P beside zeros: [p 0] takes the even elements and [0 p] the odd ones.  That doubles the
// matrix instructions of the second product, which have room, and saves the vector
// instructions that would part the pairs, which have none.  With R = 8 rows the two are the
// two halves of the 16 columns of one product, with R = 16 two products.
template <int D, int R>
__global__ __launch_bounds__(kAttnWaves * 64, D == 64 ? 4 : D == 128 ? 3 : 2) void attn4_kernel(Attn4 a) {
  constexpr int KW = D / 32, kRow = D + 4, P = R / 8;
  __shared__ float so[kAttnWaves][R][kRow];
  __shared__ float sm[kAttnWaves][R], sl[kAttnWaves][R];
  __shared__ __attribute__((aligned(16))) float sx[kAttnWaves][2][64];
  __shared__ int last;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  const int rn = R == 16 ? n16 : n16 & 7;                 // this lane's query row of the tile
  const int odd_shift = R == 16 ? 16 : (n16 >> 3) << 4;   // where p goes beside its zero
  AttnItem it;
  if (!attn_item<R>(a, blockIdx.x, it)) return;
  const int h = it.head;
  const int rows = it.nq * a.group;
  const int r0 = it.tile * R;
  const int live = min(rows - r0, R);   // rows of the tile; lanes past them repeat the last

  // the query tokens of the tile, this lane's, and the tokens [from, to) that it sees
  const int qa = r0 / a.group, ra = r0 - qa * a.group;
  const int qb = qa + small_div(ra + live - 1, a.group);
  const int mine_r = min(rn, live - 1);
  const int dq = small_div(ra + mine_r, a.group);
  const int head = h * a.group + ra + mine_r - dq * a.group;
  const int to = a.causal ? it.n - it.nq + qa + dq + 1 : it.n;
  const int from = a.window ? to - a.window : 0;
  const int end = a.causal ? it.n - it.nq + qb + 1 : it.n;         // some row sees [begin, end)
  const int all_to = a.causal ? it.n - it.nq + qa + 1 : it.n;      // every row sees [all_from, all_to)
  const int begin = a.window ? max(all_to - a.window, 0) : 0;
  const int all_from = a.window ? end - a.window : 0;
  const int lo = it.lo + it.split * it.span;
  const int hi = it.split + 1 < it.splits ? min(end, lo + it.span) : end;

  // the query row as f16 with its largest magnitude in [2^14, 2^15)
  f16x8 q[KW];
  float kc;
  {
    uint4 x[KW];
    const uint16_t* qp = a.q + (it.q0 + qa + dq) * a.q_stride + (int64_t)head * D + g * (D / 4);
    uint32_t amax = 0;
#pragma unroll
    for (int s = 0; s < KW; ++s) {
      x[s] = *(const uint4*)(qp + 8 * s);
      u16x2 t = max_u16x2(max_u16x2(abs_bits2(x[s].x), abs_bits2(x[s].y)),
                          max_u16x2(abs_bits2(x[s].z), abs_bits2(x[s].w)));
      amax = umax(amax, hmax_u16x2(t));
    }
    amax = umax(amax, (uint32_t)__shfl_xor((int)amax, 16));
    amax = umax(amax, (uint32_t)__shfl_xor((int)amax, 32));
    const int e = amax ? (int)(amax >> 7) - 127 - 14 : 0;   // subnormal rows: -141, still exact
    kc = __builtin_ldexpf(a.scale_log2e, e);
    if (amax >= kBf16InfBits) kc = __builtin_nanf("");
#pragma unroll
    for (int s = 0; s < KW; ++s) {
      const uint32_t w[4] = {x[s].x, x[s].y, x[s].z, x[s].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[s][2 * i] = (_Float16)__builtin_ldexpf(bf16_lo(w[i]), -e);
        q[s][2 * i + 1] = (_Float16)__builtin_ldexpf(bf16_hi(w[i]), -e);
      }
    }
  }

  f32x4 o[P][KW];
#pragma unroll
  for (int y = 0; y < P; ++y)
#pragma unroll
    for (int j = 0; j < KW; ++j) o[y][j] = f32x4{0, 0, 0, 0};
  float m = kNoMax, l = 0.0f;
  const int32_t* table = a.table + (int64_t)it.b * a.table_stride;
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
    return a.data + gi * kv4_group_bytes(D);
  };

  Keys4<D> f[2];
  Values4<D> fv[2];
  const uint8_t* grp[2];
  bool ok[2] = {false, false};
  int x = 0;
  if (lo + wave * 32 < hi) {
    look_up(0);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      ok[u] = __builtin_amdgcn_readlane(pages, u) >= 0;
      grp[u] = group_at(u, lo + wave * 32 + 16 * u);
      load_keys<D>(f[u], grp[u], lane);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) load_values<D>(fv[u], grp[u], lane);
  }
  for (int t0 = lo + wave * 32; t0 < hi; t0 += kAttnWaves * 32) {
    // what depends on the token alone is worked out by one lane a token and shared: 2^ek, ev + 127
    // and 2^(-9 - ev) at 0, 16 and 32 of sx
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t b23 = f[u].e << 23;
      const float ve = (float)f[u].e;
      const float w = g == 0 ? __uint_as_float(b23) : g == 1 ? ve : __uint_as_float((245u << 23) - b23);
      sx[wave][u][lane] = w;
    }
    __builtin_amdgcn_wave_barrier();
    f32x4 c[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const f16x2 s01 = scales2<false>(f[u].ks), s23 = scales2<true>(f[u].ks);
      c[u] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KW; ++s) {
        const f16x2 sp = both((s >> 1) < 2 ? s01[(s >> 1) & 1] : s23[(s >> 1) & 1]);
        c[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(scaled8(f[u].k[s], sp, sp, sp, sp), q[s], c[u], 0, 0, 0);
      }
    }
    f32x4 kf[2], ve[2], lf[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      kf[u] = *(const f32x4*)&sx[wave][u][4 * g];
      ve[u] = *(const f32x4*)&sx[wave][u][16 + 4 * g];
      lf[u] = *(const f32x4*)&sx[wave][u][32 + 4 * g];
      kf[u] *= kc;
      const int t = t0 + 16 * u;
      if (!ok[u] || t < all_from || t + 16 > all_to) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = t + 4 * g + i;
          if (!(ok[u] && tok >= from && tok < to)) {
            c[u][i] = 0.0f;
            kf[u][i] = 0.0f;
            ve[u][i] = -__builtin_inff();
            lf[u][i] = 0.0f;
          }
        }
        // tokens that no row sees may be memory that was never written: no NaN from their scales
        const int t4 = t + 4 * g;
        const int skip = min(max(begin - t4, 0), 4), keep = ok[u] ? min(max(it.n - t4, 0), 4) : 0;
        const uint32_t mask = (uint32_t)(((uint64_t)1 << (8 * keep)) - 1) & ~(uint32_t)(((uint64_t)1 << (8 * skip)) - 1);
#pragma unroll
        for (int j = 0; j < KW; ++j) fv[u].vs[j] &= mask;
      }
    }
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
        load_keys<D>(f[u], grp[u], lane);
      }
    }
    float p[2][4], top = -__builtin_inff();
    const float base = 9.0f - 127.0f - m;   // ve holds ev + 127
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[u][i] = __builtin_fmaf(c[u][i], kf[u][i], ve[u][i] + base);
        top = __builtin_fmaxf(top, p[u][i]);
      }
    if (__any(top > 15.0f)) {  // the maximum moves: w again in full, the sums to the new one
      float w = -__builtin_inff();
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[u][i] = __builtin_fmaf(c[u][i], kf[u][i], ve[u][i] - 127.0f);
          w = __builtin_fmaxf(w, p[u][i]);
        }
      w = __builtin_fmaxf(w, __shfl_xor(w, 16));
      w = __builtin_fmaxf(w, __shfl_xor(w, 32));
      const float mn = __builtin_fmaxf(m, w), shrink = __builtin_exp2f(m - mn);
      m = mn;
      l *= shrink;
#pragma unroll
      for (int y = 0; y < P; ++y)
#pragma unroll
        for (int j = 0; j < KW; ++j) o[y][j] *= shrink;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[u][i] = p[u][i] - m + 9.0f;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
      u32x4 pe, po;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = __builtin_amdgcn_exp2f(p[u][i]);
        l = __builtin_fmaf(e, lf[u][i], l);
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
#pragma unroll
    for (int u = 0; u < 2; ++u) load_values<D>(fv[u], grp[u], lane);
  }
  if (__any(bad_page) && lane == 0) atomicOr(a.status, (int32_t)kStatusBadItem);

  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
#pragma unroll
  for (int y = 0; y < P; ++y)
#pragma unroll
    for (int j = 0; j < KW; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        so[wave][rn][32 * j + 8 * g + 2 * i + (R == 16 ? y : n16 >> 3)] = o[y][j][i];
  if (g == 0 && n16 < R) {
    sm[wave][rn] = m;
    sl[wave][rn] = l;
  }
  __syncthreads();
  // E elements of a row a thread
  constexpr int E = R * D / (kAttnWaves * 64) < 4 ? 4 : R * D / (kAttnWaves * 64), kPer = D / E;
  const int orow = threadIdx.x / kPer, part = threadIdx.x % kPer;
  const bool mine = orow < live;
  const int src = mine ? orow : 0;
  float top = sm[0][src];
#pragma unroll
  for (int w = 1; w < kAttnWaves; ++w) top = __builtin_fmaxf(top, sm[w][src]);
  float acc[E], lsum = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll
  for (int w = 0; w < kAttnWaves; ++w) {
    const float s = __builtin_exp2f(sm[w][src] - top);
    lsum += s * sl[w][src];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += s * so[w][src][part * E + e];
  }
  if (it.splits > 1) {
    constexpr uint32_t kBytes = attn_part_bytes<D, R>();
    const __amdgpu_buffer_rsrc_t rs = dev_rsrc(a.parts);
    const uint32_t at = (uint32_t)(it.part + it.split) * kBytes;
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
    wait_stores();
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t* c = a.counters + it.part;
      const uint32_t old = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = old == (uint32_t)it.splits - 1;
      if (last) st_dev_u32(c, 0u);
    }
    __syncthreads();
    if (!last || !mine) return;
    const uint32_t first = (uint32_t)it.part * kBytes;
    const uint32_t* ml = (const uint32_t*)(a.parts + first + R * D * 4) + src;
    top = kNoMax;
    for (int s = 0; s < it.splits; ++s) top = __builtin_fmaxf(top, __uint_as_float(ld_dev_u32(ml + s * (kBytes / 4))));
    lsum = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll 4
    for (int s = 0; s < it.splits; ++s) {
      const float w = __builtin_exp2f(__uint_as_float(ld_dev_u32(ml + s * (kBytes / 4))) - top);
      lsum += w * __uint_as_float(ld_dev_u32(ml + s * (kBytes / 4) + R));
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const f32x4 v = ld_dev4v(rs, first + (uint32_t)s * kBytes + mine_at + 4 * e);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[e + i] += w * v[i];
      }
    }
  }
  if (!mine) return;
  const int oq = qa + small_div(ra + src, a.group), oh = h * a.group + (r0 + src) - oq * a.group;
  const float inv = lsum == 0.0f ? 0.0f : 0.001953125f / lsum;  // a row that sees nothing: zeros
  uint16_t* op = a.out + (it.q0 + oq) * a.out_stride + (int64_t)oh * D + part * E;
#pragma unroll
  for (int e = 0; e < E; e += 4)
    *(uint2*)(op + e) = make_uint2(pack_bf16x2_rne(acc[e] * inv, acc[e + 1] * inv),
                                   pack_bf16x2_rne(acc[e + 2] * inv, acc[e + 3] * inv));
  if (a.lse && part == 0)
    a.lse[(it.q0 + oq) * a.q_heads + oh] =
        lsum == 0.0f ? -__builtin_inff() : (__builtin_log2f(lsum) + top) * 0.6931471805599453f;
}

// Items of split sequences: each has fewer than 2 tokens / span of them, so at most 2 kAttnItems.
static_assert(2 * kAttnItems * 4 + kWsCounterOff <= kWsReserved, "one counter a split item");

size_t attn4_scratch_bytes(int32_t head_dim) { return (size_t)2 * kAttnItems * 16 * (head_dim + 2) * 4; }

template <int D, int R>
static hipError_t launch_r(const Attn4& a, hipStream_t s) {
  // every R rows of every KV head, at most one tile a sequence more, and the splits
  const int64_t tiles = a.total_q * a.group / R + a.batch;
  const int64_t items = tiles * a.heads + kAttnItems;
  if (items > (int64_t)INT32_MAX) return hipErrorInvalidValue;
  attn4_kernel<D, R><<<(unsigned)items, kAttnWaves * 64, 0, s>>>(a);
  return hipGetLastError();
}

template <int D>
static hipError_t launch_d(const Attn4& a, hipStream_t s) {
  return (int64_t)a.max_q * a.group <= 8 ? launch_r<D, 8>(a, s) : launch_r<D, 16>(a, s);
}

hipError_t launch_attn4(const Attn4& a, int head_dim, hipStream_t s) {
  if (head_dim == 64) return launch_d<64>(a, s);
  if (head_dim == 128) return launch_d<128>(a, s);
  return launch_d<256>(a, s);
}

}  // namespace ql
