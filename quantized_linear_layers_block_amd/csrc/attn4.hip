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
struct Frag4 {
  uint32_t k[D / 32];   // token lane % 16, elements (lane / 16) D / 4 on
  uint32_t ks;          // their D / 64 scales
  uint32_t ke, ve;      // exponent bytes of tokens 4 (lane / 16) + 0..3
  uint32_t v[D / 32];   // pair 16 j + lane % 16 of those tokens
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
__device__ __forceinline__ void load_frag(Frag4<D>& f, const uint8_t* grp, int lane) {
  const int m = lane & 15, g = lane >> 4;
  load_words<D / 32>(f.k, grp + m * (D / 2) + g * (D / 8));
  const uint8_t* ks = grp + kv4_k_scales(D) + m * (D / 16) + g * (D / 64);
  if constexpr (D == 64) f.ks = *ks;
  if constexpr (D == 128) f.ks = *(const uint16_t*)ks;
  if constexpr (D == 256) f.ks = *(const uint32_t*)ks;
  f.ke = *(const uint32_t*)(grp + kv4_k_exps(D) + 4 * g);
  load_words<D / 32>(f.v, grp + kv4_v_codes(D) + lane * (D / 8));
  load_words<D / 32>(f.vs, grp + kv4_v_scales(D) + g * (D / 4) + (m >> 3) * (D / 8));
  f.ve = *(const uint32_t*)(grp + kv4_v_exps(D) + 4 * g);
}

// Eight key elements times their scale (0xFF, a NaN token, gives NaN).
__device__ __forceinline__ f16x8 key8(uint32_t codes, uint32_t scale_byte) {
  const uint32_t s = (scale_byte << 7) & 0x7F80u;
  const f16x2 sp = __builtin_bit_cast(f16x2, s | (s << 16));
  const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 256.0f, 0) * sp;
  const f16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 256.0f, 1) * sp;
  const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 256.0f, 2) * sp;
  const f16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 256.0f, 3) * sp;
  return f16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

struct ValuePair {  // four tokens of the even and of the odd element
  f16x2 even[2], odd[2];
};

// One dword of V (a pair of elements of four tokens) times the four tokens' scales.  A scale
// byte of unwritten memory may be anything: bit 7 is dropped, which leaves finite numbers.
__device__ __forceinline__ ValuePair value4(uint32_t w, uint32_t scales) {
  const uint32_t s = scales & 0x7F7F7F7Fu;
  const f16x2 s01 = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0u, s, 0x010C000Cu) >> 1);
  const f16x2 s23 = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0u, s, 0x030C020Cu) >> 1);
  // nibbles of the even (low) and odd (high) elements of tokens (0, 1) to byte 0, (2, 3) to byte 2
  const uint32_t m = 0x000F000Fu, w4 = w >> 4, w8 = w >> 8;
  const uint32_t ev = (w & m) | (w4 & ~m), od = (w4 & m) | (w8 & ~m);
  ValuePair r;
  r.even[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(ev, 256.0f, 0) * s01;
  r.even[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(ev, 256.0f, 2) * s23;
  r.odd[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(od, 256.0f, 0) * s01;
  r.odd[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(od, 256.0f, 2) * s23;
  return r;
}

__device__ __forceinline__ f16x8 join8(const f16x2* a, const f16x2* b) {
  return f16x8{a[0][0], a[0][1], a[1][0], a[1][1], b[0][0], b[0][1], b[1][0], b[1][1]};
}

// One workgroup: 16 query rows (token, head of the group) of one sequence and KV head; the
// waves take alternate 32-token steps and their sums are joined through shared memory.
template <int D>
__global__ __launch_bounds__(kAttnWaves * 64) void attn4_kernel(Attn4 a) {
  constexpr int KW = D / 32, kRow = D + 4;
  __shared__ float so[kAttnWaves][16][kRow];
  __shared__ float sm[kAttnWaves][16], sl[kAttnWaves][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  const int b = blockIdx.z, h = blockIdx.y;
  const AttnRange rg = attn_range(a, b);
  if (rg.bad && threadIdx.x == 0 && h == 0 && blockIdx.x == 0) atomicOr(a.status, (int32_t)kStatusBadItem);
  const int rows = rg.nq * a.group;
  const int r0 = blockIdx.x * 16;
  if (r0 >= rows) return;

  // this lane's query row, and the tokens [from, to) that it sees
  const int row = r0 + n16;
  const bool live = row < rows;
  const int qi = (live ? row : rows - 1) / a.group;
  const int head = h * a.group + (live ? row : rows - 1) - qi * a.group;
  const int to = a.causal ? rg.n - rg.nq + qi + 1 : rg.n;
  const int from = a.window ? to - a.window : 0;
  // the tile's first and last row bound what the workgroup reads
  const int qa = r0 / a.group, qb = (r0 + 16 < rows ? r0 + 15 : rows - 1) / a.group;
  const int hi = a.causal ? rg.n - rg.nq + qb + 1 : rg.n;          // some row sees [lo, hi)
  const int lo = a.window ? max(rg.n - rg.nq + qa + 1 - a.window, 0) & ~31 : 0;
  const int all_to = a.causal ? rg.n - rg.nq + qa + 1 : rg.n;      // every row sees [all_from, all_to)
  const int all_from = a.window ? hi - a.window : 0;

  // the query row as f16 with its largest magnitude in [2^14, 2^15)
  f16x8 q[KW];
  float kc;
  {
    uint4 x[KW];
    const uint16_t* qp = a.q + (rg.q0 + qi) * a.q_stride + (int64_t)head * D + g * (D / 4);
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

  f32x4 o[2 * KW];
#pragma unroll
  for (int j = 0; j < 2 * KW; ++j) o[j] = f32x4{0, 0, 0, 0};
  float m = kNoMax, l = 0.0f;
  const int32_t* table = a.table + (int64_t)b * a.table_stride;
  const int per = 1 << (a.page_shift - 4);
  bool bad_page = false;

  for (int t0 = lo + wave * 32; t0 < hi; t0 += kAttnWaves * 32) {
    Frag4<D> f[2];
    bool ok[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = t0 + 16 * u < hi ? t0 + 16 * u : t0;   // a second group past the end: the first again, masked
      const int64_t pg = table[t >> a.page_shift];
      ok[u] = pg >= 0 && pg < a.pages;
      bad_page |= !ok[u];
      ok[u] = ok[u] && t0 + 16 * u < hi;
      const int64_t gi = (((pg >= 0 && pg < a.pages ? pg : 0) * a.heads + h) << (a.page_shift - 4)) + ((t >> 4) & (per - 1));
      load_frag<D>(f[u], a.data + gi * kv4_group_bytes(D), lane);
    }
    f32x4 c[2];
    float kf[2][4], ve[2][4], lf[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      c[u] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KW; ++s)
        c[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key8(f[u].k[s], (f[u].ks >> (8 * (s >> 1))) & 0xFFu), q[s], c[u],
                                                      0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t eb = (f[u].ke >> (8 * i)) & 0xFFu, vb = (f[u].ve >> (8 * i)) & 0xFFu;
        kf[u][i] = __uint_as_float(eb << 23) * kc;
        ve[u][i] = (float)vb;
        lf[u][i] = __uint_as_float((245u - vb) << 23);
      }
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
      for (int j = 0; j < 2 * KW; ++j) o[j] *= shrink;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[u][i] = p[u][i] - m + 9.0f;
    }
    f16x8 pf;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = __builtin_amdgcn_exp2f(p[u][i]);
        l = __builtin_fmaf(x, lf[u][i], l);
        pf[4 * u + i] = (_Float16)x;
      }
#pragma unroll
    for (int j = 0; j < KW; ++j) {
      const ValuePair v0 = value4(f[0].v[j], f[0].vs[j]), v1 = value4(f[1].v[j], f[1].vs[j]);
      o[2 * j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(join8(v0.even, v1.even), pf, o[2 * j], 0, 0, 0);
      o[2 * j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(join8(v0.odd, v1.odd), pf, o[2 * j + 1], 0, 0, 0);
    }
  }
  if (bad_page && lane == 0) atomicOr(a.status, (int32_t)kStatusBadItem);

  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
#pragma unroll
  for (int j = 0; j < KW; ++j)  // elements 32 j + 8 g + 2 i (even) and + 1 (odd)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      so[wave][n16][32 * j + 8 * g + 2 * i] = o[2 * j][i];
      so[wave][n16][32 * j + 8 * g + 2 * i + 1] = o[2 * j + 1][i];
    }
  if (g == 0) {
    sm[wave][n16] = m;
    sl[wave][n16] = l;
  }
  __syncthreads();
  // 16 threads a row, D / 16 elements each
  constexpr int E = D / 16;
  const int orow = threadIdx.x >> 4, part = threadIdx.x & 15;
  if (r0 + orow >= rows) return;
  float top = sm[0][orow];
#pragma unroll
  for (int w = 1; w < kAttnWaves; ++w) top = __builtin_fmaxf(top, sm[w][orow]);
  float acc[E], lsum = 0.0f;
#pragma unroll
  for (int x = 0; x < E; ++x) acc[x] = 0.0f;
#pragma unroll
  for (int w = 0; w < kAttnWaves; ++w) {
    const float s = __builtin_exp2f(sm[w][orow] - top);
    lsum += s * sl[w][orow];
#pragma unroll
    for (int x = 0; x < E; ++x) acc[x] += s * so[w][orow][part * E + x];
  }
  const int oq = (r0 + orow) / a.group, oh = h * a.group + (r0 + orow) - oq * a.group;
  const float inv = lsum == 0.0f ? 0.0f : 0.001953125f / lsum;  // a row that sees nothing: zeros
  uint16_t* op = a.out + (rg.q0 + oq) * a.out_stride + (int64_t)oh * D + part * E;
#pragma unroll
  for (int x = 0; x < E; x += 2) *(uint32_t*)(op + x) = pack_bf16x2_rne(acc[x] * inv, acc[x + 1] * inv);
  if (a.lse && part == 0)
    a.lse[(rg.q0 + oq) * a.q_heads + oh] =
        lsum == 0.0f ? -__builtin_inff() : (__builtin_log2f(lsum) + top) * 0.6931471805599453f;
}

size_t attn4_scratch_bytes(int64_t batch, int64_t total_q, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                           int32_t max_q) {
  (void)batch, (void)total_q, (void)q_heads, (void)kv_heads, (void)head_dim, (void)max_q;
  return 0;
}

hipError_t launch_attn4(const Attn4& a, int head_dim, void* scratch, hipStream_t s) {
  (void)scratch;
  const dim3 grid((unsigned)(((int64_t)a.max_q * a.group + 15) / 16), (unsigned)a.heads, (unsigned)a.batch);
  if (head_dim == 64) attn4_kernel<64><<<grid, kAttnWaves * 64, 0, s>>>(a);
  if (head_dim == 128) attn4_kernel<128><<<grid, kAttnWaves * 64, 0, s>>>(a);
  if (head_dim == 256) attn4_kernel<256><<<grid, kAttnWaves * 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ql
