// The gate of the feed-forward block, g / (1 + exp(-g)) u, and its derivatives in float32, for the kernels of
// both directions.
#pragma once
#include "common.hpp"

namespace ql {

// exp(-g) = 2^t with t = -g log2(e): what the product's rounding lost goes back in as a factor 1 + d ln 2, so the
// result is within a few units of 2^-24.  Beyond +-128 it is 0 or infinite in float32 anyhow (and 1 / (1 + it) exactly
// 1 or 0).
__device__ __forceinline__ float gate_exp(float g) {
  const float c = __builtin_amdgcn_fmed3f(g, -128.0f, 128.0f);
  const float t = c * -1.44269504f;
  const float d = __builtin_fmaf(c, -1.44269504f, -t) + c * -1.92596299e-8f;   // log2(e) = 1.44269502 + 1.926e-8
  return __builtin_amdgcn_exp2f(t) * __builtin_fmaf(d, 0.693147181f, 1.0f);
}

// Gates below this are taken apart: 1 / (1 + exp(-g)) nears the end of float32's normal range (2^-126 at -87.3),
// where g, u and gradients that meet it may still give ordinary numbers.  (-Inf stays with the rest: -Inf * 0.)
constexpr float kGateFar = -86.0f;
__device__ __forceinline__ uint32_t gate_bits(float g) { return __float_as_uint(g); }   // the further below zero, the larger
constexpr uint32_t kGateFarBits = 0xC2AC0000u;
__device__ __forceinline__ bool gate_far(float g) { return g < kGateFar && g >= -3.4028235e38f; }

// There exp(g) = 1 / (1 + exp(-g)) to 2^-124: as f 2^e, f in [0.7, 1.5).  c is g, or -300 from there on: exp(c) is
// 2^-433, and c exp(c) times two numbers of float32 (2^256) still rounds to 0.
struct GateFar {
  float c, f;
  int e;
};
__device__ __forceinline__ GateFar gate_exp_far(float g) {
  GateFar o;
  o.c = g < -300.0f ? -300.0f : g;
  const float t = o.c * 1.44269504f;
  const float d = __builtin_fmaf(o.c, 1.44269504f, -t) + o.c * 1.92596299e-8f;
  const float n = __builtin_rintf(t);
  o.e = (int)n;
  o.f = __builtin_amdgcn_exp2f(t - n) * __builtin_fmaf(d, 0.693147181f, 1.0f);
  return o;
}
// a b c 2^e where a product of two of them may leave float32's range: mantissas and exponents apart.
__device__ __forceinline__ float product_apart(float a, float b, float c, int e) {
  const float m = (__builtin_amdgcn_frexp_mantf(a) * __builtin_amdgcn_frexp_mantf(b)) * __builtin_amdgcn_frexp_mantf(c);
  return __builtin_amdgcn_ldexpf(m, e + __builtin_amdgcn_frexp_expf(a) + __builtin_amdgcn_frexp_expf(b) + __builtin_amdgcn_frexp_expf(c));
}

// h = g / (1 + exp(-g)) u; the second form for any gate.
__device__ __forceinline__ float gate_product(float g, float u) { return (g * __builtin_amdgcn_rcpf(1.0f + gate_exp(g))) * u; }
__device__ __forceinline__ float gate_product_any(float g, float u) {
  if (!gate_far(g)) return gate_product(g, u);
  const GateFar x = gate_exp_far(g);
  return product_apart(x.c * x.f, u, 1.0f, x.e);
}
// The N by M fours of a lane in place of its g.  One look at all of them: a look at each four cost 0.5% at
// 8192 x 14336 x 4096.
template <int N, int M>
__device__ __forceinline__ void gate_products(f32x4 (&g)[N][M], const f32x4 (&u)[N][M]) {
  uint32_t low = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) low = umax(low, gate_bits(g[i][j][e]));
  if (__builtin_expect(low > kGateFarBits, 0)) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < M; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) g[i][j][e] = gate_product_any(g[i][j][e], u[i][j][e]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < M; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) g[i][j][e] = gate_product(g[i][j][e], u[i][j][e]);
  }
}
__device__ __forceinline__ f32x4 gate_product4(const f32x4& g, const f32x4& u) {
  f32x4 h[1][1] = {{g}};
  const f32x4 v[1][1] = {{u}};
  gate_products(h, v);
  return h[0][0];
}

// dg = dh u s (1 + g (1 - s)),  du = dh g s,  s = 1 / (1 + exp(-g))
__device__ __forceinline__ void gate_grad(float g, float u, float dh, float& dg, float& du) {
  const float e = gate_exp(g), s = __builtin_amdgcn_rcpf(1.0f + e);
  const float q = e < 3e38f ? e * s : 1.0f;   // 1 - s without cancellation
  const float gs = g * s;
  du = dh * gs;
  dg = (dh * u) * (s + gs * q);
}
// The same for gates far below zero, and where dh u alone passes float32.
__device__ __forceinline__ void gate_grad_far(float g, float u, float dh, float& dg, float& du) {
  if (gate_far(g)) {
    const GateFar x = gate_exp_far(g);
    du = product_apart(x.c * x.f, dh, 1.0f, x.e);
    dg = product_apart((1.0f + x.c) * x.f, dh, u, x.e);
  } else if (__builtin_isinf(dh * u)) {
    const float e = gate_exp(g), s = __builtin_amdgcn_rcpf(1.0f + e);
    dg = product_apart(s + (g * s) * (e < 3e38f ? e * s : 1.0f), dh, u, 0);
  }
}
// Eight columns of bf16.  Whether one of them needs the second look is told by the packed words: the largest 16 bits of
// g as they are (the lowest negative one, or a NaN) and the product of the largest magnitudes of u and dh.  The second
// look unpacks again: the values of the first would take 25 registers more through the kernel, and a workgroup's place on
// the CU with them.
__device__ __forceinline__ void gate_grad8(uint4 g, uint4 u, uint4 dh, float (&dg)[8], float (&du)[8]) {
  auto word = [](const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; };
  auto value = [&](const uint4& v, int e) { return e & 1 ? bf16_hi(word(v, e / 2)) : bf16_lo(word(v, e / 2)); };
  u16x2 low = {0, 0}, hu = low, hd = low;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    low = max_u16x2(low, __builtin_bit_cast(u16x2, word(g, i)));
    hu = max_u16x2(hu, abs_bits2(word(u, i)));
    hd = max_u16x2(hd, abs_bits2(word(dh, i)));
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) gate_grad(value(g, e), value(u, e), value(dh, e), dg[e], du[e]);
  const float high = __uint_as_float(hmax_u16x2(hu) << 16) * __uint_as_float(hmax_u16x2(hd) << 16);
  if (__builtin_expect(hmax_u16x2(low) > (kGateFarBits >> 16) || !(high < INFINITY), 0)) {
    asm volatile("" : "+v"(g.x), "+v"(g.y), "+v"(g.z), "+v"(g.w), "+v"(u.x), "+v"(u.y), "+v"(u.z), "+v"(u.w));
    asm volatile("" : "+v"(dh.x), "+v"(dh.y), "+v"(dh.z), "+v"(dh.w));
#pragma unroll
    for (int e = 0; e < 8; ++e) gate_grad_far(value(g, e), value(u, e), value(dh, e), dg[e], du[e]);
  }
}

}  // namespace ql
