// NVFP4 KV-cache codec for gfx950: keys and values written as E2M1 codes with an E4M3 scale
// for 16 elements and one power-of-two scale for the row, and read back to bf16.
//
// A row (token, head) has x = E2M1 * E4M3 * 2^e.  e is the smallest integer with
// amax <= 2688 * 2^e (2688 = 6 * 448, the largest product), so the E4M3 block scales
// amax_b 2^-e / 6 use their whole range, and the product (at most 2 + 4 significant bits) is
// exact in bf16: what is loaded is what attention reads, with no further rounding.  A power of
// two costs one byte a row and no precision, since E4M3 is a floating format.
//
// One lane holds 8 elements of four tokens' key rows and of the value rows beside them; the
// D / 8 lanes of a row form an aligned group inside a wave.  Both kernels are streaming copies, bound
// by the bytes: loading 65536 tokens of 8 heads of 128 takes 74 us (4.65 TB/s; a large copy moves 5.2),
// storing 16384 20 us (4.3 TB/s).  Four tokens a lane, since the value codes of four lie together and
// go as one dword: that load took 104 us with a token a lane, the store and a load of the same 53, now 38.
#include "../../include/qlinear.h"
#include "kv4_common.hpp"
#include "launch.hpp"

namespace ql {

constexpr int kKv4Threads = 256;

struct Kv4Row {
  int64_t token;
  int head;
};

__device__ __forceinline__ Kv4Row kv4_row(int64_t v, int heads, bool narrow) {
  if (narrow) {  // every row index fits in 32 bits
    const uint32_t q = (uint32_t)v / (uint32_t)heads;
    return {q, (int)((uint32_t)v - q * (uint32_t)heads)};
  }
  const int64_t t = v / heads;
  return {t, (int)(v - t * heads)};
}

__device__ __forceinline__ uint8_t* kv4_group(uint8_t* data, int64_t slot, int head, int heads, int page_shift, int gb) {
  const int64_t page = slot >> page_shift;
  const int64_t grp = (slot & ((1 << page_shift) - 1)) >> 4;
  return data + (((page * heads + head) << (page_shift - 4)) + grp) * gb;
}

__device__ __forceinline__ uint32_t kv4_amax8(uint4 x) {
  u16x2 m = abs_bits2(x.x);
  m = max_u16x2(m, abs_bits2(x.y));
  m = max_u16x2(m, abs_bits2(x.z));
  m = max_u16x2(m, abs_bits2(x.w));
  return hmax_u16x2(m);
}

// e of a row whose largest magnitude has the bf16 bits `amax` (1.3125 = 2688 / 2^11 = mantissa 40).
__device__ __forceinline__ int kv4_exponent(uint32_t amax) {
  const int e = (int)(amax >> 7) - 138 + ((amax & 127u) > 40u);
  return e < kKv4MinExp ? kKv4MinExp : (e > kKv4MaxExp ? kKv4MaxExp : e);
}

// Eight elements of a block whose largest magnitude is amax_b: the codes and the block's scale.
__device__ __forceinline__ uint32_t kv4_encode8(uint4 x, uint32_t amax_b, int e, uint32_t& scale) {
  const float want = __builtin_ldexpf(__uint_as_float(amax_b << 16), -e) / 6.0f;
  scale = e4m3_encode(want);
  const float s = e4m3_value(scale);
  const float r = s > 0.0f ? 1.0f / s : 0.0f;
  float q[8] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y),
                bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w)};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // y / s for an 8-bit y and a 4-bit s: a quotient that is no rounding border of E2M1 is at
    // least 2^-12 away from one, and the remainder step makes the ones that are exact
    const float y = __builtin_ldexpf(q[i], -e);
    const float a = y * r;
    q[i] = __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-a, s, y), r, a), y);  // -0 keeps its sign
  }
  return e2m1_pack8(q);
}

// Where chunk `part` (8 elements) of a row lies in a group: K codes of token t at k(t); V codes of the
// chunk's four pairs, a byte of token t each, at v(t >> 2) + i (D / 8) + (t & 3); its block's scale.
template <int D>
struct Kv4At {
  int part;
  __device__ __forceinline__ int k(int t) const { return t * (D / 2) + part * 4; }
  __device__ __forceinline__ int ks(int t) const { return kv4_k_scales(D) + t * (D / 16) + (part >> 1); }
  __device__ __forceinline__ int v(int quad) const {
    return kv4_v_codes(D) + quad * (2 * D) + (part & 3) * 4 * (D / 8) + (part >> 2) * 4;
  }
  __device__ __forceinline__ int vs(int quad) const {
    const int b = part >> 1;
    return kv4_v_scales(D) + quad * (D / 4) + (b & 1) * (D / 8) + (b >> 1) * 4;
  }
};

// Byte i of four dwords as one dword.
__device__ __forceinline__ uint32_t byte_of4(const uint32_t* w, int i) {
  const uint32_t sel = 0x0C0C0400u + 0x0101u * i;
  return __builtin_amdgcn_perm(w[1], w[0], sel) | __builtin_amdgcn_perm(w[3], w[2], sel) << 16;
}

// Four tokens of one head are taken together: where their slots are four in a row from a
// multiple of four (prompts, nearly always), the four bytes that V keeps side by side are written
// as one dword.  Any other four go one by one.
template <int D>
__global__ __launch_bounds__(kKv4Threads) void kv4_store_kernel(
    const uint16_t* __restrict__ k, int64_t k_stride, const uint16_t* __restrict__ v, int64_t v_stride, int64_t tokens,
    int64_t quads, int heads, const int64_t* __restrict__ slots, uint8_t* __restrict__ data, int64_t cache_slots,
    int page_shift, int32_t* status, bool narrow) {
  constexpr int kLanes = D / 8, kPer = kKv4Threads / kLanes;
  const int part = (int)(threadIdx.x & (kLanes - 1));
  const Kv4At<D> at{part};
  for (int64_t r0 = (int64_t)blockIdx.x * kPer; r0 < quads; r0 += (int64_t)gridDim.x * kPer) {
    const int64_t row = r0 + threadIdx.x / kLanes;
    const bool in = row < quads;
    const Kv4Row p = kv4_row(in ? row : quads - 1, heads, narrow);   // .token: of fours
    int64_t slot[4];
    uint4 xk[4], xv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = min(4 * p.token + i, tokens - 1);
      slot[i] = slots[t];
      xk[i] = *(const uint4*)(k + t * k_stride + p.head * D + part * 8);
      xv[i] = *(const uint4*)(v + t * v_stride + p.head * D + part * 8);
    }
    const int count = (int)min(tokens - 4 * p.token, (int64_t)4);
    bool run = count == 4 && (slot[0] & 3) == 0 && slot[0] >= 0 && slot[0] < cache_slots;
#pragma unroll
    for (int i = 1; i < 4; ++i) run = run && slot[i] == slot[0] + i;
    uint32_t ck[4], cv[4], sk[4], sv[4], ek = 0, ev = 0;
    bool bad = false, nan = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t bk = max_pair(kv4_amax8(xk[i])), bv = max_pair(kv4_amax8(xv[i]));
      uint32_t ak = bk, av = bv;
#pragma unroll
      for (int o = kLanes / 2; o >= 2; o >>= 1) {
        ak = umax(ak, (uint32_t)__shfl_xor((int)ak, o));
        av = umax(av, (uint32_t)__shfl_xor((int)av, o));
      }
      int e = kv4_exponent(ak), f = kv4_exponent(av);
      ck[i] = kv4_encode8(xk[i], bk, e, sk[i]);
      cv[i] = kv4_encode8(xv[i], bv, f, sv[i]);
      if (umax(ak, av) >= kBf16InfBits) {  // a token with Inf or NaN is a NaN token, marked in its key scales
        ck[i] = cv[i] = 0;
        sk[i] = 0xFF;
        sv[i] = 0;
        e = f = 0;
        nan = nan || (i < count && slot[i] >= 0 && slot[i] < cache_slots);
      }
      ek |= (uint32_t)(e + 127) << (8 * i);
      ev |= (uint32_t)(f + 127) << (8 * i);
    }
    if (!in) continue;
    if (run) {
      uint8_t* g = kv4_group(data, slot[0], p.head, heads, page_shift, kv4_group_bytes(D));
      const int t = (int)(slot[0] & 15), quad = t >> 2;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        *(uint32_t*)(g + at.k(t + i)) = ck[i];
        *(uint32_t*)(g + at.v(quad) + i * (D / 8)) = byte_of4(cv, i);
      }
      if ((part & 1) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) g[at.ks(t + i)] = (uint8_t)sk[i];
        *(uint32_t*)(g + at.vs(quad)) = sv[0] | sv[1] << 8 | sv[2] << 16 | sv[3] << 24;
      }
      if (part == 0) {
        *(uint32_t*)(g + kv4_k_exps(D) + t) = ek;
        *(uint32_t*)(g + kv4_v_exps(D) + t) = ev;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= count) break;
        if (slot[i] < 0 || slot[i] >= cache_slots) {
          bad = true;
          continue;
        }
        uint8_t* g = kv4_group(data, slot[i], p.head, heads, page_shift, kv4_group_bytes(D));
        const int t = (int)(slot[i] & 15), quad = t >> 2;
        *(uint32_t*)(g + at.k(t)) = ck[i];
#pragma unroll
        for (int y = 0; y < 4; ++y) g[at.v(quad) + y * (D / 8) + (t & 3)] = (uint8_t)(cv[i] >> (8 * y));
        if ((part & 1) == 0) {
          g[at.ks(t)] = (uint8_t)sk[i];
          g[at.vs(quad) + (t & 3)] = (uint8_t)sv[i];
        }
        if (part == 0) {
          g[kv4_k_exps(D) + t] = (uint8_t)(ek >> (8 * i));
          g[kv4_v_exps(D) + t] = (uint8_t)(ev >> (8 * i));
        }
      }
    }
    if (part == 0 && status && (bad || nan))
      atomicOr(status, (bad ? (int32_t)kStatusBadItem : 0) | (nan ? (int32_t)kStatusNonFinite : 0));
  }
}

// Eight codes times their scale as bf16 (exact; Inf where 2112 * 2^117 passes the format).
__device__ __forceinline__ uint4 kv4_decode8(uint32_t codes, uint32_t scale, uint32_t exp) {
  const float s = __builtin_ldexpf(e4m3_value(scale), (int)exp - 127);
  const f32x2 a = e2m1_unpack2<0>(codes), b = e2m1_unpack2<1>(codes), c = e2m1_unpack2<2>(codes),
              d = e2m1_unpack2<3>(codes);
  return make_uint4(pack_bf16x2_rne(a[0] * s, a[1] * s), pack_bf16x2_rne(b[0] * s, b[1] * s),
                    pack_bf16x2_rne(c[0] * s, c[1] * s), pack_bf16x2_rne(d[0] * s, d[1] * s));
}

template <int D>
__global__ __launch_bounds__(kKv4Threads) void kv4_load_kernel(
    const uint8_t* __restrict__ data, int64_t cache_slots, int page_shift, const int64_t* __restrict__ slots,
    int64_t tokens, int64_t quads, int heads, uint16_t* __restrict__ k, int64_t k_stride, uint16_t* __restrict__ v,
    int64_t v_stride, int32_t* status, bool narrow) {
  constexpr int kLanes = D / 8, kPer = kKv4Threads / kLanes;
  const int part = (int)(threadIdx.x & (kLanes - 1));
  const Kv4At<D> at{part};
  for (int64_t r0 = (int64_t)blockIdx.x * kPer; r0 < quads; r0 += (int64_t)gridDim.x * kPer) {
    const int64_t row = r0 + threadIdx.x / kLanes;
    if (row >= quads) continue;
    const Kv4Row p = kv4_row(row, heads, narrow);
    int64_t slot[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) slot[i] = slots[min(4 * p.token + i, tokens - 1)];
    const int count = (int)min(tokens - 4 * p.token, (int64_t)4);
    bool run = count == 4 && (slot[0] & 3) == 0 && slot[0] >= 0 && slot[0] < cache_slots, bad = false;
#pragma unroll
    for (int i = 1; i < 4; ++i) run = run && slot[i] == slot[0] + i;
    uint32_t ck[4], cv[4], sk[4], sv[4], mark[4], ek = 0, ev = 0;
    if (run) {
      const uint8_t* g = kv4_group((uint8_t*)data, slot[0], p.head, heads, page_shift, kv4_group_bytes(D));
      const int t = (int)(slot[0] & 15), quad = t >> 2;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ck[i] = *(const uint32_t*)(g + at.k(t + i));
        sk[i] = g[at.ks(t + i)];
        mark[i] = g[kv4_k_scales(D) + (t + i) * (D / 16)];
        w[i] = *(const uint32_t*)(g + at.v(quad) + i * (D / 8));
      }
      const uint32_t s4 = *(const uint32_t*)(g + at.vs(quad));
      ek = *(const uint32_t*)(g + kv4_k_exps(D) + t);
      ev = *(const uint32_t*)(g + kv4_v_exps(D) + t);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cv[i] = byte_of4(w, i);
        sv[i] = (s4 >> (8 * i)) & 0xFFu;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool ok = slot[i] >= 0 && slot[i] < cache_slots;
        bad = bad || (i < count && !ok);
        // a slot outside the cache is read from slot 0 and dropped
        const uint8_t* g = kv4_group((uint8_t*)data, ok ? slot[i] : 0, p.head, heads, page_shift, kv4_group_bytes(D));
        const int t = ok ? (int)(slot[i] & 15) : 0, quad = t >> 2;
        ck[i] = ok ? *(const uint32_t*)(g + at.k(t)) : 0u;
        cv[i] = 0;
#pragma unroll
        for (int y = 0; y < 4; ++y) cv[i] |= (uint32_t)g[at.v(quad) + y * (D / 8) + (t & 3)] << (8 * y);
        cv[i] = ok ? cv[i] : 0u;
        sk[i] = ok ? g[at.ks(t)] : 0u;
        sv[i] = ok ? g[at.vs(quad) + (t & 3)] : 0u;
        mark[i] = ok ? g[kv4_k_scales(D) + t * (D / 16)] : 0u;
        ek |= (uint32_t)g[kv4_k_exps(D) + t] << (8 * i);
        ev |= (uint32_t)g[kv4_v_exps(D) + t] << (8 * i);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= count) break;
      const int64_t t = 4 * p.token + i;
      if (k) *(uint4*)(k + t * k_stride + p.head * D + part * 8) = kv4_decode8(ck[i], sk[i], (ek >> (8 * i)) & 0xFFu);
      if (v)
        *(uint4*)(v + t * v_stride + p.head * D + part * 8) =
            kv4_decode8(cv[i], mark[i] == 0xFF ? 0xFFu : sv[i], (ev >> (8 * i)) & 0xFFu);
    }
    if (part == 0 && status && bad) atomicOr(status, (int32_t)kStatusBadItem);
  }
}

static unsigned kv4_grid(int64_t quads, int d) {
  const int64_t per = kKv4Threads / (d / 8);
  const int64_t blocks = (quads + per - 1) / per;
  return (unsigned)(blocks < 8192 ? blocks : 8192);
}

template <int D>
static hipError_t store_d(const Kv4Cache& c, const uint16_t* k, int64_t ks, const uint16_t* v, int64_t vs,
                          int64_t tokens, const int64_t* slots, int32_t* status, hipStream_t s) {
  const int64_t quads = (tokens + 3) / 4 * c.heads;
  kv4_store_kernel<D><<<kv4_grid(quads, D), kKv4Threads, 0, s>>>(k, ks, v, vs, tokens, quads, c.heads, slots, c.data,
                                                                c.pages << c.page_shift, c.page_shift, status,
                                                                quads <= (int64_t)UINT32_MAX);
  return hipGetLastError();
}

template <int D>
static hipError_t load_d(const Kv4Cache& c, const int64_t* slots, int64_t tokens, uint16_t* k, int64_t ks, uint16_t* v,
                         int64_t vs, int32_t* status, hipStream_t s) {
  const int64_t quads = (tokens + 3) / 4 * c.heads;
  kv4_load_kernel<D><<<kv4_grid(quads, D), kKv4Threads, 0, s>>>(c.data, c.pages << c.page_shift, c.page_shift, slots,
                                                               tokens, quads, c.heads, k, ks, v, vs, status,
                                                               quads <= (int64_t)UINT32_MAX);
  return hipGetLastError();
}

hipError_t launch_kv4_store(const Kv4Cache& c, const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                            int64_t tokens, const int64_t* slots, int32_t* status, hipStream_t s) {
  if (c.head_dim == 64) return store_d<64>(c, k, k_stride, v, v_stride, tokens, slots, status, s);
  if (c.head_dim == 128) return store_d<128>(c, k, k_stride, v, v_stride, tokens, slots, status, s);
  return store_d<256>(c, k, k_stride, v, v_stride, tokens, slots, status, s);
}

hipError_t launch_kv4_load(const Kv4Cache& c, const int64_t* slots, int64_t tokens, uint16_t* k, int64_t k_stride,
                           uint16_t* v, int64_t v_stride, int32_t* status, hipStream_t s) {
  if (c.head_dim == 64) return load_d<64>(c, slots, tokens, k, k_stride, v, v_stride, status, s);
  if (c.head_dim == 128) return load_d<128>(c, slots, tokens, k, k_stride, v, v_stride, status, s);
  return load_d<256>(c, slots, tokens, k, k_stride, v, v_stride, status, s);
}

}  // namespace ql
