// Root-mean-square norm with the residual's addition, and its backward pass, on gfx950.
//
//   h = bf16(x + r)            the residual stream, held in bf16; the norm is the norm of what is held
//   y = h s w,  s = 1 / sqrt(mean(h^2) + eps)
//   y in bf16 and/or as E4M3 codes with a scale for 128 columns (fp8_out.hpp), from float32 values
//
// Bound by memory: a row is read once, kept in registers, and everything is written from there.
// T threads take a row, NV units of 8 elements (16 bytes) each, unit i T + t: 16 neighbouring lanes
// hold a segment of 128, so its maximum is four DPP steps.  A workgroup goes through rows with the
// weight's elements in registers.  Measured: 8192 x 4096 with the residual and all outputs 57 us (302 MB at 5.3
// TB/s), 1777 x 3584 to 8 bits 6.6 us, one row of 4096 3.2 us; backward 16384 x 5120 127 us (671 MB at 5.3 TB/s).
// That holds up to 16384 columns (16384: forward 5.3, backward 5.0 TB/s).  Behind, 1024 threads with 128 registers each
// do not hold a row's share of everything, and the rest goes through scratch memory: the backward, which has h, dy, dh, w
// and dw, spills 91 registers up to 32768 columns (20480: 1.5 TB/s, 32768: 1.8) and 394 up to 65536 (0.6 to 0.8 TB/s), the
// forward 25 to 48 beyond 32768 (40960: 4.4 TB/s to bf16, 2.9 to 8 bits; 65536: 4.6 and 3.4).
#include <type_traits>

#include "common.hpp"
#include "fp8_out.hpp"
#include "launch.hpp"

namespace ql {

namespace {

constexpr int kNormThreads = 256;

template <int T>
constexpr int norm_block() { return T > kNormThreads ? T : kNormThreads; }

__device__ __forceinline__ float bf16_at(const uint4& v, int e) {
  const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
  return e & 1 ? bf16_hi(w) : bf16_lo(w);
}
__device__ __forceinline__ uint4 bf16_pack8(const float* f) {
  return make_uint4(pack_bf16x2_rne(f[0], f[1]), pack_bf16x2_rne(f[2], f[3]), pack_bf16x2_rne(f[4], f[5]),
                    pack_bf16x2_rne(f[6], f[7]));
}

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) { return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v))); }
// Sum over the wave in a fixed order, the same bits in every lane.
__device__ __forceinline__ float sum_wave(float v) {
  v += dpp_f32<0xB1>(v);
  v += dpp_f32<0x4E>(v);
  v += dpp_f32<0x141>(v);
  v += dpp_f32<0x140>(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// Sums over the T threads of a row.  Two sets of LDS words in turn: a set is written again only after
// the barrier of the sum between, which every wave reaches after reading it.  MOST is the largest N of a
// kernel's sums: sets of sums of any N then lie in the same two places, which the turns rely on.
template <int T, int MOST, int N>
__device__ __forceinline__ void sum_row(float (&v)[N], float* red, int& turn) {
  static_assert(N <= MOST, "a set holds MOST sums");
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = sum_wave(v[n]);
  if (T > kWave) {
    constexpr int W = T / kWave;
    float* p = red + turn * (MOST * W);
    turn ^= 1;
    if ((threadIdx.x & (kWave - 1)) == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) p[n * W + threadIdx.x / kWave] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float s = p[n * W];
#pragma unroll
      for (int w = 1; w < W; ++w) s += p[n * W + w];
      v[n] = s;
    }
  }
}

// The factor that brings a row's squares into float32's range, by v = mean(h^2) + eps as it came out: squares pass the
// range where an element passes 2^63, and lose bits below it where v is (an eps below 2^-90, and elements like it).
__device__ __forceinline__ float row_scale(float v) { return v == INFINITY ? 0x1p-80f : v < 0x1p-90f ? 0x1p70f : 1.0f; }
// s / scale of a row from its elements times scale (eps is lost beside large ones).
template <int T, int MOST, int NV>
__device__ __forceinline__ float row_rstd_scaled(const uint4 (&h)[NV], float k, float eps, float scale, float* red, int& turn) {
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float f = bf16_at(h[i], e) * scale;
      s[0] += f * f;
    }
  sum_row<T, MOST>(s, red, turn);
  return 1.0f / sqrtf(s[0] / k + (eps * scale) * scale);
}

template <int T, int NV, int FMT>
__global__ __launch_bounds__(norm_block<T>()) void rms_norm_kernel(Norm a) {
  constexpr int ROWS = norm_block<T>() / T;
  __shared__ float red[2 * (T > kWave ? T / kWave : 1)];
  const int t = ROWS > 1 ? threadIdx.x % T : threadIdx.x;
  const int64_t units = a.k / 8;
  const float k = (float)a.k;
  int turn = 0;
  uint4 w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t u = (int64_t)i * T + t;
    w[i] = u < units ? *(const uint4*)(a.w + u * 8) : make_uint4(0, 0, 0, 0);
  }
  // every wave of a workgroup of several rows works alone, so a row past the end just leaves
  for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / T; row < a.m; row += (int64_t)gridDim.x * ROWS) {
    uint4 h[NV], r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t u = (int64_t)i * T + t;
      h[i] = u < units ? *(const uint4*)(a.x + row * a.x_stride + u * 8) : make_uint4(0, 0, 0, 0);
    }
    if (a.r) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t u = (int64_t)i * T + t;
        r[i] = u < units ? *(const uint4*)(a.r + row * a.r_stride + u * 8) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = bf16_at(h[i], e) + bf16_at(r[i], e);
        h[i] = bf16_pack8(f);
      }
    }
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = bf16_at(h[i], e);
        ss[0] += f * f;
      }
    if (a.h) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t u = (int64_t)i * T + t;
        if (u < units) *(uint4*)(a.h + row * a.h_stride + u * 8) = h[i];
      }
    }
    sum_row<T, 1>(ss, red, turn);
    const float v = ss[0] / k + a.eps, scale = row_scale(v);
    float s = 1.0f / sqrtf(v);
    if (__builtin_expect(scale != 1.0f, 0)) s = row_rstd_scaled<T, 1>(h, k, a.eps, scale, red, turn) * scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t u = (int64_t)i * T + t;
      float f[8];
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[e] = (bf16_at(h[i], e) * s) * bf16_at(w[i], e);
        if (FMT) top = umax(top, abs_bits(f[e]));
      }
      if (a.y && u < units) *(uint4*)(a.y + row * a.k + u * 8) = bf16_pack8(f);
      if (FMT) {
        const Fp8Seg sc = fp8_seg_scale<FMT == 2>(max_row16(top));
        if (u < units) {
          *(uint2*)(a.yq + row * a.k + u * 8) = make_uint2(fp8_encode4(f, sc), fp8_encode4(f + 4, sc));
          if ((t & 15) == 0) {
            const int64_t seg = row * (a.k / 128) + u / 16;
            if (FMT == 2)
              ((uint8_t*)a.sy)[seg] = (uint8_t)sc.stored;
            else
              ((uint32_t*)a.sy)[seg] = sc.stored;
          }
        }
      }
    }
  }
}

// Backward: with a = dy w and c = mean(a h),
//   dx = dh + s (a - h s^2 c),   dw = sum over rows of dy (h s).
// A workgroup keeps its rows' share of dw in registers and leaves it as one row of `part`
// ([gridDim.x][k] float32); rms_norm_dw_kernel adds those in a fixed order.
template <int T, int NV>
__global__ __launch_bounds__(norm_block<T>()) void rms_norm_backward_kernel(NormBackward a) {
  constexpr int ROWS = norm_block<T>() / T;
  __shared__ float red[4 * (T > kWave ? T / kWave : 1)];
  __shared__ float join[ROWS > 1 ? (ROWS - 1) * T * 8 : 1];
  const int t = ROWS > 1 ? threadIdx.x % T : threadIdx.x;
  const int64_t units = a.k / 8;
  const float k = (float)a.k;
  int turn = 0;
  uint4 w[NV];
  float dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t u = (int64_t)i * T + t;
    w[i] = u < units ? *(const uint4*)(a.w + u * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
  }
  for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / T; row < a.m; row += (int64_t)gridDim.x * ROWS) {
    uint4 h[NV], dy[NV], dh[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t u = (int64_t)i * T + t;
      h[i] = u < units ? *(const uint4*)(a.h + row * a.h_stride + u * 8) : make_uint4(0, 0, 0, 0);
      dy[i] = u < units ? *(const uint4*)(a.dy + row * a.dy_stride + u * 8) : make_uint4(0, 0, 0, 0);
    }
    if (a.dh) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t u = (int64_t)i * T + t;
        dh[i] = u < units ? *(const uint4*)(a.dh + row * a.dh_stride + u * 8) : make_uint4(0, 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) dh[i] = make_uint4(0, 0, 0, 0);
    }
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = bf16_at(h[i], e);
        sum[0] += f * f;
        sum[1] += (bf16_at(dy[i], e) * bf16_at(w[i], e)) * f;
      }
    sum_row<T, 2>(sum, red, turn);
    const float v = sum[0] / k + a.eps, scale = row_scale(v);
    float s = 1.0f / sqrtf(v);
    float sc = (s * (sum[1] / k)) * s;   // s^2 c without a square of its own, which may leave the range
    const bool finite = __builtin_fabsf(sum[1]) < INFINITY;
    if (__builtin_expect(scale != 1.0f || !finite, 0)) {   // a sum left the range: both again of scaled factors
      const float rs = row_rstd_scaled<T, 2>(h, k, a.eps, scale, red, turn);
      const float down = finite ? 1.0f : 0x1p-100f, up = finite ? 1.0f : 0x1p100f;
      float c[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          c[0] += ((bf16_at(dy[i], e) * down) * bf16_at(w[i], e)) * (bf16_at(h[i], e) * scale);
      sum_row<T, 2>(c, red, turn);
      s = rs * scale;
      sc = ((rs * (c[0] / k)) * up) * s;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t u = (int64_t)i * T + t;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float hv = bf16_at(h[i], e), dv = bf16_at(dy[i], e);
        f[e] = bf16_at(dh[i], e) + s * (dv * bf16_at(w[i], e) - hv * sc);
        dw[i][e] += dv * (hv * s);
      }
      if (u < units) *(uint4*)(a.dx + row * a.dx_stride + u * 8) = bf16_pack8(f);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t u = (int64_t)i * T + t;
    if (ROWS > 1) {  // the waves' sums, in their order
      const int me = threadIdx.x / T;
      __syncthreads();
      if (me > 0)
#pragma unroll
        for (int e = 0; e < 8; ++e) join[((me - 1) * 8 + e) * T + t] = dw[i][e];
      __syncthreads();
      if (me > 0) continue;
#pragma unroll
      for (int q = 0; q + 1 < ROWS; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] += join[(q * 8 + e) * T + t];
    }
    if (u < units) {
      float* p = a.part + (int64_t)blockIdx.x * a.k + u * 8;
      *(f32x4*)p = f32x4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
      *(f32x4*)(p + 4) = f32x4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
    }
  }
}

// dw[c] = sum over p of part[p][c]: 32 columns a workgroup, 8 lanes of 4 columns by 32 rows, four of them under way.
__global__ __launch_bounds__(256) void rms_norm_dw_kernel(const float* __restrict__ part, int parts, int64_t k,
                                                          float* __restrict__ dw) {
  __shared__ f32x4 red[4][8];
  const int lane = threadIdx.x & 7, slot = threadIdx.x >> 3, wave = threadIdx.x / kWave;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane * 4;
  const f32x4 zero = {0, 0, 0, 0};
  f32x4 s[4] = {zero, zero, zero, zero};
  if (c < k)
    for (int p = slot; p < parts; p += 128) {
      f32x4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = p + 32 * i < parts ? *(const f32x4*)(part + (p + 32 * i) * k + c) : zero;
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += v[i];
    }
  f32x4 t = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
  for (int e = 0; e < 4; ++e) {   // the wave's eight rows
    t[e] += __shfl_xor(t[e], 8);
    t[e] += __shfl_xor(t[e], 16);
    t[e] += __shfl_xor(t[e], 32);
  }
  if ((threadIdx.x & (kWave - 1)) < 8) red[wave][lane] = t;
  __syncthreads();
  if (slot == 0 && c < k) *(f32x4*)(dw + c) = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
}

// Threads of a row, (T, NV) for up to 8 T NV elements: as many as keep a row's units few, or a wave alone, which has no
// barrier.  Alone: the forward up to 1024 elements if there are more than 1024 rows (8192 x 1024 12.1 us against 15.0
// with a workgroup a row, 256 x 1024 3.7 against 3.3, 8192 x 2048 23.0 against 20.0); the backward, whose workgroup
// then joins four rows' shares of dw, up to 2048 (256 x 1024 6.2 against 8.0, 32768 x 1024 39 against 71, 32768 x 2048
// 83 against 101).
template <typename F>
hipError_t norm_dispatch(int64_t m, int64_t k, F&& f) {
  const int64_t units = k / 8;
  if (units <= 64) return f.template run<64, 1>();
  if constexpr (std::remove_reference_t<F>::kBackward) {
    if (units <= 128) return f.template run<64, 2>();
    if (units <= 256) return f.template run<64, 4>();
  } else {
    if (m > 1024 && units <= 128) return f.template run<64, 2>();
    if (units <= 256) return f.template run<256, 1>();
  }
  if (units <= 512) return f.template run<256, 2>();
  if (units <= 768) return f.template run<256, 3>();
  if (units <= 1024) return f.template run<256, 4>();
  if (units <= 2048) return f.template run<1024, 2>();
  if (units <= 4096) return f.template run<1024, 4>();
  return f.template run<1024, 8>();
}

constexpr int64_t kNormGrid = 2048;          // workgroups of 256 threads that fill the chip

template <int T>
unsigned norm_grid(int64_t m, int64_t most) {
  const int64_t rows = norm_block<T>() / T, g = (m + rows - 1) / rows;
  return (unsigned)(g < most ? g : most);
}

struct RunNorm {
  static constexpr bool kBackward = false;
  const Norm& a;
  int fmt;
  hipStream_t s;
  template <int T, int NV>
  hipError_t run() {
    const unsigned grid = norm_grid<T>(a.m, kNormGrid * kNormThreads / norm_block<T>());
    constexpr int block = norm_block<T>();
    if (fmt == 0) rms_norm_kernel<T, NV, 0><<<grid, block, 0, s>>>(a);
    else if (fmt == 1) rms_norm_kernel<T, NV, 1><<<grid, block, 0, s>>>(a);
    else rms_norm_kernel<T, NV, 2><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
  }
};

// Rows of dw's partial sums: few enough that adding them is short beside the pass over the rows, which one workgroup
// a CU makes alone up to 1024 rows (700 x 4096: 256 parts 10.6 us, 512 12.3; 2048 x 4096: 17.9, 16.4; 16384 x 5120: 124,
// 97.5, 1024 parts 113).
int64_t norm_parts(int64_t m) { return m <= 1024 ? 256 : 512; }

struct RunNormBackward {
  static constexpr bool kBackward = true;
  const NormBackward& a;
  hipStream_t s;
  template <int T, int NV>
  hipError_t run() {
    const unsigned grid = norm_grid<T>(a.m, norm_parts(a.m));
    rms_norm_backward_kernel<T, NV><<<grid, norm_block<T>(), 0, s>>>(a);
    if (a.dw)
      rms_norm_dw_kernel<<<(unsigned)((a.k + 31) / 32), 256, 0, s>>>(a.part, (int)grid, a.k, a.dw);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_rms_norm(const Norm& a, int fmt, hipStream_t s) {
  if (a.m <= 0 || a.k <= 0 || a.k % 8 != 0 || a.k > kNormMaxK) return hipErrorInvalidValue;
  return norm_dispatch(a.m, a.k, RunNorm{a, fmt, s});
}

size_t rms_norm_backward_bytes(int64_t m, int64_t k) {
  return (size_t)(m < norm_parts(m) ? m : norm_parts(m)) * (size_t)k * 4;
}

hipError_t launch_rms_norm_backward(const NormBackward& a, hipStream_t s) {
  if (a.m <= 0 || a.k <= 0 || a.k % 8 != 0 || a.k > kNormMaxK) return hipErrorInvalidValue;
  return norm_dispatch(a.m, a.k, RunNormBackward{a, s});
}

}  // namespace ql
