// Host-side launchers of the gfx950 kernels (internal to libqlinear; the C ABI in
// api.cpp validates arguments before calling any of these).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/qlinear.h"

namespace ql {

// hipGetLastError reports the last failure of any HIP call on the thread, not only of the
// launches just made: every entry point clears it before its first launch, so a launch
// status reflects this library's launches alone.
inline void clear_hip_error() { (void)hipGetLastError(); }

// qlinear_forward's checks and dispatch (api.cpp), shared with the allocation-free variant.
qlinear_status forward_impl(const qlinear_qweight* w, const uint16_t* x, int64_t m,
                            const uint16_t* lora_a, const uint16_t* lora_b, int32_t rank,
                            float lora_scale, void* y, int32_t out_dtype, void* ws, size_t ws_bytes,
                            void* stream);

// ---- forward workspace layout, shared by every path
// [0, kWsReserved): the status word (int32 at offset 0) and, from kWsCounterOff on, the
// integer counters and flags through which the workgroups of one launch coordinate.  They
// must be zero before the first call and every call returns the ones it used to zero, so
// calls of any shape may share one workspace.  No path ever uses this region as scratch.
// [kWsReserved, ...): per-call scratch, always written before it is read within a call.
constexpr size_t kWsReserved = 128 * 1024;
constexpr size_t kWsCounterOff = 256;
constexpr uint32_t kStatusNonFinite = 1u;  // a weight input held Inf or NaN
constexpr uint32_t kStatusTimeout = 2u;    // a bounded wait for another workgroup gave up
constexpr uint32_t kStatusBadItem = 4u;    // a requantization item failed its checks
inline int32_t* ws_status(void* ws) { return (int32_t*)ws; }
inline uint32_t* ws_counters(void* ws) { return (uint32_t*)((char*)ws + kWsCounterOff); }
inline char* ws_scratch(void* ws) { return (char*)ws + kWsReserved; }

// ---- quantizers (quant.hip)
constexpr int kAmaxParts = 1024;  // partial maxima written by the NVFP4 amax pass
hipError_t launch_nvfp4_quantize(const uint16_t* w, int64_t n, int64_t k, uint8_t* codes,
                                 uint8_t* scales, float* tensor_scale, int32_t* status,
                                 uint32_t* partials, hipStream_t s);
// FP8 scales: float32 amax/448, or with pow2 the E8M0 byte of the power-of-two scale.
hipError_t launch_fp8_weight_quantize(const uint16_t* w, int64_t n, int64_t k, uint8_t* codes,
                                      void* scales, bool pow2, int32_t* status, hipStream_t s);
hipError_t launch_fp8_act_quantize(const uint16_t* x, int64_t m, int64_t k, uint8_t* xq,
                                   void* sx, bool pow2, hipStream_t s);

// ---- whole-policy requantization (quant.hip)
// Workspace: status word | header | descriptors[count] | per-tensor maxima[count].  The
// descriptors are rebuilt on the device from the caller's item array by every call.  With
// deltas (a device array of count update pointers) each weight is first updated in place.
size_t requant_workspace(int32_t count);
hipError_t launch_requant(const void* items, const uint16_t* const* deltas, int32_t count,
                          int32_t format, void* ws, hipStream_t s);

// ---- FP8 KV-cache codec (kv.hip); head_dim a power of two in [16, 512]
hipError_t launch_kv_store(const uint16_t* kv, int64_t tokens, int heads, int head_dim, const int64_t* slots,
                           uint8_t* codes, float* scales, int64_t cache_slots, int32_t* status, hipStream_t s);
hipError_t launch_kv_load(const uint8_t* codes, const float* scales, int64_t cache_slots, const int64_t* slots,
                          int64_t tokens, int heads, int head_dim, uint16_t* out, int32_t* status, hipStream_t s);

// ---- NVFP4 KV cache: codec (kv4.hip) and attention (attn4.hip); head_dim 64, 128 or 256
struct Kv4Cache {
  uint8_t* data;
  int64_t pages;
  int page_shift;  // log2 of the page size (16 tokens or more)
  int heads;
  int head_dim;
};
hipError_t launch_kv4_store(const Kv4Cache& c, const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                            int64_t tokens, const int64_t* slots, int32_t* status, hipStream_t s);
hipError_t launch_kv4_load(const Kv4Cache& c, const int64_t* slots, int64_t tokens, uint16_t* k, int64_t k_stride,
                           uint16_t* v, int64_t v_stride, int32_t* status, hipStream_t s);
struct Attn4 {
  const uint8_t* data;
  int64_t pages;
  int page_shift, heads;
  const uint16_t* q;
  int64_t q_stride;
  int q_heads, group;       // group = q_heads / heads query heads share a KV head
  int batch, max_q;
  int64_t total_q;
  const int32_t* q_starts;  // null: max_q query tokens in every sequence
  const int32_t* kv_lens;
  const int32_t* table;
  int64_t table_stride, table_pages;
  float scale_log2e;
  int causal, window;
  uint16_t* out;
  int64_t out_stride;
  float* lse;               // may be null
  int32_t* status;
  uint32_t* counters;       // zero before and after a call
  uint8_t* parts;           // attn4_scratch_bytes
  // set by the launcher
  int few;                  // most query rows of a sequence for the few-row kernel
  int join;                 // a second kernel joins the parts of its units
  int wide;                 // positions in the call's work may pass 32 bits
  int most_units;           // of the prompt kernel
  int parts_each;           // most parts of a unit of the prompt kernel
};
bool attn4_launchable(int64_t batch, int64_t total_q, int64_t group, int64_t heads, int head_dim, int64_t max_q);
size_t attn4_scratch_bytes(int64_t batch, int64_t total_q, int64_t group, int64_t heads, int head_dim, int64_t max_q);
hipError_t launch_attn4(const Attn4& a, int head_dim, hipStream_t s);

// ---- backward of the NVFP4 + LoRA layer (backward.hip); n % 64 == 0, k % 128 == 0
size_t backward_scratch_bytes(int64_t m, int64_t n, int64_t k, int32_t rank);
hipError_t launch_backward_nvfp4(const uint16_t* x, const uint16_t* dy, int64_t m, int64_t n, int64_t k,
                                 const uint8_t* codes, const uint8_t* scales, const float* tensor_scale,
                                 const uint16_t* lora_a, const uint16_t* lora_b, int32_t rank, float lora_scale,
                                 void* dx, int out_f32, float* da, float* db, void* scratch, hipStream_t s);

// ---- NVFP4 layer for up to 64 tokens (gemv16.hip)
struct G16Plan {
  int mt;             // m tiles of 16 (1, 2 or 4)
  int rt;             // row tiles of 16 per workgroup (1 or 2)
  int64_t tiles_w;    // weight tiles of 16 * rt rows (64 rows for 33..64 tokens)
  int64_t kchunks;    // 256-wide K chunks
  int64_t tiles_l;    // LoRA row tiles of 16
  int64_t lgroups;    // LoRA chunk groups
  int lc;             // chunks per LoRA item
  int rank_pad;
  int64_t cps;        // chunks per K split
  int splits;
  int64_t n_pad;
  int xstride;        // LDS row stride of the staged activations
  int64_t kst = 0;    // 128-wide K stages of the 33..64-token stage path (0: not used)
  int64_t sps = 0;    // stages per K split on that path
  int64_t full = 0;   // that path: tiles [0, full) whole, the others split `splits` ways
  size_t lds_bytes;
  int ctr_stride = 0; // words between two counters in the reserved region (0: does not fit)
};
G16Plan plan_g16(int64_t m, int64_t n, int64_t k, int32_t rank);
// false if the launch cannot run this shape (counters do not fit the reserved region,
// partial offsets beyond 32 bits): the C ABI reports QL_ERR_SHAPE before launching.
bool g16_plan_ok(const G16Plan& p, int64_t m);
size_t g16_workspace(const G16Plan& p, int64_t m);  // scratch bytes after the reserved region
hipError_t launch_g16(const G16Plan& p, const uint16_t* x, int64_t m, int64_t n, int64_t k,
                      const uint8_t* codes, const uint8_t* scales, const float* tensor_scale,
                      const uint16_t* lora_a, const uint16_t* lora_b, int32_t rank,
                      float lora_scale, void* y, int out_f32, void* ws, hipStream_t s);

// ---- LoRA down-projection for the GEMM paths (gemm_nvfp4.hip)
// t = bf16(s x A^T) as [m][rank_pad] (zero past the rank) in `scratch`; two kernels (split-K
// partials, then their fixed-order sum), no inter-workgroup counters.  k % 16 == 0.
size_t lora_down_bytes(int64_t m, int64_t k, int32_t rank);
// The same product s . x . A^T kept in higher precision: bf16 [m][2 rank_pad], row = the
// rounded value hi (columns [0, rank_pad)) and the rounded remainder lo (columns [rank_pad,
// 2 rank_pad)).
size_t lora_down_hilo_bytes(int64_t m, int64_t k, int32_t rank);
hipError_t launch_lora_down_hilo(const uint16_t* x, int64_t m, int64_t k, const uint16_t* lora_a,
                                 int32_t rank, float lora_scale, void* scratch, uint16_t** t_hl_out,
                                 hipStream_t s);
hipError_t launch_lora_down(const uint16_t* x, int64_t m, int64_t k, const uint16_t* lora_a,
                            int32_t rank, float lora_scale, void* scratch, uint16_t** t_out,
                            hipStream_t s);

// ---- large-M GEMMs (gemm_nvfp4.hip, gemm_fp8.hip)
// Generic K (k % 16 == 0): t = bf16(s x A^T) computed beforehand, or null.
hipError_t launch_gemm_nvfp4(const uint16_t* x, int64_t m, int64_t n, int64_t k,
                             const uint8_t* codes, const uint8_t* scales, const float* tensor_scale,
                             const uint16_t* t, const uint16_t* lora_b, int32_t rank, void* y,
                             int out_f32, hipStream_t s);
// k % 64 == 0 and k < kNvF16MaxK: f16 activations, row factors and the LoRA intermediate
// are formed in `scratch` (gemm_nvfp4_f16_workspace bytes) by a pre-pass.
constexpr int64_t kNvF16MaxK = int64_t(1) << 22;
hipError_t launch_gemm_nvfp4_f16(const uint16_t* x, int64_t m, int64_t n, int64_t k,
                                 const uint8_t* codes, const uint8_t* scales,
                                 const float* tensor_scale, const uint16_t* lora_a,
                                 const uint16_t* lora_b, int32_t rank, float lora_scale, void* y,
                                 int out_f32, void* scratch, hipStream_t s);
size_t gemm_nvfp4_f16_workspace(int64_t m, int64_t n, int64_t k, int32_t rank);
// Up to kNvMaxSeg layers that read the same x (a fused projection) as one pre-pass and one
// GEMM over all their n tiles (each layer's n rounded up to whole 256-row tiles); the
// adapters (all of rank `rank`, a multiple of 32 for more than one layer, nl * rank <= 128)
// are stacked for the pre-pass.  nl == 1 is launch_gemm_nvfp4_f16.
constexpr int kNvMaxSeg = 4;
struct NvLayer {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* tensor_scale;
  const uint16_t* lora_a;
  const uint16_t* lora_b;
  void* y;
  int64_t n;
};
size_t gemm_nvfp4_f16_layers_workspace(int64_t m, int64_t k, const int64_t* n, int nl, int32_t rank);
hipError_t launch_gemm_nvfp4_f16_layers(const uint16_t* x, int64_t m, int64_t k, const NvLayer* layers, int nl,
                                        int32_t rank, float lora_scale, int out_f32, void* scratch, hipStream_t s);
// x as f16 rows scaled by powers of two (x16 [m][k], rs [m]: x[r] = rs[r] x16[r], exact but
// for values below about 2^-29 of the row maximum) and, with rank > 0, t = s x A^T as hi | lo
// bf16 pairs [m][2 rank_pad] (null without).  k % 64 == 0, k < kNvF16MaxK.
size_t f16_rows_bytes(int64_t m, int64_t k, int32_t rank);
hipError_t launch_f16_rows(const uint16_t* x, int64_t m, int64_t k, const uint16_t* lora_a, int32_t rank,
                           float lora_scale, void* scratch, uint16_t** x16, float** rs, uint16_t** t_hl,
                           hipStream_t s);
// Backward dX [m][k] = S rs[m] (dY16 W)[m][k] + (du A)[m][k] over the n weight rows, with
// A^T [k][rank_pad] and du [m][du_stride] (first rank_pad columns) zero past the rank
// (rank_pad 0: no adapter).  n % 64 == 0, n < kNvF16MaxK, k % 128 == 0, k < kNvDxMaxK (copy
// offsets within a stage are 32-bit); part: nvfp4_dx_part_bytes of split-tile partials.
constexpr int64_t kNvDxMaxK = int64_t(1) << 27;
size_t nvfp4_dx_part_bytes(int64_t m, int64_t n, int64_t k);
hipError_t launch_nvfp4_dx(const uint16_t* dy16, const float* rs, int64_t m, int64_t n, int64_t k,
                           const uint8_t* codes, const uint8_t* scales, const float* tensor_scale,
                           const uint16_t* at, const uint16_t* du, int32_t rank_pad, int64_t du_stride, void* dx,
                           int out_f32, float* part, hipStream_t s);
// k % 128 == 0 and k < kFp8MaxK (copy offsets within a 256-row tile are 32-bit).
constexpr int64_t kFp8MaxK = int64_t(1) << 24;
// pow2: sx, sw are E8M0 bytes applied by the scaled MFMA; else float32, folded per K block.
hipError_t launch_gemm_fp8(const uint8_t* xq, const void* sx, int64_t m, int64_t n, int64_t k,
                           const uint8_t* wq, const void* sw, bool pow2, const uint16_t* t,
                           const uint16_t* lora_b, int32_t rank, void* y, int out_f32,
                           hipStream_t s);

// ---- root-mean-square norm with the residual's addition, and its backward pass (norm.hip);
// k % 8 == 0, strides in elements (multiples of 8), 16-byte aligned rows
constexpr int64_t kNormMaxK = 65536;
struct Norm {
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* r;        // residual, or null
  int64_t r_stride;
  const uint16_t* w;
  float eps;
  int64_t m, k;
  uint16_t* h;              // x + r, or null
  int64_t h_stride;
  uint16_t* y;              // bf16 [m][k], or null
  uint8_t* yq;              // with fmt 1 (float32 scales) or 2 (powers of two): E4M3 [m][k]
  void* sy;                 // [m][k / 128]
};
hipError_t launch_rms_norm(const Norm& a, int fmt, hipStream_t s);
struct NormBackward {
  const uint16_t* dy;
  int64_t dy_stride;
  const uint16_t* h;
  int64_t h_stride;
  const uint16_t* w;
  float eps;
  const uint16_t* dh;       // or null
  int64_t dh_stride;
  int64_t m, k;
  uint16_t* dx;
  int64_t dx_stride;
  float* dw;                // float32 [k], or null
  float* part;              // rms_norm_backward_bytes with dw, else null
};
size_t rms_norm_backward_bytes(int64_t m, int64_t k);
hipError_t launch_rms_norm_backward(const NormBackward& a, hipStream_t s);

// ---- gated feed-forward block on FP8 weights (gated.hip); n % 128 == 0, k % 128 == 0
struct Gated {
  const uint8_t* xq;        // E4M3 [m][k]
  const void* sx;           // [m][k / 128]: float32, or E8M0 bytes with pow2, as all scales here
  const uint8_t* wg;        // E4M3 [n][k]
  const void* sg;           // [n / 128][k / 128]
  const uint8_t* wu;
  const void* su;
  bool pow2;
  int64_t m, n, k;
  uint16_t* h;              // bf16 [m][n], or null
  uint8_t* hq;              // E4M3 [m][n], or null
  void* sh;                 // [m][n / 128]
  uint16_t* gu;             // bf16 [m][2 n], or null
  uint32_t* counters;       // zero before and after a call
  float* scratch;           // gated_scratch_bytes
  // set by the launcher
  int64_t tiles_m, tiles_n;
  int split;                // parts of K, each of blocks_each blocks of 128
  int64_t blocks_each;
};
bool gated_launchable(int64_t m, int64_t n, int64_t k);
size_t gated_scratch_bytes(int64_t m, int64_t n, int64_t k);
hipError_t launch_gated(Gated a, hipStream_t s);

// ---- its backward pass (gated_bwd.hip)
struct GatedBackward {
  const uint16_t* dh;       // bf16 [m][n]
  const uint16_t* gu;       // bf16 [m][2 n]
  const uint16_t* x;        // bf16 [m][k], read for dgate and dup
  const uint8_t* wg;
  const void* sg;
  const uint8_t* wu;
  const void* su;
  bool pow2;
  int64_t m, n, k;
  uint16_t* dx;             // bf16 [m][k], or null
  uint16_t* dgate;          // bf16 [n][k], both or neither
  uint16_t* dup;
  void* scratch;            // gated_backward_bytes
};
bool gated_backward_launchable(int64_t m, int64_t n, int64_t k);
size_t gated_backward_bytes(int64_t m, int64_t n, int64_t k);
hipError_t launch_gated_backward(const GatedBackward& a, hipStream_t s);

}  // namespace ql
