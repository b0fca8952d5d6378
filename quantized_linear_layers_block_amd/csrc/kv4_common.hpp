// Layout of the NVFP4 KV cache, shared by the codec (kv4.hip) and the attention (attn4.hip).
//
// The cache is [page][head][page_size / 16] groups; a group holds 16 tokens of one head:
//   K codes  [16 t][D/2]                    two E2M1 codes a byte, even element in the low nibble
//   K scales [16 t][D/16]                   E4M3, one for 16 elements
//   K exps   [16 t]                         e + 127 of the row's power-of-two scale 2^e
//   V codes  [4 t/4][16 m][D/32 j][4 t%4]   the byte of elements 2p and 2p + 1, p = 16 j + m
//   V scales [4 t/4][2 b%2][D/32 b/2][4 t%4]  E4M3 of block b
//   V exps   [16 t]
// K rows are in the order in which a lane of a 16x16x32 MFMA takes them as the row operand (one
// token, D/4 consecutive elements).  V is turned by four tokens at a time: a lane takes one
// pair of elements of four tokens as one dword, so V^T is a row operand without a transposition
// through shared memory.  18 D + 32 bytes a group: 73 bytes a row at D = 128, 256 in bf16.
#pragma once

#include "common.hpp"

namespace ql {

constexpr int kKv4Group = 16;   // tokens of a group
constexpr int kKv4MinExp = -100, kKv4MaxExp = 117;

__host__ __device__ constexpr int kv4_group_bytes(int d) { return 18 * d + 32; }
__host__ __device__ constexpr int kv4_k_scales(int d) { return 8 * d; }
__host__ __device__ constexpr int kv4_k_exps(int d) { return 9 * d; }
__host__ __device__ constexpr int kv4_v_codes(int d) { return 9 * d + 16; }
__host__ __device__ constexpr int kv4_v_scales(int d) { return 17 * d + 16; }
__host__ __device__ constexpr int kv4_v_exps(int d) { return 18 * d + 16; }

}  // namespace ql
