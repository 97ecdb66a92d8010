// The 8-bit KV page record with one scale per block and KV head: byte positions
// shared by the kernels that write, read and attend over it.
//
// One record per (block, KV head) holds K and V of 16 tokens, 16 d bytes each,
// and their two fp32 scales, so that a page is one bulk copy.  A stored byte is
// the code + 128, |code| <= 127: bytes 0 .. 255 turn into f16 numbers by being
// dropped into the mantissa of 1024 (one byte permute for a pair) and
// subtracting 1152.  value = code * scale.
//
//   K planes  at 1024 hh               (hh = dim / 64)
//     the row of token r = 4a + 2n + j is row 8n + 2a + j, 64 dims in order:
//     lane 4 (2a + j) + c of a decode warp reads its 16 dims 16c .. 16c + 15 of
//     fragment n as chunk 32n + lane, without bank conflicts
//   V planes  at 16 d + 1024 hh
//     chunk 32q + 4g + c (16 bytes): dims 8g .. 8g + 7 of token 4c + 2q, then of
//     token 4c + 2q + 1
//   scales    at 32 d: fp32 of K, fp32 of V; 8 bytes unused
// Eight dims of a token are eight neighbouring bytes in both, so one token is
// written without touching its neighbours' bytes.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace photon {

__host__ __device__ constexpr int int8_record_bytes(int head_dim) { return 32 * head_dim + 16; }

// First byte of dims e .. e + 7 (e a multiple of 8) of token r's K row.
__device__ __forceinline__ int int8_k_byte(int r, int e) {
  return 1024 * (e >> 6) + 64 * (8 * ((r >> 1) & 1) + 2 * (r >> 2) + (r & 1)) + (e & 63);
}

// The same of its V row.
__device__ __forceinline__ int int8_v_byte(int d, int r, int e) {
  return 16 * d + 1024 * (e >> 6) + 512 * ((r >> 1) & 1) + 16 * (4 * ((e & 63) >> 3) + (r >> 2)) + 8 * (r & 1);
}

// First byte of the scale; v: 0 for K, 1 for V.
__host__ __device__ constexpr int int8_scale_byte(int d, int v) { return 32 * d + 4 * v; }

constexpr float kInt8Least = 0x1p-100f;  // smaller scales count as zero

}  // namespace photon
