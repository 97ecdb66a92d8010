// The 4-bit (E2M1) KV page record: byte positions and code conversions shared
// by the kernels that write, read and attend over it.
//
// One record per (block, KV head) holds K and V of 16 tokens in 1088 bytes per
// 64 head dims, ordered so that a warp's tensor-core fragments are whole
// 16-byte chunks, lane l's chunk at byte 16 l of a 512-byte plane (one plane
// per 64 dims): a decode warp reads a plane with one coalesced 16-byte load
// per lane and no shuffle.  No byte is shared by two tokens, so tokens of one
// page may be written concurrently.
//
//   K planes  at 512 hh                (hh = dim / 64)
//     token r = 4c' + 2n + j of the page is column 2c' + j of score fragment n;
//     lane 4 (2c' + j) + c holds its dims 16c .. 16c + 15 of the plane in bytes
//     8n .. 8n + 7, two dims per byte, the even one in the low nibble
//   V planes  at 8 d + 512 hh
//     lane 4g + c holds dims 8g .. 8g + 7 of tokens 4c .. 4c + 3, one 32-bit
//     word per token, dim 8g + i in nibble i
//   scales    at 16 d + 64 hh
//     chunk c (16 bytes): bf16 K scales of tokens 4c .. 4c + 3, then their V
//     scales
// value = code * scale.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace photon {

constexpr int kFp4Group = 64;  // head dims that share a scale

__host__ __device__ constexpr int fp4_record_bytes(int head_dim) { return 17 * head_dim; }

// Byte of dims (e, e + 1), e even, of token r's K row.
__device__ __forceinline__ int fp4_k_byte(int r, int e) {
  const int lane = 4 * (2 * (r >> 2) + (r & 1)) + ((e & 63) >> 4);
  return 512 * (e >> 6) + 16 * lane + 8 * ((r >> 1) & 1) + ((e & 15) >> 1);
}

// Byte of dims (e, e + 1), e even, of token r's V row.
__device__ __forceinline__ int fp4_v_byte(int d, int r, int e) {
  const int lane = 4 * ((e & 63) >> 3) + (r >> 2);
  return 8 * d + 512 * (e >> 6) + 16 * lane + 4 * (r & 3) + ((e & 7) >> 1);
}

// First byte of token r's scale of dims 64 hh .. 64 hh + 63; v: 0 for K, 1 for V.
__device__ __forceinline__ int fp4_scale_byte(int d, int r, int hh, int v) {
  return 16 * d + 64 * hh + 16 * (r >> 2) + 8 * v + 2 * (r & 3);
}

// Eight values -> their nearest E2M1 codes (halves to the even code, saturating
// at +-6), value i in nibble i.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&y)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 p0, p1, p2, p3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 p1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 p3, %8, %7;\n\t"
      "mov.b32 %0, {p0, p1, p2, p3};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// The four code pairs of a word -> f16x2 (exact), byte i to out[i].
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&out)[4]) {
  asm("{\n\t.reg .b8 p0, p1, p2, p3;\n\tmov.b32 {p0, p1, p2, p3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, p0;\n\tcvt.rn.f16x2.e2m1x2 %1, p1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, p2;\n\tcvt.rn.f16x2.e2m1x2 %3, p3;\n\t}"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(w));
}

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t b) { return __uint_as_float(b << 16); }

}  // namespace photon
