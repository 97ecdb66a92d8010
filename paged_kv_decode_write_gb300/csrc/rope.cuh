// Rotary embedding and asynchronous staging shared by the cache-write kernels:
// the fp64 rotation table of a position and a rotated element's single
// rounding into the storage type.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace photon {

// 2*pi = kTwoPiHi + kTwoPiLo: kTwoPiHi holds the leading 30 significant bits
// (so k * kTwoPiHi is exact for |k| < 2^23) and kTwoPiLo the remainder,
// rounded to double.  Used to reduce angles before sincos.
constexpr double kTwoPiHi = 0x1.921fb548p+2;
constexpr double kTwoPiLo = -0x1.de973dcb3b39ap-29;
constexpr double kInvTwoPi = 0x1.45f306dc9c883p-3;

// Nearest-even bf16 of a double in one rounding: truncate to float, keep an
// inexact-sticky bit in the last place (round-to-odd), then round the float
// to bf16.  Round-to-odd to 24 bits followed by round-to-nearest to 8 bits
// equals direct rounding to 8 bits (Boldo & Melquiond, "Emulation of FMA and
// correctly rounded sums: proved algorithms using rounding to odd", 2008).
__device__ __forceinline__ __nv_bfloat16 f64_to_bf16(double x) {
  float f = __double2float_rz(x);
  if (static_cast<double>(f) != x) f = __uint_as_float(__float_as_uint(f) | 1u);
  return __float2bfloat16_rn(f);
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Rotation table of one position: cs[i] = (cos, sin) of pos * inv_freq[i] in
// fp64 (the angle first reduced to [-pi, pi] with the two-term 2*pi), cs32
// the same rounded to fp32.  Visible after the caller's next barrier.
template <int THREADS>
__device__ __forceinline__ void rope_table(const WriteArgs &a, int pos, double (*cs)[2],
                                           float (*cs32)[2]) {
  const double p = static_cast<double>(pos);
#pragma unroll 1
  for (int i = threadIdx.x; i < a.head_dim / 2; i += THREADS) {
    const double ang = p * a.inv_freq[i];
    const double k = rint(ang * kInvTwoPi);
    double sn, c;
    sincos(fma(-k, kTwoPiLo, fma(-k, kTwoPiHi, ang)), &sn, &c);
    cs[i][0] = c;
    cs[i][1] = sn;
    cs32[i][0] = static_cast<float>(c);
    cs32[i][1] = static_cast<float>(sn);
  }
}

// The rare fp64 decisions, out of line (kept off the instruction stream of
// the common path).
static __device__ __noinline__ __nv_bfloat16 rotate_bf16_fp64(float u, float w, double c, double t) {
  return f64_to_bf16(static_cast<double>(u) * c + static_cast<double>(w) * t);
}

// One rotated element y = u*c + w*t (t = -sin for the first of a pair, +sin
// for the second) of pair i, rounded once from its exact value into the
// storage type.
template <typename Tag>
struct Rotate;

template <>
struct Rotate<F32Tag> {
  // fp64 products, one rounding to fp32
  __device__ __forceinline__ static float run(float u, float w, float, float, const double (*cs)[2],
                                              int i, bool first) {
    const double t = first ? -cs[i][1] : cs[i][1];
    return __double2float_rn(static_cast<double>(u) * cs[i][0] + static_cast<double>(w) * t);
  }
};

template <>
struct Rotate<BF16Tag> {
  // fp32 first: y = fl(u*c32 + fl(w*t32)) with c32, t32 the fp32 roundings of
  // the fp64 cos / sin is within 2^-23 * (|u| + |w| + |y|) of the exact
  // u*c + w*t (three relative roundings of 2^-24, |cos|, |sin| <= 1).  With
  // twice that margin, if y - e and y + e round to the same bf16, so does
  // the exact value (rounding is monotonic), and that bf16 is the answer.
  // Otherwise -- a value within the margin of a rounding boundary, rare --
  // the fp64 products decide.
  __device__ __forceinline__ static __nv_bfloat16 run(float u, float w, float c32, float t32,
                                                      const double (*cs)[2], int i, bool first) {
    const float y = fmaf(u, c32, w * t32);
    const float e = fmaf(fabsf(y) + fabsf(u) + fabsf(w), 0x1p-22f, 0x1p-126f);
    const __nv_bfloat16 lo = __float2bfloat16_rn(y - e);
    const __nv_bfloat16 hi = __float2bfloat16_rn(y + e);
    if (__bfloat16_as_ushort(lo) == __bfloat16_as_ushort(hi)) return lo;
    return rotate_bf16_fp64(u, w, cs[i][0], first ? -cs[i][1] : cs[i][1]);
  }
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

}  // namespace photon
