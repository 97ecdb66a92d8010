// 4-bit (E2M1) KV cache: the RoPE-fused quantising write and the dequantising
// read (sm_103a).  Record layout in fp4.cuh.
//
// Write, per token and KV head: y = the row, K rotated, rounded to fp32 and
// then to the input type; per 64 dims the scale s = bf16(max|y| / 6) and the
// codes round(y / s), to nearest with halves to the even code.  Read: code * s
// rounded to the output type.
//
// Both work in words of 8 dims, which lie in one 32-bit word of a record for K
// and for V alike: the read turns a word into one 16-byte (bf16) store, a
// write's lane holds words w and w + D/16 of a row, so that both halves of
// every rotation pair, of either style, are in the lane.
#include <cuda_fp16.h>

#include <climits>
#include <cmath>

#include "fp4.cuh"
#include "rope.cuh"

namespace photon {
namespace {

constexpr int kFp4Threads = 256;

// ---- rotation angles -----------------------------------------------------------
// The fp64 pipe is too narrow for a sine and cosine per (token, pair) of a long
// prompt (16384 tokens of d 64: 50 us of fp64 work beside 6 us of memory
// traffic), so angles are fixed-point fractions of a turn and the trigonometry
// is fp32 pairs (value = hi + lo):
//   pos * F mod 2^64, F = 2^64 * theta^(-2i/d) / 2 pi, is the turn's fraction,
//   reduced exactly by the integer wrap; its leading 8 bits (rounded) name a
//   table angle a_k = 2 pi k / 256, the rest is delta, |delta| <= pi / 256;
//   cos(a + delta) = cos a + (cos a (cos delta - 1) - sin a sin delta), the
//   bracket below 0.0124, so that fp32 products with their fma remainders keep
//   about 2^-38 of absolute error: no bf16 rounding of a rotated value is ever
//   in doubt by more than the fp64 angle's own rounding puts it.

struct TurnTable {
  float v[256][4];  // cos hi, cos lo, sin hi, sin lo
};

constexpr double kTurn = 6.283185307179586476925286766559;

// Taylor series on |x| <= pi / 4 (17 terms are far past fp64's precision).
constexpr double taylor_sin(double x) {
  double term = x, sum = x;
  for (int n = 1; n < 12; ++n) {
    term *= -x * x / ((2 * n) * (2 * n + 1));
    sum += term;
  }
  return sum;
}
constexpr double taylor_cos(double x) {
  double term = 1, sum = 1;
  for (int n = 1; n < 12; ++n) {
    term *= -x * x / ((2 * n - 1) * (2 * n));
    sum += term;
  }
  return sum;
}

constexpr TurnTable make_turn_table() {
  TurnTable t{};
  for (int k = 0; k < 256; ++k) {
    const int oct = ((k + 32) / 64) & 3;          // nearest quarter turn
    const int rest = k - 64 * ((k + 32) / 64);     // -32 .. 31
    const double x = kTurn * rest / 256, s0 = taylor_sin(x), c0 = taylor_cos(x);
    const double c = oct == 0 ? c0 : oct == 1 ? -s0 : oct == 2 ? -c0 : s0;
    const double s = oct == 0 ? s0 : oct == 1 ? c0 : oct == 2 ? -s0 : -c0;
    t.v[k][0] = static_cast<float>(c);
    t.v[k][1] = static_cast<float>(c - static_cast<double>(t.v[k][0]));
    t.v[k][2] = static_cast<float>(s);
    t.v[k][3] = static_cast<float>(s - static_cast<double>(t.v[k][2]));
  }
  return t;
}

__device__ __align__(16) const TurnTable g_turn = make_turn_table();

// hi + lo = a + b exactly (the intrinsics keep the compiler from contracting
// a product into a sum, which would break the remainders).
__device__ __forceinline__ void two_sum(float a, float b, float &hi, float &lo) {
  hi = __fadd_rn(a, b);
  const float t = __fsub_rn(hi, a);
  lo = __fadd_rn(__fsub_rn(a, __fsub_rn(hi, t)), __fsub_rn(b, t));
}

// p + e = a * b exactly.
__device__ __forceinline__ void two_prod(float a, float b, float &p, float &e) {
  p = __fmul_rn(a, b);
  e = __fmaf_rn(a, b, -p);
}

// (cos hi, cos lo, sin hi, sin lo) of the fraction `turn` / 2^64 of a turn.
__device__ __forceinline__ float4 cos_sin_turn(unsigned long long turn) {
  const unsigned k = static_cast<unsigned>((turn + (1ull << 55)) >> 56) & 255u;
  const long long rest = static_cast<long long>(turn - (static_cast<unsigned long long>(k) << 56));
  const float4 a = *reinterpret_cast<const float4 *>(g_turn.v[k]);
  // delta = 2 pi rest / 2^64 as dh + dl; rest has at most 56 bits
  const float rh = __ll2float_rn(rest);
  const float rl = __ll2float_rn(rest - static_cast<long long>(rh));
  constexpr float kPiHi = static_cast<float>(kTurn * 0x1p-64);
  constexpr float kPiLo = static_cast<float>(kTurn * 0x1p-64 - static_cast<double>(kPiHi));
  float dh, de;
  two_prod(rh, kPiHi, dh, de);
  const float dl = de + fmaf(rh, kPiLo, rl * kPiHi);
  const float d2 = dh * dh;
  // sin delta = dh + sl;  cos delta - 1 = cm
  const float sl = fmaf(dh * d2, fmaf(d2, 1.f / 120.f, -1.f / 6.f), dl);
  const float cm = fmaf(d2, fmaf(d2, 1.f / 24.f, -0.5f), -dh * dl);
  float4 r;
  float p, pe, h, l;
  two_prod(-a.z, dh, p, pe);
  two_sum(a.x, p, h, l);
  two_sum(h, l + (fmaf(a.x, cm, pe) + (a.y - fmaf(a.z, sl, a.w * dh))), r.x, r.y);
  two_prod(a.x, dh, p, pe);
  two_sum(a.z, p, h, l);
  two_sum(h, l + (fmaf(a.z, cm, pe) + (a.w + fmaf(a.x, sl, a.y * dh))), r.z, r.w);
  return r;
}

// fp32 rounding of u c + w t, c and t given as hi + lo: exact products (fma
// remainders), exact sum of the leading parts, the rest in fp32.
__device__ __forceinline__ float rotated(float u, float w, float ch, float cl, float th, float tl) {
  float p, pe, q, qe, s, se;
  two_prod(u, ch, p, pe);
  two_prod(w, th, q, qe);
  two_sum(p, q, s, se);
  return s + (se + (fmaf(u, cl, pe) + fmaf(w, tl, qe)));
}

// ---- codes -----------------------------------------------------------------------

// max that keeps a NaN of either operand
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Scale of a group whose largest magnitude is m (bf16 bits); a group that
// holds an infinity or a NaN gets a NaN scale.
__device__ __forceinline__ uint32_t group_scale(float m) {
  if (!(m <= 3.4028234663852886e38f)) return 0x7fffu;
  return __bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(m, 6.f)));
}

// x / s close enough for the code: y0 = x fl(1/s) corrected once by its exact
// residual is the quotient when it has few bits, a midpoint of two codes among
// them, and within an ulp otherwise.  A bf16 x (8 bits) over a bf16 s is never
// within 2^-11 of a midpoint without being it; an fp32 x may be, and its y may
// round onto the midpoint: the residual's sign then says which side it is on.
template <typename Tag>
__device__ __forceinline__ float quotient(float x, float s, float is) {
  const float y0 = x * is;
  float y = fmaf(fmaf(-y0, s, x), is, y0);
  if (sizeof(typename Tag::T) == 4 && (__float_as_uint(y) & 0x1fffffu) == 0u) {
    const float r = fmaf(-y, s, x);  // exact
    if (r != 0.f && y != 0.f)
      y = __uint_as_float(__float_as_uint(y) + ((r > 0.f) == (y > 0.f) ? 1 : -1));
  }
  return y;
}

// Code of x / s for scales whose reciprocal or residuals leave fp32's range:
// comparisons with midpoints (at most three bits) times s (eight), exact.
__device__ __noinline__ uint32_t code_by_midpoints(float x, float s) {
  const float m = fabsf(x);
  const uint32_t c = (m > 0.25f * s) + (m >= 0.75f * s) + (m > 1.25f * s) + (m >= 1.75f * s) +
                     (m > 2.5f * s) + (m >= 3.5f * s) + (m > 5.f * s);
  return c | (x < 0.f ? 8u : 0u);
}

// The codes of 8 dims, dim i in nibble i.
template <typename Tag>
__device__ __forceinline__ uint32_t quant_word(const float (&x)[8], uint32_t sbits) {
  const float s = bf16_bits_to_f32(sbits);
  if (!(s > 0.f)) return 0u;  // an all-zero (or non-finite) group
  uint32_t w = 0;
  if (s < 0x1p-100f) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) w |= code_by_midpoints(x[i], s) << (4 * i);
    return w;
  }
  const float is = __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= cvt_e2m1x2(quotient<Tag>(x[2 * i], s, is), quotient<Tag>(x[2 * i + 1], s, is)) << (8 * i);
  return w;
}

__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
  Unpack<BF16Tag>::run(*reinterpret_cast<const uint4 *>(p), x);
}

// fp32 value of v rounded to the storage type
__device__ __forceinline__ float stored(float v, const float *) { return v; }
__device__ __forceinline__ float stored(float v, const __nv_bfloat16 *) {
  return __bfloat162float(__float2bfloat16_rn(v));
}

// One CTA per tile of tokens (all heads): the tile's rotation table in shared
// memory, then rows (K or V, head, token), token fastest, D/16 lanes each.
template <typename Tag, int D>
__global__ void __launch_bounds__(kFp4Threads)
    kv_cache_write_fp4_kernel(const __grid_constant__ Fp4WriteArgs a, unsigned int *err) {
  using T = typename Tag::T;
  constexpr int LPR = D / 16;  // lanes of a row
  constexpr int HALF = D / 2;
  __shared__ float4 cs[kFp4MaxTile][HALF];
  __shared__ int64_t slots[kFp4MaxTile];
  pdl_wait();
  pdl_launch_dependents();
  const int H = a.num_kv_heads;
  const int t0 = blockIdx.x * a.tile, n = min(a.tile, a.num_tokens - t0);
  const bool rotate = a.rope_style != PHOTON_ROPE_NONE;
  const bool gptj = a.rope_style == PHOTON_ROPE_GPTJ;
  if (threadIdx.x < n) {
    const int64_t slot = a.slot_mapping[t0 + threadIdx.x];
    if (slot >= a.num_slots) atomicOr(err, PHOTON_DEVERR_SLOT_RANGE);
    slots[threadIdx.x] = slot < a.num_slots ? slot : -1;
  }
  if (rotate)
    for (int i = threadIdx.x; i < n * HALF; i += kFp4Threads)
      cs[i / HALF][i % HALF] =
          cos_sin_turn(static_cast<unsigned long long>(static_cast<long long>(a.positions[t0 + i / HALF])) *
                       a.turns[i % HALF]);
  __syncthreads();
  const int w = threadIdx.x % LPR;
  const int rows = 2 * H * n;
  // whole rows per warp: every lane of a row takes part in its shuffles
  for (int row = threadIdx.x / LPR; row - (threadIdx.x & 31) / LPR < rows; row += kFp4Threads / LPR) {
    const bool in = row < rows;
    const int tt = in ? row % n : 0, hv = in ? row / n : 0;
    const int v = hv >= H, h = hv - (v ? H : 0);  // K rows first
    const int64_t slot = slots[tt];
    const bool live = in && slot >= 0;
    const T *src = static_cast<const T *>(v ? a.v : a.k) + (static_cast<int64_t>(t0 + tt) * H + h) * D + 8 * w;
    float x0[8], x1[8];
    load8(src, x0);
    load8(src + HALF, x1);
    if (rotate && !v) {
      if (gptj) {  // pairs (2i, 2i + 1): 4w .. 4w + 3, and D/4 + those in the upper half
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 p = cs[tt][4 * w + i], q = cs[tt][D / 4 + 4 * w + i];
          const float a0 = x0[2 * i], b0 = x0[2 * i + 1], a1 = x1[2 * i], b1 = x1[2 * i + 1];
          x0[2 * i] = stored(rotated(a0, b0, p.x, p.y, -p.z, -p.w), src);
          x0[2 * i + 1] = stored(rotated(b0, a0, p.x, p.y, p.z, p.w), src);
          x1[2 * i] = stored(rotated(a1, b1, q.x, q.y, -q.z, -q.w), src);
          x1[2 * i + 1] = stored(rotated(b1, a1, q.x, q.y, q.z, q.w), src);
        }
      } else {     // pairs (e, e + D/2)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 p = cs[tt][8 * w + i];
          const float a0 = x0[i], b0 = x1[i];
          x0[i] = stored(rotated(a0, b0, p.x, p.y, -p.z, -p.w), src);
          x1[i] = stored(rotated(b0, a0, p.x, p.y, p.z, p.w), src);
        }
      }
    }
    float m0 = fabsf(x0[0]), m1 = fabsf(x1[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      m0 = max_nan(m0, fabsf(x0[i]));
      m1 = max_nan(m1, fabsf(x1[i]));
    }
    if (D == 64) m0 = max_nan(m0, m1);  // one group of 64 dims; at D = 128 x0 and x1 are one each
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
      m0 = max_nan(m0, __shfl_xor_sync(0xffffffffu, m0, o));
      if (D > 64) m1 = max_nan(m1, __shfl_xor_sync(0xffffffffu, m1, o));
    }
    if (!live) continue;
    const uint32_t s0 = group_scale(m0), s1 = D > 64 ? group_scale(m1) : s0;
    const int64_t blk = slot / kBlockSize;
    const int r = static_cast<int>(slot - blk * kBlockSize);
    unsigned char *rec = static_cast<unsigned char *>(a.kv_cache) + (blk * H + h) * fp4_record_bytes(D);
    const int e0 = 8 * w, e1 = 8 * w + HALF;
    *reinterpret_cast<uint32_t *>(rec + (v ? fp4_v_byte(D, r, e0) : fp4_k_byte(r, e0))) = quant_word<Tag>(x0, s0);
    *reinterpret_cast<uint32_t *>(rec + (v ? fp4_v_byte(D, r, e1) : fp4_k_byte(r, e1))) = quant_word<Tag>(x1, s1);
    if (w < D / kFp4Group)
      *reinterpret_cast<uint16_t *>(rec + fp4_scale_byte(D, r, w, v)) = static_cast<uint16_t>(w ? s1 : s0);
  }
}

// ---- read --------------------------------------------------------------------------

__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
  uint4 w;
  uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  *reinterpret_cast<uint4 *>(p) = w;
}

// One CTA per (16 consecutive tokens, KV head): tokens of one page then share
// the sectors they read.  A lane takes one word of 8 dims of K or V per step,
// all steps' loads in flight at once.
constexpr int kFp4ReadTile = 16;

template <typename Tag, int D>
__global__ void __launch_bounds__(kFp4Threads)
    kv_cache_read_fp4_kernel(const Fp4ReadArgs a, unsigned int *err) {
  using T = typename Tag::T;
  constexpr int WORDS = D / 4;                              // of K and V of a token and head
  constexpr int STEPS = kFp4ReadTile * WORDS / kFp4Threads;  // 1 or 2
  static_assert(STEPS * kFp4Threads == kFp4ReadTile * WORDS, "whole steps");
  pdl_wait();
  pdl_launch_dependents();
  const int H = a.num_kv_heads;
  const int tile = blockIdx.x / H, h = blockIdx.x - tile * H;
  const int v = (threadIdx.x / (WORDS / 2)) & 1, e = 8 * (threadIdx.x % (WORDS / 2));
  uint32_t code[STEPS], scale[STEPS];
  int64_t row[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t t = static_cast<int64_t>(tile) * kFp4ReadTile + (i * kFp4Threads + threadIdx.x) / WORDS;
    row[i] = -1;
    if (t >= a.num_tokens) continue;
    const int64_t slot = a.slot_mapping[t];
    if (slot < 0) continue;
    if (slot >= a.num_slots) {
      atomicOr(err, PHOTON_DEVERR_SLOT_RANGE);
      continue;
    }
    const int64_t blk = slot / kBlockSize;
    const int r = static_cast<int>(slot - blk * kBlockSize);
    const unsigned char *rec = static_cast<const unsigned char *>(a.pool) + (blk * H + h) * fp4_record_bytes(D);
    code[i] = *reinterpret_cast<const uint32_t *>(rec + (v ? fp4_v_byte(D, r, e) : fp4_k_byte(r, e)));
    scale[i] = *reinterpret_cast<const uint16_t *>(rec + fp4_scale_byte(D, r, e / kFp4Group, v));
    row[i] = t * H + h;
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    if (row[i] < 0) continue;
    uint32_t f[4];
    e2m1x8_to_f16(code[i], f);
    const float s = bf16_bits_to_f32(scale[i]);
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&f[j]));
      x[2 * j] = p.x * s;
      x[2 * j + 1] = p.y * s;
    }
    store8(static_cast<T *>(v ? a.v_out : a.k_out) + row[i] * D + e, x);
  }
}

template <typename Tag>
cudaError_t launch_write(const Fp4WriteArgs &a, unsigned int *err, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.num_tokens) + a.tile - 1) / a.tile));
  auto kern = a.head_dim == 64 ? kv_cache_write_fp4_kernel<Tag, 64> : kv_cache_write_fp4_kernel<Tag, 128>;
  return launch_pdl(kern, grid, dim3(kFp4Threads), 0, st, a, err);
}

template <typename Tag>
cudaError_t launch_read(const Fp4ReadArgs &a, unsigned int *err, cudaStream_t st) {
  const int64_t tiles = (static_cast<int64_t>(a.num_tokens) + kFp4ReadTile - 1) / kFp4ReadTile;
  if (tiles * a.num_kv_heads > INT32_MAX) return cudaErrorInvalidValue;
  auto kern = a.head_dim == 64 ? kv_cache_read_fp4_kernel<Tag, 64> : kv_cache_read_fp4_kernel<Tag, 128>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(tiles * a.num_kv_heads)), dim3(kFp4Threads), 0, st, a, err);
}

}  // namespace

cudaError_t launch_kv_cache_write_fp4(const WriteArgs &wa, photon_dtype in_dt, unsigned int *err,
                                      cudaStream_t st) {
  if (wa.num_tokens == 0) return cudaSuccess;
  Fp4WriteArgs a{};
  a.k = wa.k;
  a.v = wa.v;
  a.positions = wa.positions;
  a.slot_mapping = wa.slot_mapping;
  a.kv_cache = wa.k_cache;
  a.num_slots = wa.num_slots;
  a.num_tokens = wa.num_tokens;
  a.num_kv_heads = wa.num_kv_heads;
  a.head_dim = wa.head_dim;
  a.rope_style = wa.rope_style;
  for (int i = 0; i < wa.head_dim / 2; ++i) {
    const double x = wa.inv_freq[i] / kTurn;
    a.turns[i] = static_cast<unsigned long long>(std::ldexp(x - std::floor(x), 64));
  }
  // tokens per CTA: as many as leave two CTAs per SM
  const int64_t per = wa.num_tokens / (2 * static_cast<int64_t>(device_sm_count()));
  a.tile = per >= 8 ? 8 : per >= 4 ? 4 : per >= 2 ? 2 : 1;
  return in_dt == PHOTON_BF16 ? launch_write<BF16Tag>(a, err, st) : launch_write<F32Tag>(a, err, st);
}

cudaError_t launch_kv_cache_read_fp4(const Fp4ReadArgs &a, photon_dtype out_dt, unsigned int *err,
                                     cudaStream_t st) {
  if (a.num_tokens == 0) return cudaSuccess;
  return out_dt == PHOTON_BF16 ? launch_read<BF16Tag>(a, err, st) : launch_read<F32Tag>(a, err, st);
}

}  // namespace photon
