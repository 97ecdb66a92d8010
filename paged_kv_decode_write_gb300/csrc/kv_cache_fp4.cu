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
#include "row_lanes.cuh"

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
//   bracket below 0.0124: its leading product and sum keep their remainders,
//   the rest, cos a (cos delta - 1) the largest of it, takes six fp32 roundings
//   of values below 2^-13: within 2^-35.4 (2^-35.8 the worst of 2^22 angles).
// F carries the 53 bits of an fp64 frequency, so the angle itself is within
// 2^-50 of its radians, as an fp64 product of position and frequency would be.

struct TurnTable {
  float v[256][4];  // cos hi, cos lo, sin hi, sin lo
};

constexpr double kTurn = 6.283185307179586476925286766559;

// Taylor series on |x| <= pi / 4 (12 terms are past fp64's precision).
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
  const unsigned long long up = turn + (1ull << 55);
  const float4 a = *reinterpret_cast<const float4 *>(g_turn.v[up >> 56]);
  // rest = delta in units of 2^-64 turn, 56 bits: its leading 20 bits (signed)
  // and the next 22 as exact floats through the mantissa (no conversion unit)
  const unsigned hi = static_cast<unsigned>((up >> 24) & 0xffffffffu) ^ 0x80000000u;  // signed, 2^-40 turn
  const unsigned lo = static_cast<unsigned>(up) & 0xffffffu;                            // 24 more bits
  const float r1 = __uint_as_float(0x4b400000u + static_cast<unsigned>(static_cast<int>(hi) >> 12)) - 12582912.f;
  const float r2 = __uint_as_float(0x4b000000u | ((hi & 0xfffu) << 10) | (lo >> 14)) - 8388608.f;
  // in units of 2^-28 turn: rh + rl = r1 + r2 2^-22
  const float rs = r2 * 0x1p-22f;
  const float rh = __fadd_rn(r1, rs);
  const float rl = __fsub_rn(rs, __fsub_rn(rh, r1));
  constexpr float kPiHi = static_cast<float>(kTurn * 0x1p-28);
  constexpr float kPiLo = static_cast<float>(kTurn * 0x1p-28 - static_cast<double>(kPiHi));
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

// The same of bf16 u and w, rounded to bf16 as well; ch and th have 16 bits
// (table_entry), so that both products are exact and need no remainder.
__device__ __forceinline__ float rotated_bf16(float u, float w, float ch, float cl, float th, float tl) {
  float s, se;
  two_sum(__fmul_rn(u, ch), __fmul_rn(w, th), s, se);
  return __bfloat162float(__float2bfloat16_rn(s + (se + fmaf(u, cl, w * tl))));
}

// A position's (cos, sin) as the rotation of T takes it.
template <typename T>
__device__ __forceinline__ float4 table_entry(unsigned long long turn) {
  float4 p = cos_sin_turn(turn);
  if (sizeof(T) == 2) {
    const float c = __uint_as_float(__float_as_uint(p.x) & 0xffffff00u);
    const float s = __uint_as_float(__float_as_uint(p.z) & 0xffffff00u);
    p = make_float4(c, (p.x - c) + p.y, s, (p.z - s) + p.w);
  }
  return p;
}

// The 8 pairs of a lane, rotated and rounded to fp32 and then to the storage
// type.  NEOX: (x0[i], x1[i]); GPT-J: (x0[2i], x0[2i + 1]), then those of x1.
// cs: step i's entry at cs[i * stride].  (fp32 arithmetic first, with the
// accurate sums only where an error bound leaves the bf16 rounding open, took
// more registers and local memory: 30.5 -> 36.8 us for 16384 tokens.)
template <typename T, bool GPTJ>
__device__ __forceinline__ void rotate_lane(float (&x0)[8], float (&x1)[8], const float4 *cs, int stride) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float &u = GPTJ ? (i < 4 ? x0[2 * i] : x1[2 * i - 8]) : x0[i];
    float &w = GPTJ ? (i < 4 ? x0[2 * i + 1] : x1[2 * i - 7]) : x1[i];
    const float4 p = cs[i * stride];
    const float a = u, b = w;
    if constexpr (sizeof(T) == 2) {
      u = rotated_bf16(a, b, p.x, p.y, -p.z, -p.w);
      w = rotated_bf16(b, a, p.x, p.y, p.z, p.w);
    } else {
      u = rotated(a, b, p.x, p.y, -p.z, -p.w);
      w = rotated(b, a, p.x, p.y, p.z, p.w);
    }
  }
}

// ---- codes -----------------------------------------------------------------------

// max |.| that keeps a NaN of any operand
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Scale of a group whose largest magnitude is m (bf16 bits): the quotient m / 6
// rounded to fp32 (the product with 1/6 and one exact residual give it in the
// normal range) and to bf16.  A group that holds an infinity or a NaN gets a
// NaN scale.
__device__ __forceinline__ uint32_t group_scale(float m) {
  if (!(m <= 3.4028234663852886e38f)) return 0x7fffu;
  constexpr float kSixth = 1.f / 6.f;
  const float q0 = __fmul_rn(m, kSixth);
  const float q = m < 0x1p-100f ? __fdiv_rn(m, 6.f) : __fmaf_rn(__fmaf_rn(-q0, 6.f, m), kSixth, q0);
  return __bfloat16_as_ushort(__float2bfloat16_rn(q));
}

// 1 / s within an ulp (s normal, below 2^126).
__device__ __forceinline__ float rcp_approx(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// x / s close enough for the code: y0 = x is, is the reciprocal within an ulp,
// corrected once by its exact residual is the quotient when that has few bits,
// a midpoint of two codes among them, and within an ulp otherwise.  A bf16 x
// (8 bits) over a bf16 s is never within 2^-11 of a midpoint without being it;
// an fp32 x may be, and its y may round onto the midpoint: the residual's sign
// then says which side it is on.
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
  if (s < 0x1p-100f) {
    uint32_t w = 0;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) w |= code_by_midpoints(x[i], s) << (4 * i);
    return w;
  }
  const float is = rcp_approx(s);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = quotient<Tag>(x[i], s, is);
  return cvt_e2m1x8(y);
}

// One CTA per tile of tokens (all heads): the tile's rotation table in shared
// memory, then rows (K or V, head, token), token fastest, D/16 lanes each.
// Four CTAs per SM: at their 64 registers the fp32 kernels spill 36 bytes.
template <typename Tag, int D>
__global__ void __launch_bounds__(kFp4Threads, 4)
    kv_cache_write_fp4_kernel(const __grid_constant__ Fp4WriteArgs a, unsigned int *err) {
  using T = typename Tag::T;
  constexpr int LPR = D / 16;  // lanes of a row
  constexpr int HALF = D / 2;
  // a token's (cos, sin) in the order its lanes read them: step i of lane w at
  // i * LPR + w, rows padded so that a quarter warp's 16-byte reads meet no bank twice
  __shared__ float4 cs[kFp4MaxTile][HALF + (D == 64 ? 4 : 0)];
  pdl_wait();
  pdl_launch_dependents();
  const int H = a.num_kv_heads;
  const int t0 = blockIdx.x << a.tile_log2, tile = 1 << a.tile_log2, n = min(tile, a.num_tokens - t0);
  const bool rotate = a.rope_style != PHOTON_ROPE_NONE;
  const bool gptj = a.rope_style == PHOTON_ROPE_GPTJ;
  // a lane keeps its token; its first row is on the way while the table is made
  const int w = threadIdx.x % LPR, row = threadIdx.x / LPR;
  const int tt = min(row & (tile - 1), n - 1);  // past the last token: its rows again, not written
  const int64_t token = static_cast<int64_t>(t0 + tt) * H * D + 8 * w;
  const T *k_src = static_cast<const T *>(a.k) + token, *v_src = static_cast<const T *>(a.v) + token;
  const int first = row >> a.tile_log2, step = (kFp4Threads / LPR) >> a.tile_log2;
  // rows: K of every head, then V; the same number of turns for every lane
  auto source = [&](int hv) -> const T * {
    hv = min(hv, 2 * H - 1);
    return hv >= H ? v_src + (hv - H) * D : k_src + hv * D;
  };
  RowLoad<T> next;
  next.load(source(first), HALF);
  const int64_t slot_in = a.slot_mapping[t0 + tt];
  if (rotate)
    for (int i = threadIdx.x; i < n * HALF; i += kFp4Threads) {
      const int tt = i / HALF, pair = i % HALF;
      // NEOX: lane w takes pairs 8w ..; GPT-J: 4w .. of either half
      const int at = gptj ? (pair / (D / 4) * 4 + pair % 4) * LPR + pair % (D / 4) / 4 : pair % 8 * LPR + pair / 8;
      cs[tt][at] = table_entry<T>(
          static_cast<unsigned long long>(static_cast<long long>(a.positions[t0 + tt])) * a.turns[pair]);
    }
  __syncthreads();
  if (slot_in >= a.num_slots && w == 0) atomicOr(err, PHOTON_DEVERR_SLOT_RANGE);
  const bool live = (row & (tile - 1)) < n && slot_in >= 0 && slot_in < a.num_slots;
  const int64_t slot = live ? slot_in : 0;
  const int r = static_cast<int>(slot) & (kBlockSize - 1);
  const int e0 = 8 * w, e1 = 8 * w + HALF;
  const int k_at[2] = {fp4_k_byte(r, e0), fp4_k_byte(r, e1)};
  const int v_at[2] = {fp4_v_byte(D, r, e0), fp4_v_byte(D, r, e1)};
  const int s_at = fp4_scale_byte(D, r, w < D / kFp4Group ? w : 0, 0);
  unsigned char *block = static_cast<unsigned char *>(a.kv_cache) +
                         (slot >> 4) * (static_cast<int64_t>(H) * fp4_record_bytes(D));
  for (int base = 0; base < 2 * H; base += step) {
    const int hv = min(base + first, 2 * H - 1);
    const bool in = base + first < 2 * H;
    const int v = hv >= H, h = hv - (v ? H : 0);
    float x0[8], x1[8];
    RowLoad<T>::widen(next.lo, x0);
    RowLoad<T>::widen(next.hi, x1);
    if (base + step < 2 * H) next.load(source(base + step + first), HALF);
    if (rotate && !v) {
      if (gptj)
        rotate_lane<T, true>(x0, x1, cs[tt] + w, LPR);
      else
        rotate_lane<T, false>(x0, x1, cs[tt] + w, LPR);
    }
    // the largest magnitude of each group: at D = 64 one of all dims, at D = 128
    // one of x0 and one of x1
    float m0 = max_abs(x0[0], x0[1], x0[2]), m1 = max_abs(x1[0], x1[1], x1[2]);
    m0 = max_abs(max_abs(m0, x0[3], x0[4]), x0[5], x0[6]);
    m1 = max_abs(max_abs(m1, x1[3], x1[4]), x1[5], x1[6]);
    if (D == 64) {
      m0 = max_abs(max_abs(m0, m1, x0[7]), x1[7], 0.f);
    } else {
      m0 = max_abs(m0, x0[7], 0.f);
      m1 = max_abs(m1, x1[7], 0.f);
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
      m0 = max_abs(m0, __shfl_xor_sync(0xffffffffu, m0, o), 0.f);
      if (D > 64) m1 = max_abs(m1, __shfl_xor_sync(0xffffffffu, m1, o), 0.f);
    }
    if (!live || !in) continue;
    const uint32_t s0 = group_scale(m0), s1 = D > 64 ? group_scale(m1) : s0;
    unsigned char *rec = block + h * fp4_record_bytes(D);
    *reinterpret_cast<uint32_t *>(rec + (v ? v_at[0] : k_at[0])) = quant_word<Tag>(x0, s0);
    *reinterpret_cast<uint32_t *>(rec + (v ? v_at[1] : k_at[1])) = quant_word<Tag>(x1, s1);
    if (w < D / kFp4Group)
      *reinterpret_cast<uint16_t *>(rec + s_at + 8 * v) = static_cast<uint16_t>(w ? s1 : s0);
  }
}

// ---- read --------------------------------------------------------------------------

// One CTA per (tile of consecutive tokens, KV head): tokens of one page then
// share the sectors they read.  A lane takes the same 8 dims of a token's K and
// V, so that the slot's arithmetic serves two words.
template <typename Tag, int D>
__global__ void __launch_bounds__(kFp4Threads)
    kv_cache_read_fp4_kernel(const CacheReadArgs a, int tile, unsigned int *err) {
  using T = typename Tag::T;
  constexpr int LANES = D / 8;  // of a token
  pdl_wait();
  pdl_launch_dependents();
  const int H = a.num_kv_heads, h = blockIdx.x;
  const int e = 8 * (threadIdx.x % LANES);
  // a token's place in the record is a sum of a lane's part and a token's part
  const unsigned char *base = static_cast<const unsigned char *>(a.pool) + static_cast<int64_t>(h) * fp4_record_bytes(D);
  const int k_at = fp4_k_byte(0, e), v_at = fp4_v_byte(D, 0, e), s_at = fp4_scale_byte(D, 0, e / kFp4Group, 0);
  const uint32_t block_bytes = static_cast<uint32_t>(H) * fp4_record_bytes(D);
  const int64_t first = static_cast<int64_t>(blockIdx.y) * tile;
  const int left = static_cast<int>(min(static_cast<int64_t>(tile), a.num_tokens - first));
  const int64_t *slots = a.slot_mapping + first;
  const int64_t out_at = (first * H + h) * D + e;
  T *k_out = static_cast<T *>(a.k_out) + out_at, *v_out = static_cast<T *>(a.v_out) + out_at;
  const uint32_t out_step = static_cast<uint32_t>(H) * D;
#pragma unroll 1  // more loads in flight per lane measured slower (32768 tokens of d 128: 30.0 us, unrolled twice 33.3)
  for (int t = threadIdx.x / LANES; t < left; t += kFp4Threads / LANES) {
    const int64_t slot = slots[t];
    if (static_cast<uint64_t>(slot) >= static_cast<uint64_t>(a.num_slots)) {
      if (slot >= 0) atomicOr(err, PHOTON_DEVERR_SLOT_RANGE);
      continue;
    }
    const uint32_t quad = static_cast<uint32_t>(slot) >> 2 & 3u, odd = static_cast<uint32_t>(slot) & 1u,
                   two = static_cast<uint32_t>(slot) & 2u;
    const unsigned char *rec = base + static_cast<uint64_t>(static_cast<uint32_t>(slot >> 4)) * block_bytes;
    const unsigned char *s = rec + (s_at + 16 * quad + 2 * odd + 2 * two);
    const uint32_t code[2] = {*reinterpret_cast<const uint32_t *>(rec + (k_at + 128 * quad + 64 * odd + 4 * two)),
                              *reinterpret_cast<const uint32_t *>(rec + (v_at + 16 * quad + 4 * odd + 4 * two))};
    const uint32_t scale[2] = {*reinterpret_cast<const uint16_t *>(s), *reinterpret_cast<const uint16_t *>(s + 8)};
    const uint64_t row = static_cast<uint64_t>(static_cast<uint32_t>(t)) * out_step;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      uint32_t f[4];
      e2m1x8_to_f16(code[v], f);
      const float sc = bf16_bits_to_f32(scale[v]);
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&f[j]));
        x[2 * j] = p.x * sc;
        x[2 * j + 1] = p.y * sc;
      }
      store8((v ? v_out : k_out) + row, x);
    }
  }
}

template <typename Tag>
cudaError_t launch_write(const Fp4WriteArgs &a, unsigned int *err, cudaStream_t st) {
  const int64_t tile = int64_t{1} << a.tile_log2;
  const dim3 grid(static_cast<unsigned>((a.num_tokens + tile - 1) / tile));
  auto kern = a.head_dim == 64 ? kv_cache_write_fp4_kernel<Tag, 64> : kv_cache_write_fp4_kernel<Tag, 128>;
  return launch_pdl(kern, grid, dim3(kFp4Threads), 0, st, a, err);
}

template <typename Tag>
cudaError_t launch_read(const CacheReadArgs &a, unsigned int *err, cudaStream_t st) {
  using T = typename Tag::T;
  // 64 tokens per CTA where that leaves eight CTAs per SM, else 16
  const int64_t ctas = (static_cast<int64_t>(a.num_tokens) + 63) / 64 * a.num_kv_heads;
  const int tile = ctas >= 8 * static_cast<int64_t>(device_sm_count()) ? 64 : 16;
  const int64_t tiles = (static_cast<int64_t>(a.num_tokens) + tile - 1) / tile;
  auto kern = a.head_dim == 64 ? kv_cache_read_fp4_kernel<Tag, 64> : kv_cache_read_fp4_kernel<Tag, 128>;
  // the grid's y extent is at most 65535 tiles: longer reads in pieces
  constexpr int64_t kMaxTiles = 65535;
  for (int64_t t = 0; t < tiles; t += kMaxTiles) {
    CacheReadArgs p = a;
    const int64_t first = t * tile, offset = first * a.num_kv_heads * a.head_dim;
    p.slot_mapping = a.slot_mapping + first;
    p.k_out = static_cast<T *>(a.k_out) + offset;
    p.v_out = static_cast<T *>(a.v_out) + offset;
    p.num_tokens = static_cast<int32_t>(a.num_tokens - first);
    const int64_t y = tiles - t < kMaxTiles ? tiles - t : kMaxTiles;
    const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(a.num_kv_heads), static_cast<unsigned>(y)),
                                     dim3(kFp4Threads), 0, st, p, tile, err);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
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
  // tokens per CTA: up to 8, as many as leave two CTAs per SM (16384 tokens written
  // and read back: 23.8 us, 26.4 with four each)
  const int64_t per = wa.num_tokens / (2 * static_cast<int64_t>(device_sm_count()));
  a.tile_log2 = per >= 8 ? 3 : per >= 4 ? 2 : per >= 2 ? 1 : 0;
  return in_dt == PHOTON_BF16 ? launch_write<BF16Tag>(a, err, st) : launch_write<F32Tag>(a, err, st);
}

cudaError_t launch_kv_cache_read_fp4(const CacheReadArgs &a, photon_dtype out_dt, unsigned int *err,
                                     cudaStream_t st) {
  if (a.num_tokens == 0) return cudaSuccess;
  return out_dt == PHOTON_BF16 ? launch_read<BF16Tag>(a, err, st) : launch_read<F32Tag>(a, err, st);
}

}  // namespace photon
