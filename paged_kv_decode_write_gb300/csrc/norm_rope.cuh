// RMS norms of query and key rows with the rotation in the same pass: what the
// q/k-norm writes (bf16 / fp32 caches and the 8-bit cache) share.
//
//   y = R_pos(x * w / sqrt(mean_e x_e^2 + eps))
//
// A row lies in D / 16 neighbouring lanes (row_lanes.cuh), so its mean square is
// a sum of 16 squares per lane and log2(D / 16) shuffles, and both halves of a
// rotation pair are in one lane.  Everything is fp32 with one rounding to the
// storage type at the end.
//
// Angles are 64-bit fractions of a turn: pos * F mod 2^64, F = 2^64 theta^(-2i/d)
// / 2 pi rounded, is reduced exactly by the integer wrap, so far positions lose
// nothing (F carries an fp64 frequency's 53 bits).  The nearest quarter turn
// comes off exactly as well; the rest, at most an eighth of a turn, is taken from its
// leading 32 bits (2^-29 radians) to the Taylor series of sine and cosine at 0, whose
// terms past x^9 and x^10 are below 2^-29 there: with the roundings within 2^-23.
#pragma once

#include "row_lanes.cuh"

namespace photon {

constexpr int kNormThreads = 256;
constexpr int kNormMaxTile = 8;    // tokens of a CTA
constexpr int kNormDivBits = 28;   // row / heads = row * div >> 28

// A lane's 16 values of a row, as pairs of neighbouring dims for the packed fp32
// instructions (two elements each): a: dims 8w .. 8w + 7, b: those + D/2.
struct LaneRow {
  float2 a[4], b[4];
};

template <typename T>
__device__ __forceinline__ void widen_row(const RowLoad<T> &r, LaneRow &x) {
  float f[8];
  RowLoad<T>::widen(r.lo, f);
#pragma unroll
  for (int j = 0; j < 4; ++j) x.a[j] = make_float2(f[2 * j], f[2 * j + 1]);
  RowLoad<T>::widen(r.hi, f);
#pragma unroll
  for (int j = 0; j < 4; ++j) x.b[j] = make_float2(f[2 * j], f[2 * j + 1]);
}

// To the storage type, one rounding each; dst: the lane's dims 8w.
template <typename T>
__device__ __forceinline__ void store_row(T *dst, int half, const LaneRow &x) {
  const float lo[8] = {x.a[0].x, x.a[0].y, x.a[1].x, x.a[1].y, x.a[2].x, x.a[2].y, x.a[3].x, x.a[3].y};
  const float hi[8] = {x.b[0].x, x.b[0].y, x.b[1].x, x.b[1].y, x.b[2].x, x.b[2].y, x.b[3].x, x.b[3].y};
  store8(dst, lo);
  store8(dst + half, hi);
}

// A token's rotations in the order its lanes read them: step j of lane w, two
// pairs, is the chunk (cos, cos, sin, sin) at 4 (j LPR + w) floats.  At D = 64 rows
// are padded so that two tokens read by one quarter of a warp meet no bank twice.
template <int D>
struct RopeRow {
  static constexpr int LPR = D / 16;  // lanes of a row
  static constexpr int HALF = D / 2;
  static constexpr int STRIDE = 2 * HALF + (D == 64 ? 16 : 0);
  // Where a pair's cosine lies (its sine 2 further).  NEOX lane w takes pairs
  // 8w .. 8w + 7 in order; GPT-J 4w .. 4w + 3, then those + D/4.
  __device__ __forceinline__ static int at(int pair, bool gptj) {
    const int p = pair % (D / 4);
    const int lane = gptj ? p / 4 : pair / 8, i = gptj ? pair / (D / 4) * 4 + p % 4 : pair % 8;
    return 4 * (i / 2 * LPR + lane) + i % 2;
  }
};

// (cos, sin) of a fraction of a turn, in units of 2^-32.
__device__ __forceinline__ float2 cos_sin_of_turn(unsigned turn) {
  const unsigned up = turn + 0x20000000u;                            // nearest quarter: the top two bits
  const int rest = static_cast<int>(up & 0x3fffffffu) - 0x20000000;  // |rest| <= 2^29
  const float x = static_cast<float>(rest) * static_cast<float>(6.283185307179586476925286766559 * 0x1p-32);
  const float x2 = x * x;
  float s = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
  s = fmaf(x2, s, 1.f / 120.f);
  s = fmaf(x2, s, -1.f / 6.f);
  s = fmaf(x * x2, s, x);
  float c = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
  c = fmaf(x2, c, -1.f / 720.f);
  c = fmaf(x2, c, 1.f / 24.f);
  c = fmaf(x2, c, -0.5f);
  c = fmaf(x2, c, 1.f);
  // a quarter turn on: (c, s) -> (-s, c)
  const bool odd = up & 0x40000000u;
  const unsigned flip = up & 0x80000000u;
  const float u = odd ? -s : c, v = odd ? c : s;
  return make_float2(__uint_as_float(__float_as_uint(u) ^ flip), __uint_as_float(__float_as_uint(v) ^ flip));
}

// The leading 32 bits of pos * turns mod 2^64.
__device__ __forceinline__ unsigned turn_of(int pos, unsigned long long turns) {
  const unsigned p = static_cast<unsigned>(pos);
  return __umulhi(p, static_cast<unsigned>(turns)) + p * static_cast<unsigned>(turns >> 32);
}

// Table rows 0 .. n - 1, by all threads of the CTA: a thread keeps its pair.
// position(t): that of row t, asked for by whole warps where D >= 64.
template <int D, typename Position>
__device__ __forceinline__ void rope_table_rows(float (*cs)[RopeRow<D>::STRIDE], int n,
                                                const unsigned long long *turns, bool gptj, Position position) {
  using R = RopeRow<D>;
  const int pair = threadIdx.x % R::HALF;
  const unsigned long long turn = turns[pair];
  const int at = R::at(pair, gptj);
#pragma unroll 1
  for (int t = threadIdx.x / R::HALF; t < n; t += kNormThreads / R::HALF) {
    const float2 v = cos_sin_of_turn(turn_of(position(t), turn));
    cs[t][at] = v.x;
    cs[t][at + 2] = v.y;
  }
}

// Rotates a lane's 8 pairs.  NEOX: (a, b) element by element; GPT-J: the
// neighbours of a, then of b.  cs: the token's table row.
template <int D>
__device__ __forceinline__ void rotate_row(LaneRow &x, const float *cs, int w, bool gptj) {
  using R = RopeRow<D>;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 t = *reinterpret_cast<const float4 *>(cs + 4 * (j * R::LPR + w));
    if (gptj) {
      float2 &p = j < 2 ? x.a[2 * j] : x.b[2 * j - 4], &q = j < 2 ? x.a[2 * j + 1] : x.b[2 * j - 3];
      p = make_float2(fmaf(p.x, t.x, -(p.y * t.z)), fmaf(p.y, t.x, p.x * t.z));
      q = make_float2(fmaf(q.x, t.y, -(q.y * t.w)), fmaf(q.y, t.y, q.x * t.w));
    } else {
      const float2 c = make_float2(t.x, t.y), s = make_float2(t.z, t.w), u = x.a[j], v = x.b[j];
      const float2 vs = __fmul2_rn(v, s);
      x.a[j] = __ffma2_rn(u, c, make_float2(-vs.x, -vs.y));
      x.b[j] = __ffma2_rn(v, c, __fmul2_rn(u, s));
    }
  }
}

// The lane's weights of a norm, as fp32.
template <typename T>
__device__ __forceinline__ void load_weights(const void *weight, int w, int half, LaneRow &out) {
  RowLoad<T> r;
  r.load(static_cast<const T *>(weight) + 8 * w, half);
  widen_row(r, out);
}

__device__ __forceinline__ void scale_row(LaneRow &x, const LaneRow &f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x.a[j] = __fmul2_rn(x.a[j], f.a[j]);
    x.b[j] = __fmul2_rn(x.b[j], f.b[j]);
  }
}
__device__ __forceinline__ void scale_row(LaneRow &x, float f) {
  const float2 ff = make_float2(f, f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x.a[j] = __fmul2_rn(x.a[j], ff);
    x.b[j] = __fmul2_rn(x.b[j], ff);
  }
}

// 1 / sqrt(mean square + eps) of a row of D values; all lanes of the warp take part.
template <int D>
__device__ __forceinline__ float inv_rms(const LaneRow &x, float eps) {
  float2 s = __fmul2_rn(x.a[0], x.a[0]), t = __fmul2_rn(x.b[0], x.b[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) {
    s = __ffma2_rn(x.a[j], x.a[j], s);
    t = __ffma2_rn(x.b[j], x.b[j], t);
  }
  s = __fadd2_rn(s, t);
  float a = s.x + s.y;
#pragma unroll
  for (int o = RopeRow<D>::LPR / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  return rsqrtf(fmaf(a, 1.f / D, eps));
}

// Norm and rotation of a row: the sum's shuffles run beside the rotation of x w,
// the factor comes last.  cs NULL: no rotation.
template <int D>
__device__ __forceinline__ void norm_rope_row(LaneRow &x, const LaneRow &weight, float eps, const float *cs, int w,
                                              bool gptj) {
  const float inv = inv_rms<D>(x, eps);
  scale_row(x, weight);
  if (cs) rotate_row<D>(x, cs, w, gptj);
  scale_row(x, inv);
}

// One tile of query rows, [tokens][heads][D] contiguous: normalised and rotated
// in place, neighbouring rows of a token by neighbouring lanes.
template <typename Tag, int D>
__device__ __forceinline__ void norm_rope_q_tile(const NormRopeArgs &a, int tile, float (*cs)[RopeRow<D>::STRIDE]) {
  using T = typename Tag::T;
  using R = RopeRow<D>;
  constexpr int STEP = kNormThreads / R::LPR;
  const int t0 = tile << a.q_tile_log2, n = min(1 << a.q_tile_log2, a.num_q_tokens - t0);
  const int rows = n * a.num_q_heads;
  const int w = threadIdx.x % R::LPR, first = threadIdx.x / R::LPR;
  const bool rotate = a.rope_style != PHOTON_ROPE_NONE, gptj = a.rope_style == PHOTON_ROPE_GPTJ;
  T *base = static_cast<T *>(a.q) + static_cast<int64_t>(t0) * a.num_q_heads * D + 8 * w;
  RowLoad<T> next;
  next.load(base + min(first, rows - 1) * D, R::HALF);
  LaneRow weight;
  load_weights<T>(a.q_weight, w, R::HALF, weight);
  if (rotate) rope_table_rows<D>(cs, n, a.turns, gptj, [&](int t) { return a.q_positions[t0 + t]; });
  __syncthreads();
  for (int r0 = 0; r0 < rows; r0 += STEP) {  // lanes past the last row repeat it, for the shuffles
    const int r = min(r0 + first, rows - 1);
    LaneRow x;
    widen_row(next, x);
    if (r0 + STEP < rows) next.load(base + min(r0 + STEP + first, rows - 1) * D, R::HALF);
    norm_rope_row<D>(x, weight, a.eps, rotate ? cs[static_cast<uint32_t>(r) * a.q_div >> kNormDivBits] : nullptr, w,
                     gptj);
    if (r0 + first < rows) store_row(base + r * D, R::HALF, x);
  }
}

}  // namespace photon
