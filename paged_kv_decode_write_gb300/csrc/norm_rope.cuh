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
// / 2 pi cut to an integer, is reduced exactly by the integer wrap, so far positions lose
// nothing (F carries an fp64 frequency's 53 bits).  The nearest quarter turn
// comes off exactly as well; the rest, at most an eighth of a turn, is taken from its
// leading 32 bits (2^-29 radians) to the Taylor series of sine and cosine at 0, whose
// terms past x^9 and x^10 are below 2^-29 there: with the roundings within 2^-23.
#pragma once

#include "row_lanes.cuh"

namespace photon {

constexpr int kNormThreads = 256;

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

// The leading 32 bits of p * turns mod 2^64.
__device__ __forceinline__ unsigned turn_of(unsigned p, unsigned long long turns) {
  return __umulhi(p, static_cast<unsigned>(turns)) + p * static_cast<unsigned>(turns >> 32);
}
// The same of a position that may be negative (padding has -1): as unsigned it is 2^32 more.
__device__ __forceinline__ unsigned turn_of(int pos, unsigned long long turns) {
  return turn_of(static_cast<unsigned>(pos), turns) - (static_cast<unsigned>(pos >> 31) & static_cast<unsigned>(turns));
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

// Rotates a lane's 8 pairs, two per chunk of its token's row.  NEOX: (a, b) element by
// element; GPT-J: the neighbours of a, then of b.
__device__ __forceinline__ void rotate_chunk(LaneRow &x, int j, const float4 &t, bool gptj) {
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
// A lane's chunks of a token's row.
template <int D>
struct RowAt {
  const float *cs;
  int w;
  __device__ __forceinline__ float4 operator[](int j) const {
    return *reinterpret_cast<const float4 *>(cs + 4 * (j * RopeRow<D>::LPR + w));
  }
};
template <int D>
__device__ __forceinline__ void rotate_row(LaneRow &x, const RowAt<D> &row, bool gptj) {
#pragma unroll
  for (int j = 0; j < 4; ++j) rotate_chunk(x, j, row[j], gptj);
}

// The lane's weights of a norm.
template <typename T>
__device__ __forceinline__ RowLoad<T> load_weights(const void *weight, int w, int half) {
  RowLoad<T> r;
  r.load(static_cast<const T *>(weight) + 8 * w, half);
  return r;
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

// Norm and rotation (if asked for) of a row: the sum's shuffles run beside the
// rotation of x w, the factor comes last.  The weights stay as they were loaded: the
// registers of another fp32 row would cost a CTA per SM.
template <typename T, int D>
__device__ __forceinline__ void norm_rope_row(LaneRow &x, const RowLoad<T> &weight, float eps, bool rotate,
                                              const RowAt<D> &row, bool gptj) {
  const float inv = inv_rms<D>(x, eps);
  LaneRow f;
  widen_row(weight, f);
  scale_row(x, f);
  if (rotate) rotate_row(x, row, gptj);
  scale_row(x, inv);
}

// The table row of one token, by its warp; scratch: STRIDE floats of the warp's own.
template <int D>
__device__ __forceinline__ void token_turns(float *scratch, int pos, const unsigned long long *turns, bool gptj) {
  using R = RopeRow<D>;
  auto fill = [&](auto p) {
#pragma unroll 1
    for (int pair = threadIdx.x & 31; pair < R::HALF; pair += 32) {
      const float2 v = cos_sin_of_turn(turn_of(p, turns[pair]));
      float *at = scratch + R::at(pair, gptj);
      at[0] = v.x;
      at[2] = v.y;
    }
  };
  // negative positions again, in a loop of their own: one loop for both took 26.7 us for 22.8
  // (16384 tokens of 4 query and 2 KV heads of 128)
  fill(static_cast<unsigned>(pos));
  if (pos < 0) fill(pos);
  __syncwarp();
}

// A warp's share of a tile of tokens: of 8 tokens one each, of fewer a token's heads
// in turn between 8 / tokens warps, so that no warp waits for another.
struct TokenShare {
  int64_t token;  // -1: none
  int part, parts;
  __device__ __forceinline__ TokenShare(int tile, int tile_log2, int tokens) {
    const int warp = threadIdx.x >> 5, split = 3 - tile_log2;
    const int64_t t = (static_cast<int64_t>(tile) << tile_log2) + (warp >> split);
    token = t < tokens ? t : -1;
    part = warp & ((1 << split) - 1);
    parts = 1 << split;
  }
};

// One tile of query tokens: every head normalised and rotated in place, neighbouring
// heads of a token by neighbouring lanes, the next ones on their way.
template <typename Tag, int D>
__device__ __forceinline__ void norm_rope_q_tile(const NormRopeArgs &a, int tile, float (*scratch)[RopeRow<D>::STRIDE]) {
  using T = typename Tag::T;
  using R = RopeRow<D>;
  constexpr int RPP = 32 / R::LPR;  // rows of a warp
  const TokenShare mine(tile, a.q_tile_log2, a.num_q_tokens);
  if (mine.token < 0) return;
  const int lane = threadIdx.x & 31, w = lane % R::LPR, H = a.num_q_heads;
  const bool rotate = a.rope_style != PHOTON_ROPE_NONE, gptj = a.rope_style == PHOTON_ROPE_GPTJ;
  T *q = static_cast<T *>(a.q) + mine.token * H * D + 8 * w;
  // heads past the last repeat it, for the shuffles
  auto row = [&](int group) { return q + static_cast<int64_t>(min(group * RPP + lane / R::LPR, H - 1)) * D; };
  const int groups = (H + RPP - 1) / RPP;
  if (mine.part >= groups) return;
  RowLoad<T> next;
  next.load(row(mine.part), R::HALF);
  const RowLoad<T> weight = load_weights<T>(a.q_weight, w, R::HALF);
  const RowAt<D> turns{scratch[threadIdx.x >> 5], w};
  if (rotate) token_turns<D>(scratch[threadIdx.x >> 5], a.q_positions[mine.token], a.turns, gptj);
  for (int g = mine.part; g < groups; g += mine.parts) {
    LaneRow x;
    widen_row(next, x);
    if (g + mine.parts < groups) next.load(row(g + mine.parts), R::HALF);
    norm_rope_row<T, D>(x, weight, a.eps, rotate, turns, gptj);
    if (g * RPP + lane / R::LPR < H) store_row(row(g), R::HALF, x);
  }
}

}  // namespace photon
