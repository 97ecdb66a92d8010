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
// comes off exactly as well; the rest, at most an eighth of a turn, goes through
// sincospif from its leading 32 bits: |error| <= 2^-29 of the angle's radians
// plus the function's two units in the last place, 2^-23 absolute.
#pragma once

#include "row_lanes.cuh"

namespace photon {

constexpr int kNormThreads = 256;
constexpr int kNormMaxTile = 8;    // tokens of a CTA
constexpr int kNormDivBits = 28;   // row / heads = row * div >> 28

// A token's (cos, sin) in the order its lanes read them: step i of lane w at
// i * LPR + w.  Rows are padded by LPR entries: neighbouring rows of a table then
// start in different banks, where a warp's lanes read several tokens at once.
template <int D>
struct RopeRow {
  static constexpr int LPR = D / 16;  // lanes of a row
  static constexpr int HALF = D / 2;
  static constexpr int STRIDE = HALF + LPR;
  // step and lane of a pair: NEOX lane w takes pairs 8w .., GPT-J 4w .. of either half
  __device__ __forceinline__ static int at(int pair, bool gptj) {
    return gptj ? (pair / (D / 4) * 4 + pair % 4) * LPR + pair % (D / 4) / 4 : pair % 8 * LPR + pair / 8;
  }
};

// (cos, sin) of the fraction turn / 2^64 of a turn.
__device__ __forceinline__ float2 cos_sin_of_turn(unsigned long long turn) {
  const unsigned up = static_cast<unsigned>(turn >> 32) + 0x20000000u;  // nearest quarter: the top two bits
  const int rest = static_cast<int>(up & 0x3fffffffu) - 0x20000000;     // 2^-32 turn, |rest| <= 2^29
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
  const unsigned quarter = up >> 30;
  float2 r = (quarter & 1u) ? make_float2(-s, c) : make_float2(c, s);
  if (quarter & 2u) r = make_float2(-r.x, -r.y);
  return r;
}

// Table rows 0 .. n - 1 of the positions pos[0 .. n - 1], by all threads of the CTA.
template <int D>
__device__ __forceinline__ void rope_table_rows(float2 (*cs)[RopeRow<D>::STRIDE], const int32_t *pos, int n,
                                                const unsigned long long *turns, bool gptj, int threads) {
  using R = RopeRow<D>;
  for (int i = threadIdx.x; i < n * R::HALF; i += threads) {
    const int t = i / R::HALF, pair = i % R::HALF;
    cs[t][R::at(pair, gptj)] =
        cos_sin_of_turn(static_cast<unsigned long long>(static_cast<long long>(pos[t])) * turns[pair]);
  }
}

// Rotates a lane's 8 pairs.  NEOX: (x0[i], x1[i]); GPT-J: (x0[2i], x0[2i + 1]),
// then those of x1.  cs: the lane's first entry of its token's table row.
template <bool GPTJ>
__device__ __forceinline__ void rotate_pairs(float (&x0)[8], float (&x1)[8], const float2 *cs, int stride) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float &u = GPTJ ? (i < 4 ? x0[2 * i] : x1[2 * i - 8]) : x0[i];
    float &w = GPTJ ? (i < 4 ? x0[2 * i + 1] : x1[2 * i - 7]) : x1[i];
    const float2 p = cs[i * stride];
    const float a = u, b = w;
    u = fmaf(a, p.x, -(b * p.y));
    w = fmaf(b, p.x, a * p.y);
  }
}

// The lane's weights of a norm, as fp32.
template <typename T>
__device__ __forceinline__ void load_weights(const void *weight, int w, int half, float (&w0)[8], float (&w1)[8]) {
  RowLoad<T> r;
  r.load(static_cast<const T *>(weight) + 8 * w, half);
  RowLoad<T>::widen(r.lo, w0);
  RowLoad<T>::widen(r.hi, w1);
}

// x * w / sqrt(mean square + eps) of a row of D values; all lanes of the warp take part.
template <int D>
__device__ __forceinline__ void rms_norm_lane(float (&x0)[8], float (&x1)[8], const float (&w0)[8],
                                              const float (&w1)[8], float eps) {
  float a = 0.f, b = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a = fmaf(x0[i], x0[i], a);
    b = fmaf(x1[i], x1[i], b);
  }
  a += b;
#pragma unroll
  for (int o = RopeRow<D>::LPR / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  const float inv = rsqrtf(fmaf(a, 1.f / D, eps));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x0[i] *= inv * w0[i];
    x1[i] *= inv * w1[i];
  }
}

// One tile of query rows, [tokens][heads][D] contiguous: normalised and rotated
// in place, neighbouring rows of a token by neighbouring lanes.
template <typename Tag, int D>
__device__ __forceinline__ void norm_rope_q_tile(const NormRopeArgs &a, int tile, float2 (*cs)[RopeRow<D>::STRIDE]) {
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
  float w0[8], w1[8];
  load_weights<T>(a.q_weight, w, R::HALF, w0, w1);
  if (rotate) rope_table_rows<D>(cs, a.q_positions + t0, n, a.turns, gptj, kNormThreads);
  __syncthreads();
  for (int r0 = 0; r0 < rows; r0 += STEP) {  // lanes past the last row repeat it, for the shuffles
    const int r = min(r0 + first, rows - 1);
    float x0[8], x1[8];
    RowLoad<T>::widen(next.lo, x0);
    RowLoad<T>::widen(next.hi, x1);
    if (r0 + STEP < rows) next.load(base + min(r0 + STEP + first, rows - 1) * D, R::HALF);
    rms_norm_lane<D>(x0, x1, w0, w1, a.eps);
    if (rotate) {
      const float2 *row = cs[static_cast<uint32_t>(r) * a.q_div >> kNormDivBits] + w;
      if (gptj)
        rotate_pairs<true>(x0, x1, row, R::LPR);
      else
        rotate_pairs<false>(x0, x1, row, R::LPR);
    }
    if (r0 + first < rows) {
      store8(base + r * D, x0);
      store8(base + r * D + R::HALF, x1);
    }
  }
}

}  // namespace photon
