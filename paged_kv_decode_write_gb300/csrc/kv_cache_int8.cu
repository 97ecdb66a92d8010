// 8-bit KV cache with one scale per block of 16 tokens and KV head: the write
// (rotation, with or without q/k norms) and the dequantising read (sm_103a).
// Record layout in int8.cuh.
//
// Write, per block, KV head and K or V.  y: the rows that the call writes to the
// block, m = max |y|, s the block's scale so far (0 when the call writes its
// first token: the block starts anew and its other rows become 0).
//   s' = s                             if fl(m / 127) <= s
//      = max(fl(m / 127), 2 s)         otherwise
//   r  = fl(1 / s')
//   new code = rne(y r),  kept code = rne(code fl(s r)) where the scale grew
// A product with a float rounds to the nearest integer exactly when it is added
// to 1.5 * 2^23 in one fma, so a code depends on nothing but y and the scale.
// Growing by two at least bounds what a kept value loses over all growths: half
// a step each, the steps doubling, less than one step of the last scale
// together.  (Growing to exactly m / 127 may round a row 15 times at nearly the
// same step.)
//
// What a block's tokens share is the scale, so the unit of work is a run: the
// tokens of one block, next to each other in the call.  A warp takes one run's K
// or V of one head: 16 rows by offset, 16 values per lane and row in registers, one
// reduction for m, then the codes, 8 bytes per store.  A CTA takes the runs that
// begin in its tile of tokens, all heads, over one (cos, sin) table.
#include <climits>
#include <cmath>

#include "int8.cuh"
#include "norm_rope.cuh"

namespace photon {
namespace {

constexpr int kInt8Warps = 8;
constexpr int kInt8MaxTile = 16;                       // tokens of a CTA
constexpr int kInt8TableRows = kInt8MaxTile + kBlockSize - 1;  // its last run may pass the tile's end
static_assert(32 * kInt8Warps == kNormThreads, "query tiles run in the same CTAs");

constexpr float kCodeMagic = 12582912.f + 128.f;  // fma(y, r, this): low byte = rne(y r) + 128

// Eight codes + 128, value i in byte i.
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float r) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(__fmaf_rn(y[i], r, kCodeMagic));
  const uint32_t lo = __byte_perm(b[0], b[1], 0x0040u), hi = __byte_perm(b[2], b[3], 0x0040u);
  const uint32_t lo2 = __byte_perm(b[4], b[5], 0x0040u), hi2 = __byte_perm(b[6], b[7], 0x0040u);
  return make_uint2(__byte_perm(lo, hi, 0x5410u), __byte_perm(lo2, hi2, 0x5410u));
}

// Eight stored bytes as codes (exact).
__device__ __forceinline__ void codes_to_f32(uint2 w, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __byte_perm(i < 4 ? w.x : w.y, 0x4b000000u, 0x7540u + (i & 3));
    x[i] = __uint_as_float(b) - (8388608.f + 128.f);
  }
}

// max |.| that keeps a NaN of any operand
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// One warp: K (which 0) or V (1) of one head of one run.  src: this lane's token
// of row lane (0 .. 15) as an index into the tile's tokens, -1: not written.
template <typename Tag, int D, bool NORM>
__device__ __forceinline__ void write_run(const NormRopeArgs &a, int t0, int src, uint32_t written, int64_t block,
                                          int h, int which, const float2 (*cs)[RopeRow<D>::STRIDE]) {
  using T = typename Tag::T;
  using R = RopeRow<D>;
  constexpr int RPP = 32 / R::LPR, PASSES = kBlockSize / RPP;  // rows of a pass
  const int lane = threadIdx.x & 31, w = lane % R::LPR, sub = lane / R::LPR;
  const int H = a.num_kv_heads;
  unsigned char *rec = static_cast<unsigned char *>(a.k_cache) + (block * H + h) * int8_record_bytes(D);
  const T *x = static_cast<const T *>(which ? a.v : a.k) + static_cast<int64_t>(h) * D + 8 * w;
  float *scale_at = reinterpret_cast<float *>(rec + int8_scale_byte(D, which));
  const bool anew = written & 1u;
  const float old = anew ? 0.f : *scale_at;
  RowLoad<T> raw[PASSES];
  int row_src[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    row_src[p] = __shfl_sync(0xffffffffu, src, p * RPP + sub);
#pragma unroll
    for (int i = 0; i < RowLoad<T>::N; ++i) raw[p].lo[i] = raw[p].hi[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row_src[p] >= 0) raw[p].load(x + static_cast<int64_t>(t0 + row_src[p]) * H * D, R::HALF);
  }
  float y0[PASSES][8], y1[PASSES][8], m = 0.f;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    RowLoad<T>::widen(raw[p].lo, y0[p]);
    RowLoad<T>::widen(raw[p].hi, y1[p]);
    if (!(written >> (p * RPP) & ((1u << RPP) - 1))) continue;  // no row of the pass is written: zeros
    if (!which) {
      if constexpr (NORM) {
        float w0[8], w1[8];
        load_weights<T>(a.k_weight, w, R::HALF, w0, w1);
        rms_norm_lane<D>(y0[p], y1[p], w0, w1, a.eps);
      }
      if (a.rope_style != PHOTON_ROPE_NONE) {
        const float2 *row = cs[max(row_src[p], 0)] + w;
        if (a.rope_style == PHOTON_ROPE_GPTJ)
          rotate_pairs<true>(y0[p], y1[p], row, R::LPR);
        else
          rotate_pairs<false>(y0[p], y1[p], row, R::LPR);
      }
    }
    if (row_src[p] >= 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max_abs3(m, y0[p][i], y1[p][i]);
    }
  }
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));  // a NaN's bits are the largest
  float want = __fdiv_rn(m, 127.f);
  if (want < kInt8Least) want = 0.f;
  const bool finite = m <= 3.4028234663852886e38f;
  const bool grows = finite && want > old;
  const float scale = !finite ? __uint_as_float(0x7fffffffu) : grows ? fmaxf(want, 2.f * old) : old;
  const float r = scale > 0.f ? __frcp_rn(scale) : 0.f;
  const float ratio = __fmul_rn(old, r);
  if (lane == 0) *scale_at = scale;
  const bool requant = grows && !anew && old > 0.f;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const uint32_t in_pass = written >> (p * RPP) & ((1u << RPP) - 1);
    if (!in_pass && !anew && !requant) continue;
    const int row = p * RPP + sub;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int e = 8 * w + half * R::HALF;
      uint2 *at = reinterpret_cast<uint2 *>(rec + (which ? int8_v_byte(D, row, e) : int8_k_byte(row, e)));
      if (row_src[p] >= 0) {
        *at = scale > 0.f ? codes8(half ? y1[p] : y0[p], r) : make_uint2(0x80808080u, 0x80808080u);
      } else if (anew) {
        *at = make_uint2(0x80808080u, 0x80808080u);
      } else if (requant) {
        float c[8];
        codes_to_f32(*at, c);
        *at = codes8(c, ratio);
      }
    }
  }
}

template <typename Tag, int D, bool NORM>
__global__ void __launch_bounds__(kNormThreads)
    kv_cache_write_int8_kernel(const __grid_constant__ NormRopeArgs a, unsigned int *err) {
  using R = RopeRow<D>;
  __shared__ float2 cs[kInt8TableRows][R::STRIDE];
  pdl_wait();
  pdl_launch_dependents();
  if constexpr (NORM) {
    if (static_cast<int>(blockIdx.x) < a.q_tiles) {
      norm_rope_q_tile<Tag, D>(a, blockIdx.x, cs);
      return;
    }
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = (blockIdx.x - (NORM ? a.q_tiles : 0)) << a.tile_log2, tile = 1 << a.tile_log2;
  // lane i looks at token t0 - 1 + i: a run's length is at most a block's 16, so
  // the runs that begin in a tile of 16 end within the warp's 32 tokens
  const int t = t0 - 1 + lane;
  int64_t slot = t >= 0 && t < a.num_tokens ? a.slot_mapping[t] : -1;
  if (slot >= a.num_slots) {
    if (warp == 0 && lane >= 1 && lane <= tile) atomicOr(err, PHOTON_DEVERR_SLOT_RANGE);
    slot = -1;
  }
  const bool live = slot >= 0;
  const int64_t block = slot >> 4;
  const int64_t before = __shfl_up_sync(0xffffffffu, block, 1);
  const bool same = lane > 0 && live && before == block;
  const uint32_t joined = __ballot_sync(0xffffffffu, same);
  uint32_t leaders = __ballot_sync(0xffffffffu, lane >= 1 && lane <= tile && live && !same);
  if (!leaders) return;  // the same in every warp
  // tokens that follow lane i in its run
  auto follow = [&](int i) { return i == 31 ? 0 : min(__ffs(~(joined >> (i + 1))) - 1, kBlockSize - 1); };
  if (a.rope_style != PHOTON_ROPE_NONE) {
    const int i0 = __ffs(leaders) - 1, i1 = 31 - __clz(leaders);
    const int n = i1 + follow(i1) + 1 - i0;
    rope_table_rows<D>(cs + (i0 - 1), a.positions + (t0 - 1 + i0), n, a.turns,
                       a.rope_style == PHOTON_ROPE_GPTJ, kNormThreads);
    __syncthreads();
  }
  const int H = a.num_kv_heads;
  while (leaders) {  // a run: its heads' K and V over the warps
    const int i = __ffs(leaders) - 1;
    leaders &= leaders - 1;
    const int len = 1 + follow(i);
    const int64_t b = __shfl_sync(0xffffffffu, block, i);
    int src = -1;  // row lane's token, the last of those with its slot
    uint32_t written = 0;
    for (int j = 0; j < len; ++j) {
      const int off = static_cast<int>(__shfl_sync(0xffffffffu, slot, i + j)) & (kBlockSize - 1);
      if (lane == off) src = i - 1 + j;
      written |= 1u << off;
    }
    for (int hv = warp; hv < 2 * H; hv += kInt8Warps)
      write_run<Tag, D, NORM>(a, t0, src, written, b, hv >> 1, hv & 1, cs);
  }
}

// ---- read --------------------------------------------------------------------------

// One CTA per (tile of consecutive tokens, KV head); a lane takes the same 8 dims
// of a token's K and V, so that the slot's arithmetic serves two words and a
// row's lanes write whole lines.
template <typename Tag, int D>
__global__ void __launch_bounds__(kNormThreads)
    kv_cache_read_int8_kernel(const CacheReadArgs a, int tile, unsigned int *err) {
  using T = typename Tag::T;
  constexpr int LANES = D / 8;  // of a token
  pdl_wait();
  pdl_launch_dependents();
  const int H = a.num_kv_heads, h = blockIdx.x;
  const int e = 8 * (threadIdx.x % LANES);
  const unsigned char *base = static_cast<const unsigned char *>(a.pool) + static_cast<int64_t>(h) * int8_record_bytes(D);
  const int64_t block_bytes = static_cast<int64_t>(H) * int8_record_bytes(D);
  const int64_t first = static_cast<int64_t>(blockIdx.y) * tile;
  const int left = static_cast<int>(min(static_cast<int64_t>(tile), a.num_tokens - first));
  const int64_t *slots = a.slot_mapping + first;
  const int64_t out_at = (first * H + h) * D + e;
  T *k_out = static_cast<T *>(a.k_out) + out_at, *v_out = static_cast<T *>(a.v_out) + out_at;
  for (int t = threadIdx.x / LANES; t < left; t += kNormThreads / LANES) {
    const int64_t slot = slots[t];
    if (static_cast<uint64_t>(slot) >= static_cast<uint64_t>(a.num_slots)) {
      if (slot >= 0) atomicOr(err, PHOTON_DEVERR_SLOT_RANGE);
      continue;
    }
    const unsigned char *rec = base + (slot >> 4) * block_bytes;
    const int r = static_cast<int>(slot) & (kBlockSize - 1);
    const uint2 code[2] = {*reinterpret_cast<const uint2 *>(rec + int8_k_byte(r, e)),
                           *reinterpret_cast<const uint2 *>(rec + int8_v_byte(D, r, e))};
    const float2 scale = *reinterpret_cast<const float2 *>(rec + int8_scale_byte(D, 0));
    const int64_t row = static_cast<int64_t>(t) * H * D;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      float x[8];
      codes_to_f32(code[v], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= v ? scale.y : scale.x;
      store8((v ? v_out : k_out) + row, x);
    }
  }
}

template <typename Tag>
cudaError_t launch_read(const CacheReadArgs &a, unsigned int *err, cudaStream_t st) {
  using T = typename Tag::T;
  // 64 tokens per CTA where that leaves eight CTAs per SM, else 16
  const int64_t ctas = (static_cast<int64_t>(a.num_tokens) + 63) / 64 * a.num_kv_heads;
  const int tile = ctas >= 8 * static_cast<int64_t>(device_sm_count()) ? 64 : 16;
  const int64_t tiles = (static_cast<int64_t>(a.num_tokens) + tile - 1) / tile;
  auto kern = a.head_dim == 64 ? kv_cache_read_int8_kernel<Tag, 64> : kv_cache_read_int8_kernel<Tag, 128>;
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
                                     dim3(kNormThreads), 0, st, p, tile, err);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename Tag, int D>
cudaError_t launch_write(const NormRopeArgs &a, bool norm, int64_t ctas, unsigned int *err, cudaStream_t st) {
  auto kern = norm ? kv_cache_write_int8_kernel<Tag, D, true> : kv_cache_write_int8_kernel<Tag, D, false>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kNormThreads), 0, st, a, err);
}

}  // namespace

cudaError_t launch_kv_cache_write_int8(NormRopeArgs a, bool norm, photon_dtype in_dt, int head_dim,
                                       unsigned int *err, cudaStream_t st) {
  a.q_tile_log2 = norm_tile_log2(a.num_q_tokens, 3);
  a.tile_log2 = norm_tile_log2(a.num_tokens, 4);
  a.q_tiles = static_cast<int>((static_cast<int64_t>(a.num_q_tokens) + (1 << a.q_tile_log2) - 1) >> a.q_tile_log2);
  const int64_t ctas = a.q_tiles + ((static_cast<int64_t>(a.num_tokens) + (1 << a.tile_log2) - 1) >> a.tile_log2);
  if (ctas == 0) return cudaSuccess;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  if (head_dim == 64)
    return in_dt == PHOTON_BF16 ? launch_write<BF16Tag, 64>(a, norm, ctas, err, st)
                                : launch_write<F32Tag, 64>(a, norm, ctas, err, st);
  return in_dt == PHOTON_BF16 ? launch_write<BF16Tag, 128>(a, norm, ctas, err, st)
                              : launch_write<F32Tag, 128>(a, norm, ctas, err, st);
}

cudaError_t launch_kv_cache_read_int8(const CacheReadArgs &a, photon_dtype out_dt, unsigned int *err,
                                      cudaStream_t st) {
  if (a.num_tokens == 0) return cudaSuccess;
  return out_dt == PHOTON_BF16 ? launch_read<BF16Tag>(a, err, st) : launch_read<F32Tag>(a, err, st);
}

}  // namespace photon
