// q/k RMS norms, rotation and the paged write in one launch (bf16 / fp32 caches,
// sm_103a).  Qwen3-type models normalise every head of q and k between the
// projection and the rotation: done apart, that is a pass over q and k through
// memory and a launch more.
//
//   q[i][g]   <- R(q * w_q / rms(q))           in place
//   k_cache   <- R(k * w_k / rms(k)), v_cache <- v    at slot_mapping
//
// A warp takes one token's heads in turn (of few tokens, several warps share one), over
// a (cos, sin) row of its own, its next rows on their way; rows of a token are
// contiguous, so a warp's loads are whole lines, and no warp waits for another.
//
// What bounds it: loads in flight, so warps per SM.  8192 tokens with 32 query and 8
// KV heads of 64, bf16, 101 MB: 18.4 us, 0.81 of the copy rate (65536 tokens 128 us, 0.93;
// 64 tokens of 16 / 8 heads of 128 2.3 us, latency).  The bf16 kernels of d 32, 64 and 128 hold 64
// registers and spill 16 bytes for those 32 warps per SM.  With one table and a barrier for a CTA's 8
// tokens 19.5; the table row in registers, 24 warps per SM instead of 32, 19.9; two rows
// ahead 20.1; 40 warps, which spill more, 25.9.
// Of middle-sized chunks with few heads most warps have no work: a token is split over up to
// 8 warps whatever its heads, and lanes past the last head repeat it (777 fp32 tokens of 4 / 4
// heads of 128 5.0 us for a floor of 1.4, 9 % of the warps active; 16384 tokens of 2 / 1 heads of 64
// 15.0 us, of 8 / 4 17.1).
#include "norm_rope.cuh"

namespace photon {
namespace {

template <typename Tag, int D>
__global__ void __launch_bounds__(kNormThreads, D < 256 && sizeof(typename Tag::T) == 2 ? 4 : 2)
    qk_norm_rope_write_kernel(const __grid_constant__ NormRopeArgs a, unsigned int *err) {
  using T = typename Tag::T;
  using R = RopeRow<D>;
  constexpr int RPP = 32 / R::LPR;
  __shared__ __align__(16) float scratch[kNormThreads / 32][R::STRIDE];
  pdl_wait();
  pdl_launch_dependents();
  if (static_cast<int>(blockIdx.x) < a.q_tiles) {
    norm_rope_q_tile<Tag, D>(a, blockIdx.x, scratch);
    return;
  }
  const TokenShare mine(blockIdx.x - a.q_tiles, a.tile_log2, a.num_tokens);
  if (mine.token < 0) return;
  const int lane = threadIdx.x & 31, w = lane % R::LPR, H = a.num_kv_heads;
  const bool rotate = a.rope_style != PHOTON_ROPE_NONE, gptj = a.rope_style == PHOTON_ROPE_GPTJ;
  const int groups = (H + RPP - 1) / RPP;  // units: K of the groups of heads, then V
  const int64_t at = mine.token * H * D + 8 * w;
  const T *k = static_cast<const T *>(a.k) + at, *v = static_cast<const T *>(a.v) + at;
  auto head = [&](int u) { return (u < groups ? u : u - groups) * RPP + lane / R::LPR; };
  auto source = [&](int u) { return (u < groups ? k : v) + static_cast<int64_t>(min(head(u), H - 1)) * D; };
  if (mine.part >= 2 * groups) return;
  RowLoad<T> next;
  next.load(source(mine.part), R::HALF);
  const int64_t slot = a.slot_mapping[mine.token];
  const RowLoad<T> weight = load_weights<T>(a.k_weight, w, R::HALF);
  const RowAt<D> turns{scratch[threadIdx.x >> 5], w};
  if (rotate && mine.part < groups)
    token_turns<D>(scratch[threadIdx.x >> 5], a.positions[mine.token], a.turns, gptj);
  if (slot < 0 || slot >= a.num_slots) {
    if (slot >= a.num_slots && mine.part == 0 && lane == 0) atomicOr(err, PHOTON_DEVERR_SLOT_RANGE);
    return;
  }
  const int64_t first = ((slot >> 4) * H * kBlockSize + (slot & (kBlockSize - 1))) * D + 8 * w;  // head 0
  T *kd = static_cast<T *>(a.k_cache) + first, *vd = static_cast<T *>(a.v_cache) + first;
  for (int u = mine.part; u < 2 * groups; u += mine.parts) {
    const RowLoad<T> raw = next;
    if (u + mine.parts < 2 * groups) next.load(source(u + mine.parts), R::HALF);
    const int h = head(u);
    if (u < groups) {
      LaneRow x;
      widen_row(raw, x);
      norm_rope_row<T, D>(x, weight, a.eps, rotate, turns, gptj);
      if (h < H) store_row(kd + static_cast<int64_t>(h) * kBlockSize * D, R::HALF, x);
    } else if (h < H) {
      raw.store(vd + static_cast<int64_t>(h) * kBlockSize * D, R::HALF);
    }
  }
}

template <typename Tag>
cudaError_t launch(const NormRopeArgs &a, int head_dim, int64_t ctas, unsigned int *err, cudaStream_t st) {
  auto kern = head_dim == 32    ? qk_norm_rope_write_kernel<Tag, 32>
              : head_dim == 64  ? qk_norm_rope_write_kernel<Tag, 64>
              : head_dim == 128 ? qk_norm_rope_write_kernel<Tag, 128>
                                : qk_norm_rope_write_kernel<Tag, 256>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kNormThreads), 0, st, a, err);
}

}  // namespace

int norm_tile_log2(int64_t tokens, int most) {
  const int64_t per = tokens / (2 * static_cast<int64_t>(device_sm_count()));
  int t = 0;
  while (t < most && (int64_t{2} << t) <= per) ++t;
  return t;
}

cudaError_t launch_qk_norm_rope_write(NormRopeArgs a, photon_dtype dt, int head_dim, unsigned int *err,
                                      cudaStream_t st) {
  a.q_tile_log2 = norm_tile_log2(a.num_q_tokens, 3);
  a.tile_log2 = norm_tile_log2(a.num_tokens, 3);
  a.q_tiles = static_cast<int>((static_cast<int64_t>(a.num_q_tokens) + (1 << a.q_tile_log2) - 1) >> a.q_tile_log2);
  const int64_t ctas = a.q_tiles + ((static_cast<int64_t>(a.num_tokens) + (1 << a.tile_log2) - 1) >> a.tile_log2);
  if (ctas == 0) return cudaSuccess;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  return dt == PHOTON_BF16 ? launch<BF16Tag>(a, head_dim, ctas, err, st) : launch<F32Tag>(a, head_dim, ctas, err, st);
}

}  // namespace photon
