// q/k RMS norms, rotation and the paged write in one launch (bf16 / fp32 caches,
// sm_103a).  Qwen3-type models normalise every head of q and k between the
// projection and the rotation: done apart, that is a pass over q and k through
// memory and a launch more.
//
//   q[i][g]   <- R(q * w_q / rms(q))           in place
//   k_cache   <- R(k * w_k / rms(k)), v_cache <- v    at slot_mapping
//
// One CTA per tile of up to 8 tokens with all their heads: the tile's (cos, sin)
// table in shared memory is made once for all heads, the first rows are on the
// way meanwhile, and rows of a token are contiguous, so a warp's loads are whole
// lines.  Query tiles and key/value tiles are CTAs of one grid.
#include "norm_rope.cuh"

namespace photon {
namespace {

template <typename Tag, int D>
__global__ void __launch_bounds__(kNormThreads, D < 256 && sizeof(typename Tag::T) == 2 ? 4 : 2)
    qk_norm_rope_write_kernel(const __grid_constant__ NormRopeArgs a, unsigned int *err) {
  using T = typename Tag::T;
  using R = RopeRow<D>;
  constexpr int STEP = kNormThreads / R::LPR;
  __shared__ __align__(16) float cs[kNormMaxTile][R::STRIDE];
  __shared__ int64_t slots[kNormMaxTile];
  pdl_wait();
  pdl_launch_dependents();
  if (static_cast<int>(blockIdx.x) < a.q_tiles) {
    norm_rope_q_tile<Tag, D>(a, blockIdx.x, cs);
    return;
  }
  const int H = a.num_kv_heads;
  const int t0 = (blockIdx.x - a.q_tiles) << a.tile_log2, n = min(1 << a.tile_log2, a.num_tokens - t0);
  const int keys = n * H, rows = 2 * keys;  // the tile's K rows, then its V rows
  const int w = threadIdx.x % R::LPR, first = threadIdx.x / R::LPR;
  const bool rotate = a.rope_style != PHOTON_ROPE_NONE, gptj = a.rope_style == PHOTON_ROPE_GPTJ;
  const int64_t tile_at = static_cast<int64_t>(t0) * H * D + 8 * w;
  const T *k = static_cast<const T *>(a.k) + tile_at, *v = static_cast<const T *>(a.v) + tile_at;
  auto source = [&](int r) { return r < keys ? k + r * D : v + (min(r, rows - 1) - keys) * D; };
  RowLoad<T> next;
  next.load(source(first), R::HALF);
  LaneRow weight;
  load_weights<T>(a.k_weight, w, R::HALF, weight);
  if (static_cast<int>(threadIdx.x) < n) {
    const int64_t slot = a.slot_mapping[t0 + threadIdx.x];
    if (slot >= a.num_slots) atomicOr(err, PHOTON_DEVERR_SLOT_RANGE);
    slots[threadIdx.x] = slot < a.num_slots ? slot : -1;
  }
  if (rotate) rope_table_rows<D>(cs, n, a.turns, gptj, [&](int t) { return a.positions[t0 + t]; });
  __syncthreads();
  for (int r0 = 0; r0 < rows; r0 += STEP) {
    const int r = min(r0 + first, rows - 1);
    const RowLoad<T> raw = next;
    if (r0 + STEP < rows) next.load(source(r0 + STEP + first), R::HALF);
    const bool key = r < keys;
    const int rr = key ? r : r - keys;
    const int t = static_cast<uint32_t>(rr) * a.kv_div >> kNormDivBits, h = rr - t * H;
    const int64_t slot = slots[t];
    const bool live = r0 + first < rows && slot >= 0;
    T *dst = static_cast<T *>(key ? a.k_cache : a.v_cache) +
             (((slot >> 4) * H + h) * kBlockSize + (slot & (kBlockSize - 1))) * D + 8 * w;
    if (__any_sync(0xffffffffu, key)) {
      LaneRow x;
      widen_row(raw, x);
      norm_rope_row<D>(x, weight, a.eps, rotate ? cs[t] : nullptr, w, gptj);
      if (live && key) store_row(dst, R::HALF, x);
    }
    if (live && !key) raw.store(dst, R::HALF);
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
