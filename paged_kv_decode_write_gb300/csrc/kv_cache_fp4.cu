// 4-bit (E2M1) KV cache: the RoPE-fused quantising write and the dequantising
// read (sm_103a).  Record layout in fp4.cuh.
//
// Write, per token and KV head: y = the row, K rotated and rounded once to the
// input type (what a cache of that type would hold); per 64 dims the scale
// s = bf16(max|y| / 6) and the codes round(y / s), to nearest with halves to
// the even code.  Read: code * s rounded to the output type.
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "rope.cuh"

namespace photon {
namespace {

constexpr int kFp4Threads = 128;

// max that keeps a NaN of either operand
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Code of x / s from exact comparisons: a midpoint of two E2M1 values has at
// most three significant bits and s eight, so their product is exact in fp32.
__device__ __noinline__ uint32_t e2m1_exact(float x, float s) {
  const float m = fabsf(x);
  const uint32_t c = (m > 0.25f * s) + (m >= 0.75f * s) + (m > 1.25f * s) + (m >= 1.75f * s) +
                     (m > 2.5f * s) + (m >= 3.5f * s) + (m > 5.f * s);
  return c | (x < 0.f ? 8u : 0u);
}

// Nearest E2M1 code of the exact quotient x / s (s > 0), halves to the even
// code.  y = fl(x * fl(1/s)) is within 2^-22 |y| of it; when y - e and y + e
// with twice that margin give the same code, so does the quotient (rounding is
// monotonic), else the exact comparisons decide (quotients next to a midpoint).
__device__ __forceinline__ uint32_t e2m1_code(float x, float s, float is) {
  const float y = x * is;
  const float e = fabsf(y) * 0x1p-21f;
  const uint32_t b = cvt_e2m1x2(y - e, y + e);
  if ((b & 15u) == (b >> 4)) return b & 15u;
  return e2m1_exact(x, s);
}

// Scale of a group whose largest magnitude is m (bf16 bits); a group that
// holds an infinity or a NaN gets a NaN scale.
__device__ __forceinline__ uint32_t group_scale(float m) {
  if (!(m <= 3.4028234663852886e38f)) return 0x7fffu;
  return __bfloat16_as_ushort(__float2bfloat16_rn(__fdiv_rn(m, 6.f)));
}

// Codes of two neighbouring dims.
__device__ __forceinline__ uint32_t quant_pair(float x0, float x1, uint32_t sbits) {
  const float s = bf16_bits_to_f32(sbits);
  if (!(s > 0.f)) return 0u;  // all-zero (or non-finite) group
  if (s < 0x1p-100f) return e2m1_exact(x0, s) | (e2m1_exact(x1, s) << 4);  // 1/s may overflow
  const float is = __frcp_rn(s);
  return e2m1_code(x0, s, is) | (e2m1_code(x1, s, is) << 4);
}

// One CTA per token; warps take KV heads in turn.  Lane i of a row's D/4
// lanes holds dims 2i, 2i + 1, 2i + D/2, 2i + D/2 + 1, so both halves of a
// rotation pair (either style) and whole code bytes stay in the lane.  At
// D = 64 lanes 0-15 take K and 16-31 V; at D = 128 the warp takes K, then V.
template <typename Tag, int D>
__global__ void __launch_bounds__(kFp4Threads)
    kv_cache_write_fp4_kernel(const __grid_constant__ WriteArgs a, unsigned int *err) {
  using T = typename Tag::T;
  __shared__ double cs[D / 2][2];
  __shared__ float cs32[D / 2][2];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = blockIdx.x;
  const int H = a.num_kv_heads;
  const bool rotate = a.rope_style != PHOTON_ROPE_NONE;
  const bool gptj = a.rope_style == PHOTON_ROPE_GPTJ;
  const int64_t slot = a.slot_mapping[t];
  if (slot < 0 || slot >= a.num_slots) {
    if (slot >= a.num_slots && threadIdx.x == 0) atomicOr(err, PHOTON_DEVERR_SLOT_RANGE);
    return;
  }
  if (rotate) {
    rope_table<kFp4Threads>(a, a.positions[t], cs, cs32);
    __syncthreads();
  }
  const int64_t blk = slot / kBlockSize;
  const int r = static_cast<int>(slot - blk * kBlockSize);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int RL = D / 4;             // lanes of a row
  constexpr int ROWS = 32 / RL;         // rows a warp handles at once
  const int i = lane % RL;
  for (int h = warp; h < H; h += kFp4Threads / 32) {
    unsigned char *rec = static_cast<unsigned char *>(a.k_cache) + (blk * H + h) * fp4_record_bytes(D);
#pragma unroll
    for (int kv = 0; kv < 2; kv += ROWS) {
      const int v = kv + lane / RL;  // 0: K, 1: V
      const T *src = static_cast<const T *>(v ? a.v : a.k) + (t * H + h) * D + 2 * i;
      T y[4] = {src[0], src[1], src[D / 2], src[D / 2 + 1]};
      if (rotate && v == 0) {
        const float x0 = to_f32(y[0]), x1 = to_f32(y[1]), x2 = to_f32(y[2]), x3 = to_f32(y[3]);
        if (gptj) {  // pairs (2i, 2i + 1): pair i, and D/4 + i in the upper half
          const int p = i, q = i + D / 4;
          y[0] = Rotate<Tag>::run(x0, x1, cs32[p][0], -cs32[p][1], cs, p, true);
          y[1] = Rotate<Tag>::run(x1, x0, cs32[p][0], cs32[p][1], cs, p, false);
          y[2] = Rotate<Tag>::run(x2, x3, cs32[q][0], -cs32[q][1], cs, q, true);
          y[3] = Rotate<Tag>::run(x3, x2, cs32[q][0], cs32[q][1], cs, q, false);
        } else {     // pairs (e, e + D/2)
          const int p = 2 * i, q = 2 * i + 1;
          y[0] = Rotate<Tag>::run(x0, x2, cs32[p][0], -cs32[p][1], cs, p, true);
          y[2] = Rotate<Tag>::run(x2, x0, cs32[p][0], cs32[p][1], cs, p, false);
          y[1] = Rotate<Tag>::run(x1, x3, cs32[q][0], -cs32[q][1], cs, q, true);
          y[3] = Rotate<Tag>::run(x3, x1, cs32[q][0], cs32[q][1], cs, q, false);
        }
      }
      const float f0 = to_f32(y[0]), f1 = to_f32(y[1]), f2 = to_f32(y[2]), f3 = to_f32(y[3]);
      // the groups of dims 0-63 (m0) and, at D = 128, 64-127 (m1)
      float m0 = max_nan(fabsf(f0), fabsf(f1)), m1 = max_nan(fabsf(f2), fabsf(f3));
      if (D == 64) m0 = max_nan(m0, m1);
#pragma unroll
      for (int o = RL / 2; o > 0; o >>= 1) {
        m0 = max_nan(m0, __shfl_xor_sync(0xffffffffu, m0, o));
        if (D > 64) m1 = max_nan(m1, __shfl_xor_sync(0xffffffffu, m1, o));
      }
      const uint32_t s0 = group_scale(m0), s1 = D > 64 ? group_scale(m1) : s0;
      const int e0 = 2 * i, e1 = 2 * i + D / 2;
      const int b0 = v ? fp4_v_byte(D, r, e0) : fp4_k_byte(r, e0);
      const int b1 = v ? fp4_v_byte(D, r, e1) : fp4_k_byte(r, e1);
      rec[b0] = static_cast<unsigned char>(quant_pair(f0, f1, s0));
      rec[b1] = static_cast<unsigned char>(quant_pair(f2, f3, s1));
      if (i < D / kFp4Group)
        *reinterpret_cast<uint16_t *>(rec + fp4_scale_byte(D, r, i, v)) =
            static_cast<uint16_t>(i ? s1 : s0);
    }
  }
}

__device__ __forceinline__ void store2(float *p, float a, float b) {
  *reinterpret_cast<float2 *>(p) = make_float2(a, b);
}
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
}

__device__ __forceinline__ float2 e2m1_pair(unsigned char b) {
  const uint32_t h = e2m1x2_to_f16(b);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// One warp per (token, KV head); lanes as in the write.
template <typename Tag, int D>
__global__ void __launch_bounds__(kFp4Threads)
    kv_cache_read_fp4_kernel(const unsigned char *__restrict__ pool,
                             const int64_t *__restrict__ slot_mapping, typename Tag::T *k_out,
                             typename Tag::T *v_out, int64_t rows, int H, int64_t num_slots,
                             unsigned int *err) {
  using T = typename Tag::T;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kFp4Threads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const int64_t t = row / H;
  const int h = static_cast<int>(row - t * H);
  const int64_t slot = slot_mapping[t];
  if (slot < 0 || slot >= num_slots) {
    if (slot >= num_slots && lane == 0) atomicOr(err, PHOTON_DEVERR_SLOT_RANGE);
    return;
  }
  const int64_t blk = slot / kBlockSize;
  const int r = static_cast<int>(slot - blk * kBlockSize);
  const unsigned char *rec = pool + (blk * H + h) * fp4_record_bytes(D);
#pragma unroll
  for (int idx = lane; idx < D; idx += 32) {  // D/2 byte pairs of K, then of V
    const int v = idx / (D / 2), e = 2 * (idx % (D / 2));
    const float2 x = e2m1_pair(rec[v ? fp4_v_byte(D, r, e) : fp4_k_byte(r, e)]);
    const float s = bf16_bits_to_f32(
        *reinterpret_cast<const uint16_t *>(rec + fp4_scale_byte(D, r, e / kFp4Group, v)));
    store2((v ? v_out : k_out) + row * D + e, x.x * s, x.y * s);
  }
}

template <typename Tag>
cudaError_t launch_write(const WriteArgs &a, unsigned int *err, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.num_tokens));
  if (a.head_dim == 64)
    return launch_pdl(kv_cache_write_fp4_kernel<Tag, 64>, grid, dim3(kFp4Threads), 0, st, a, err);
  return launch_pdl(kv_cache_write_fp4_kernel<Tag, 128>, grid, dim3(kFp4Threads), 0, st, a, err);
}

template <typename Tag>
cudaError_t launch_read(const Fp4ReadArgs &a, unsigned int *err, cudaStream_t st) {
  using T = typename Tag::T;
  const int64_t rows = static_cast<int64_t>(a.num_tokens) * a.num_kv_heads;
  const int64_t blocks = (rows + kFp4Threads / 32 - 1) / (kFp4Threads / 32);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  auto kern = a.head_dim == 64 ? kv_cache_read_fp4_kernel<Tag, 64> : kv_cache_read_fp4_kernel<Tag, 128>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kFp4Threads), 0, st,
                    static_cast<const unsigned char *>(a.pool), a.slot_mapping,
                    static_cast<T *>(a.k_out), static_cast<T *>(a.v_out), rows, a.num_kv_heads,
                    a.num_slots, err);
}

}  // namespace

cudaError_t launch_kv_cache_write_fp4(const WriteArgs &a, photon_dtype in_dt, unsigned int *err,
                                      cudaStream_t st) {
  if (a.num_tokens == 0) return cudaSuccess;
  return in_dt == PHOTON_BF16 ? launch_write<BF16Tag>(a, err, st) : launch_write<F32Tag>(a, err, st);
}

cudaError_t launch_kv_cache_read_fp4(const Fp4ReadArgs &a, photon_dtype out_dt, unsigned int *err,
                                     cudaStream_t st) {
  if (a.num_tokens == 0) return cudaSuccess;
  return out_dt == PHOTON_BF16 ? launch_read<BF16Tag>(a, err, st) : launch_read<F32Tag>(a, err, st);
}

}  // namespace photon
