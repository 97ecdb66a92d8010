// Split-K paged decode attention over a 4-bit (E2M1) KV cache with one bf16
// scale per token and 64 head dims, head_dim 64 or 128, on the tensor cores.
// Record layout in fp4.cuh; partial / merge contract, work split and walker as
// the FP8 kernel's (paged_decode_mma.cuh).
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(x_j - m),  x_j = scale log2(e) <q, k_j>
//
//  * A record (K, V and scales of one block and KV head) is contiguous and in
//    fragment order, so a page is one bulk copy into the warp's shared-memory
//    ring and every fragment one conflict-free 16-byte load.  A step covers PP
//    pages; the lanes that hold a step's block-table entries issue its copies,
//    ST steps ahead of the arithmetic and across item boundaries.  (Loads
//    straight into registers, one step ahead, left 8 to 16 warps per SM waiting
//    on latency: 384 us where the ring took 224, 128 contexts of up to 32k.)
//  * S = K Q^T with the 16 tokens of a page as the MMA's rows and the query
//    heads as its 8 columns: four MMAs per page and 64 dims, half of what the
//    transposed product needs for up to 8 heads.  O^T = V^T P^T takes P through
//    one movmatrix per 8 tokens.
//  * Codes convert to f16 exactly in hardware (cvt.rn.f16x2.e2m1x2).  The
//    scales never touch a code: a token's K scale multiplies its scores (per
//    64 dims), its V scale the probability that weights it.
//  * q enters as f16 after an exact power-of-two scaling of its row to
//    [1, 2), so any bf16 q keeps its 8 bits down to 2^-14 of the row's largest
//    value; the factor goes into the score scale, the scale's sign into q.
//  * Weights and their sum are kept relative to 2^m, m at most 2^6 above the
//    largest score so far, and so at most 1.  The weights of the second product
//    take their V scale times 2^(14 - E), E the largest exponent of the V scales
//    of the same 64 dims so far: they lie below 2^15 whatever the values'
//    magnitude, and round to f16 with relative error 2^-12 down to 2^-22 of the
//    largest, by at most 2^-33 of it below.  The accumulators carry 2^(14 - E)
//    to the end of the item, the sum never: a V scale that dwarfs the earlier
//    ones moves no weight.  For an fp32 output the remainder of the rounding
//    follows in a second MMA (SPLIT); for a bf16 output (half a step: 2^-8) it
//    would be lost anyway.  Sums, maxima and accumulators are fp32.
//
// What bounds it: DRAM on long steps (with the merge, 128 contexts of up to 32k
// tokens, d 64: 6.3 TB/s of records, 64 of d 128: 6.6; a copy reads and writes
// 6.8), the issue slots right behind it (some 120 warp instructions per 1088-byte
// page, ALU pipe 65 %, tensor pipe 32 %); start-up, uneven ends and the merge on
// steps of some 30 pages per warp (64 ragged sequences of d 128: 4.0 TB/s);
// latency on single requests.
#include <algorithm>
#include <atomic>
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "paged_decode.cuh"
#include "paged_decode_mma.cuh"

namespace photon {
namespace {

// Least E: 2^(14 - E) and its inverse are normal fp32 numbers.
constexpr int kFp4MinExp = -112;
// Base-2 distance of a new reference above the largest score: scores may grow
// by as much before it moves again.
constexpr float kFp4Slack = 6.f;
// E is held as the bits of the least bf16 with a greater exponent.
__device__ __forceinline__ uint32_t fp4_exp_limit(int e) { return static_cast<uint32_t>(e + 128) << 7; }
// 2^(14 - E), and its inverse
__device__ __forceinline__ float fp4_scale_down(uint32_t limit) {
  return __uint_as_float((static_cast<uint32_t>(127 + 14 + 128) << 23) - (limit << 16));
}
__device__ __forceinline__ float fp4_scale_up(uint32_t limit) {
  return __uint_as_float((limit << 16) - (static_cast<uint32_t>(128 + 14 - 127) << 23));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same into fresh accumulators.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                   *reinterpret_cast<const __nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&m);
}

// Transposes an 8x8 matrix of 16-bit values spread over the warp (lane 4r + c
// holds row r, columns 2c and 2c + 1).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

// Stage ring of a warp: ST steps of PP pages, whole records.
template <int D, int PP, int ST, int NW>
struct Fp4Ring {
  static constexpr int REC = fp4_record_bytes(D);
  static constexpr int STAGE = PP * REC;
  static constexpr int SMEM = NW * ST * (STAGE + 8);
  static_assert(32 % PP == 0, "a step lies in one block-table window");
  static_assert(ST * PP <= 32, "a bit per page of the ring");
};

// TEAM: an item belongs to a CTA, whose warps take a share of its pages each
// and meet in shared memory at its end (else every warp has items of its own).
// They walk the same items, so their barriers match; a warp that gave up on a
// copy still walks on to them.
template <int D, int PP, int ST, int NW, int MIN_CTAS, bool BAL, bool SPLIT, bool TEAM>
__global__ void __launch_bounds__(NW * 32, MIN_CTAS)
    paged_decode_fp4_kernel(const DecodeArgs a, unsigned int *err) {
  using R = Fp4Ring<D, PP, ST, NW>;
  constexpr int HH = D / 64;
  constexpr int REC = R::REC;
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int G = a.num_q_heads / a.num_kv_heads;
  unsigned char *stages = smem + warp * ST * R::STAGE;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + NW * ST * R::STAGE) + warp * ST;
  if (lane == 0) {
    for (int i = 0; i < ST; ++i) mbar_init(&bars[i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  if constexpr (BAL) prefetch_tables_l2(a);
  pdl_launch_dependents();
  const uint64_t policy = l2_evict_first_policy();
  const int workers = gridDim.x * (TEAM ? 1 : NW);  // that take items

  // this warp's share of an item's pages: whole steps, in order
  auto share = [&](Walker &w) {
    if constexpr (TEAM) {
      const int part = ((w.n_pages + NW - 1) / NW + PP - 1) / PP * PP;
      const int lo = min(warp * part, w.n_pages);
      w.n_pages = min(part, w.n_pages - lo);
      w.pg0 += lo;
    }
  };
  auto next_item = [&](Walker &w) {
    walker_next<BAL>(w, a, lane, err, workers);
    if (w.valid) share(w);
  };
  Walker prod, w;  // the producer, ST steps ahead, and the consumer
  walker_start<BAL>(prod, a, lane, err, TEAM ? blockIdx.x : blockIdx.x * NW + warp, workers);
  if (prod.valid) share(prod);
  w = prod;
  // this lane's K (V) scale of token 4 (g >> 1) + 2n + (g & 1): half g & 1 of word n
  const uint32_t half_sel = (g & 1) ? 0x3244u : 0x1044u;

  // Block-table window of the producer's item: lane j holds the record row of
  // page 32 k + j, `there` which of them exist with a block id in the pool;
  // the next window's ids are on their way.
  uint32_t row = 0, there = 0, valid_bits = 0;
  int ahead = -1, c_slot = 0;
  uint32_t c_phase = 0;
  auto table_entry = [&](int page) -> int {
    return page < prod.n_pages
               ? a.block_tables[seq_table_row(a, prod.s) * a.max_blocks_per_seq + prod.pg0 + page]
               : -1;
  };
  if (prod.valid) ahead = table_entry(lane);
  // metadata only so far; pages, q and the workspace wait for the preceding kernel
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.seg_count)  // the merge's mode
    a.seg_count[static_cast<int64_t>(a.num_seqs) * a.num_q_heads] = BAL ? 1 : 0;

  // Starts the copies of the producer's next step into ring slot `slot`: the
  // lanes of its pages in the window each copy their record.  False past the
  // warp's last step.
  auto issue_next = [&](int slot) -> bool {
    while (prod.valid && prod.page >= prod.n_pages) {
      next_item(prod);
      if (prod.valid) ahead = table_entry(lane);
    }
    if (!prod.valid) return false;
    const int at = prod.page & 31;
    if (at == 0) {
      const bool in = prod.page + lane < prod.n_pages;
      const bool ok = in && ahead >= 0 && ahead < a.num_blocks;
      row = ok ? static_cast<uint32_t>(ahead) * a.num_kv_heads + prod.h : 0u;
      there = __ballot_sync(0xffffffffu, ok);
      if (in && !ok) atomicOr(err, PHOTON_DEVERR_BLOCK_RANGE);
      ahead = table_entry(prod.page + 32 + lane);
    }
    const uint32_t v = (there >> at) & ((1u << PP) - 1);
    valid_bits = (valid_bits & ~(((1u << PP) - 1) << (PP * slot))) | (v << (PP * slot));
    if (lane == 0) mbar_arrive_expect_tx(&bars[slot], __popc(v) * REC);
    const int i = lane - at;
    if (i >= 0 && i < PP && (v >> i & 1u)) {
      fence_proxy_async_smem();
      bulk_copy_g2s(stages + slot * R::STAGE + i * REC,
                    static_cast<const unsigned char *>(a.k_cache) + static_cast<int64_t>(row) * REC, REC,
                    &bars[slot], policy);
    }
    prod.page += PP;
    return true;
  };
#pragma unroll 1
  for (int k = 0; k < ST; ++k)
    if (!issue_next(k)) break;

  bool gave_up = false;
  __shared__ float team_o[TEAM ? NW - 1 : 1][HH * 16][32];  // of warps 1 ..: accumulators,
  __shared__ float team_ml[TEAM ? NW - 1 : 1][4][32];       // references and sums
  while (w.valid) {
    // ---- a new item: the query group
    uint32_t qb[HH][4][2];     // q of head g, dims 16c + 4kt + {0,1}, {2,3} of each plane
    float sl[2];               // score factor of heads 2c, 2c + 1
    {
      float f[HH][16], qm = 0.f;
#pragma unroll
      for (int hh = 0; hh < HH; ++hh)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (g < G)
            v = reinterpret_cast<const uint4 *>(
                static_cast<const __nv_bfloat16 *>(a.q) +
                (static_cast<int64_t>(w.s) * a.num_q_heads + w.h * G + g) * D + 64 * hh + 16 * c)[i];
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[hh][8 * i + 2 * j] = bf16_lo(u[j]);
            f[hh][8 * i + 2 * j + 1] = bf16_hi(u[j]);
            qm = fmaxf(qm, fmaxf(fabsf(bf16_lo(u[j])), fabsf(bf16_hi(u[j]))));
          }
        }
      qm = fmaxf(qm, __shfl_xor_sync(0xffffffffu, qm, 1));
      qm = fmaxf(qm, __shfl_xor_sync(0xffffffffu, qm, 2));
      int e = static_cast<int>(__float_as_uint(qm) >> 23) - 127;
      if (e == 128 || qm == 0.f) e = 0;
      e = max(e, -100);
      float down = __uint_as_float(static_cast<uint32_t>(127 - min(e, 126)) << 23);  // 2^-e
      if (e == 127) down = 0x1p-127f;
      float s = fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      if (a.scale_log2 < 0.f) down = -down;
      if (s == 0.f) {  // all scores 0, by way of q: a masked token's -inf must stay one
        s = 1.f;
        down = 0.f;
      }
      sl[0] = __shfl_sync(0xffffffffu, s, 8 * c);
      sl[1] = __shfl_sync(0xffffffffu, s, 8 * c + 4);
#pragma unroll
      for (int hh = 0; hh < HH; ++hh)
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          qb[hh][kt][0] = pack_half2(f[hh][4 * kt] * down, f[hh][4 * kt + 1] * down);
          qb[hh][kt][1] = pack_half2(f[hh][4 * kt + 2] * down, f[hh][4 * kt + 3] * down);
        }
    }
    float o[HH][4][4];         // O^T: dims 64 hh + 8g + 2mt + {0, 1} of heads 2c, 2c + 1
#pragma unroll
    for (int hh = 0; hh < HH; ++hh)
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) o[hh][mt][0] = o[hh][mt][1] = o[hh][mt][2] = o[hh][mt][3] = 0.f;
    // weights are kept relative to m_ref, no score's exceeding it; e_lim: E of each plane
    float m_ref[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    uint32_t e_lim[HH];
#pragma unroll
    for (int hh = 0; hh < HH; ++hh) e_lim[hh] = fp4_exp_limit(kFp4MinExp);

    while (w.page < w.n_pages && !gave_up) {
      const bool landed = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[c_slot], c_phase, kWaitBudgetCycles));
      if (!landed) {
        if (lane == 0) atomicOr(err, PHOTON_DEVERR_WAIT_TIMEOUT);
        drain_async_copies();
        if constexpr (!TEAM) return;
        gave_up = true;  // the team's other warps still wait for this one
        break;
      }
      const uint32_t valid = (valid_bits >> (PP * c_slot)) & ((1u << PP) - 1);
      const unsigned char *stage = stages + c_slot * R::STAGE;
      // ---- scores: x[i][2n + j] belongs to token 4 (g >> 1) + 2n + (g & 1) of page i, head 2c + j
      float x[PP][4];
      uint32_t sv[PP][HH][2];
#pragma unroll
      for (int i = 0; i < PP; ++i) {
#pragma unroll
        for (int hh = 0; hh < HH; ++hh) {
          const uint4 kr = *reinterpret_cast<const uint4 *>(stage + i * REC + 512 * hh + 16 * lane);
          const uint4 sr = *reinterpret_cast<const uint4 *>(stage + i * REC + 16 * D + 64 * hh + 16 * (g >> 1));
          uint32_t k0[2][4], k1[2][4];  // tokens of n = 0 and 1
          e2m1x8_to_f16(kr.x, k0[0]);
          e2m1x8_to_f16(kr.y, k0[1]);
          e2m1x8_to_f16(kr.z, k1[0]);
          e2m1x8_to_f16(kr.w, k1[1]);
          float acc[4];
          mma_f16_first(acc, k0[0][0], k1[0][0], k0[0][1], k1[0][1], qb[hh][0][0], qb[hh][0][1]);
#pragma unroll
          for (int kt = 1; kt < 4; ++kt)
            mma_f16(acc, k0[kt >> 1][2 * (kt & 1)], k1[kt >> 1][2 * (kt & 1)], k0[kt >> 1][2 * (kt & 1) + 1],
                    k1[kt >> 1][2 * (kt & 1) + 1], qb[hh][kt][0], qb[hh][kt][1]);
          const float s0 = __uint_as_float(__byte_perm(sr.x, 0u, half_sel));
          const float s1 = __uint_as_float(__byte_perm(sr.y, 0u, half_sel));
          if (hh == 0) {
            x[i][0] = acc[0] * s0;
            x[i][1] = acc[1] * s0;
            x[i][2] = acc[2] * s1;
            x[i][3] = acc[3] * s1;
          } else {
            x[i][0] = fmaf(acc[0], s0, x[i][0]);
            x[i][1] = fmaf(acc[1], s0, x[i][1]);
            x[i][2] = fmaf(acc[2], s1, x[i][2]);
            x[i][3] = fmaf(acc[3], s1, x[i][3]);
          }
          sv[i][hh][0] = sr.z;
          sv[i][hh][1] = sr.w;
        }
      }
      const int tok0 = (w.pg0 + w.page) * kBlockSize;
      w.page += PP;
      if (valid) {  // no page of the step in the pool: nothing to add
        // tokens past the context, of absent pages: weight 0 (their bytes may hold anything)
        if (valid != (1u << PP) - 1 || tok0 + PP * kBlockSize > w.tok1) {
#pragma unroll
          for (int i = 0; i < PP; ++i) {
            const int nv = (valid >> i & 1u) ? w.tok1 - (tok0 + i * kBlockSize) : 0;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int tok = 4 * (g >> 1) + 2 * n;
              if (tok + (g & 1) >= nv) x[i][2 * n] = x[i][2 * n + 1] = -INFINITY;
              const uint32_t keep = (tok < nv ? 0x0000ffffu : 0u) | (tok + 1 < nv ? 0xffff0000u : 0u);
#pragma unroll
              for (int hh = 0; hh < HH; ++hh) sv[i][hh][n] &= keep;
            }
          }
        }
        float m0 = fmaxf(x[0][0], x[0][2]), m1 = fmaxf(x[0][1], x[0][3]);
        uint32_t sm[HH];
#pragma unroll
        for (int hh = 0; hh < HH; ++hh) sm[hh] = max_bf16x2(sv[0][hh][0], sv[0][hh][1]);
#pragma unroll
        for (int i = 0; i < PP; ++i) {
          if (i > 0) {
            m0 = max3(m0, x[i][0], x[i][2]);
            m1 = max3(m1, x[i][1], x[i][3]);
          }
#pragma unroll
          for (int hh = 0; hh < HH; ++hh)
            if (i > 0) sm[hh] = max_bf16x2(sm[hh], max_bf16x2(sv[i][hh][0], sv[i][hh][1]));
        }
        bool moves = m0 * sl[0] > m_ref[0] || m1 * sl[1] > m_ref[1];
#pragma unroll
        for (int hh = 0; hh < HH; ++hh) {
          sm[hh] = max(sm[hh] & 0xffffu, sm[hh] >> 16);  // scales are not negative
          moves |= sm[hh] >= e_lim[hh];
        }
        // A reference moves only when a score passes it or a V scale's exponent passes E.
        if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, d));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, d));
          }
          float alpha[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float ref = fmaxf(m_ref[j] - kFp4Slack, (j ? m1 : m0) * sl[j]) + kFp4Slack;
            alpha[j] = exp2_approx(m_ref[j] - ref);
            m_ref[j] = ref;
            l_run[j] *= alpha[j];
          }
#pragma unroll
          for (int hh = 0; hh < HH; ++hh) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, sm[hh]) >> 7;  // 127 + exponent
            const uint32_t lim = max(e_lim[hh], fp4_exp_limit(min(static_cast<int>(top) - 127, 127)));
            // 2^(old E - new E), 0 where that is below 2^-126
            const float fall = __int_as_float(max(0x3f800000 - static_cast<int>((lim - e_lim[hh]) << 16), 0));
            e_lim[hh] = lim;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
              o[hh][mt][0] *= alpha[0] * fall;
              o[hh][mt][1] *= alpha[1] * fall;
              o[hh][mt][2] *= alpha[0] * fall;
              o[hh][mt][3] *= alpha[1] * fall;
            }
          }
        }
        float down[HH];
#pragma unroll
        for (int hh = 0; hh < HH; ++hh) down[hh] = fp4_scale_down(e_lim[hh]);
        uint32_t ph[PP][HH][2], pl[SPLIT ? PP : 1][HH][2];
#pragma unroll
        for (int i = 0; i < PP; ++i)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float p0 = exp2_approx(fmaf(x[i][2 * n], sl[0], -m_ref[0]));
            const float p1 = exp2_approx(fmaf(x[i][2 * n + 1], sl[1], -m_ref[1]));
            l_run[0] += p0;
            l_run[1] += p1;
#pragma unroll
            for (int hh = 0; hh < HH; ++hh) {
              const float s = __uint_as_float(__byte_perm(sv[i][hh][n], 0u, half_sel)) * down[hh];
              const float w0 = p0 * s, w1 = p1 * s;
              const uint32_t h = pack_half2(w0, w1);
              ph[i][hh][n] = transpose_8x8(h);
              if constexpr (SPLIT) {
                const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                pl[i][hh][n] = transpose_8x8(pack_half2(w0 - r.x, w1 - r.y));
              }
            }
          }
        // ---- O^T += V^T P^T: words of tokens 4c .. 4c+3, nibble i = dim 8g + i.
        // Pairing the same nibble of two tokens in one byte gives the f16 pairs
        // (token, token + 1) of the MMA's A operand directly.
#pragma unroll
        for (int i = 0; i < PP; ++i)
#pragma unroll
          for (int hh = 0; hh < HH; ++hh) {
            const uint4 v = *reinterpret_cast<const uint4 *>(stage + i * REC + 8 * D + 512 * hh + 16 * lane);
            uint32_t e01[4], o01[4], e23[4], o23[4];
            e2m1x8_to_f16((v.x & 0x0f0f0f0fu) | ((v.y << 4) & 0xf0f0f0f0u), e01);
            e2m1x8_to_f16(((v.x >> 4) & 0x0f0f0f0fu) | (v.y & 0xf0f0f0f0u), o01);
            e2m1x8_to_f16((v.z & 0x0f0f0f0fu) | ((v.w << 4) & 0xf0f0f0f0u), e23);
            e2m1x8_to_f16(((v.z >> 4) & 0x0f0f0f0fu) | (v.w & 0xf0f0f0f0u), o23);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
              mma_f16(o[hh][mt], e01[mt], o01[mt], e23[mt], o23[mt], ph[i][hh][0], ph[i][hh][1]);
              if constexpr (SPLIT)
                mma_f16(o[hh][mt], e01[mt], o01[mt], e23[mt], o23[mt], pl[i][hh][0], pl[i][hh][1]);
            }
          }
      }
      __syncwarp();  // the stage is read before the next copies overwrite it
      issue_next(c_slot);
      if (++c_slot == ST) {
        c_slot = 0;
        c_phase ^= 1u;
      }
    }

#pragma unroll
    for (int i = 0; i < HH * 16; ++i) o[i / 16][i / 4 % 4][i % 4] *= fp4_scale_up(e_lim[i / 16]);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l_run[j] += __shfl_xor_sync(0xffffffffu, l_run[j], d);
    if constexpr (TEAM) {  // warp 0 adds the others' shares, in order
      if (warp > 0) {
#pragma unroll
        for (int i = 0; i < HH * 16; ++i) team_o[warp - 1][i][lane] = o[i / 16][i / 4 % 4][i % 4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          team_ml[warp - 1][j][lane] = m_ref[j];
          team_ml[warp - 1][2 + j][lane] = l_run[j];
        }
      }
      __syncthreads();
      if (warp == 0) {
        float M[2] = {m_ref[0], m_ref[1]}, f[NW][2];
#pragma unroll
        for (int k = 0; k < NW - 1; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) M[j] = fmaxf(M[j], team_ml[k][j][lane]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          f[0][j] = m_ref[j] == -INFINITY ? 0.f : exp2_approx(m_ref[j] - M[j]);
          l_run[j] *= f[0][j];
          m_ref[j] = M[j];
        }
#pragma unroll
        for (int k = 0; k < NW - 1; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float mk = team_ml[k][j][lane];
            f[k + 1][j] = mk == -INFINITY ? 0.f : exp2_approx(mk - M[j]);
            l_run[j] = fmaf(team_ml[k][2 + j][lane], f[k + 1][j], l_run[j]);
          }
#pragma unroll
        for (int i = 0; i < HH * 16; ++i) {
          float &x = o[i / 16][i / 4 % 4][i % 4];
          x *= f[0][i & 1];
#pragma unroll
          for (int k = 0; k < NW - 1; ++k) x = fmaf(team_o[k][i][lane], f[k + 1][i & 1], x);
        }
      }
      __syncthreads();  // read before the next item's shares are written
      if (warp > 0) {
        next_item(w);
        continue;
      }
    }
    // ---- item done: o[hh][mt][2r + j] is head 2c + j, dim 64 hh + 8g + 2mt + r
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float l = l_run[j];
      const int head = 2 * c + j;
      if (head >= G) continue;
      const int64_t qrow = static_cast<int64_t>(w.s) * a.num_q_heads + w.h * G + head;
      if constexpr (BAL)
        if (g == 0 && w.p == 0) a.seg_count[qrow] = w.P_s;
      const bool whole = w.P_s == 1;
      const float f = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
      const int64_t prow = qrow * a.max_partitions + w.p;
#pragma unroll
      for (int hh = 0; hh < HH; ++hh) {
        float v[8];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          v[2 * mt] = o[hh][mt][j] * f;
          v[2 * mt + 1] = o[hh][mt][2 + j] * f;
        }
        if (whole && a.out_bf16) {
          *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + qrow * D + 64 * hh + 8 * g) =
              make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                         pack_bf16(v[6], v[7]));
        } else {
          float *dst = (whole ? static_cast<float *>(a.out) + qrow * D : a.o_part + prow * D) + 64 * hh + 8 * g;
          reinterpret_cast<float4 *>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<float4 *>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
      if (!whole && g == 0) {
        a.m_part[prow] = m_ref[j];
        a.l_part[prow] = l;
      }
    }
    next_item(w);
  }
}

// Long steps run one CTA of NW1 warps per SM, on steps of PP1 pages: the warp
// scheduler shares an SM evenly between the warps of one CTA but prefers older
// CTAs, and four CTAs of four warps with equal runs ended after 140, 158, 182
// and 206 us (128 contexts of up to 32k tokens; kernel and merge 213 us, one
// CTA of 16 warps 197 us, of 12 warps with steps of 8 pages 193 us; 32 of them
// 59.9 -> 56.9 us; 64 of d 128 190.7 -> 176.2 us).  Chosen when the page bound
// -- sequences x ceil(max context / 16) x KV heads -- reaches
// kFp4MinPagesPerWarp per warp; ragged batches of some 30 pages per warp
// (bounds of 120 to 140) lose 1 to 4 % with it, and grids smaller than the GPU
// need CTAs of four warps to spread over its SMs.
constexpr int64_t kFp4MinPagesPerWarp = 192;

inline int64_t page_bound(const DecodeArgs &a) {
  return static_cast<int64_t>(a.num_seqs) * ((static_cast<int64_t>(a.ctx_cap) + kBlockSize - 1) / kBlockSize) *
         a.num_kv_heads;
}

// When items are few and long, a CTA of four warps takes each: the piece count
// of a row is bounded by the partition size (the workspace has no more slots),
// and an item of 32 pages keeps a single warp busy for 10 us however idle the
// GPU.  Teams are used where the least piece, or an item without a workspace,
// has
//  * 8 pages, without a workspace 4, and all items fit the GPU as CTAs at once:
//    one warp per item -> a team, 64 sequences of 128 tokens 6.9 -> 5.8 us, 8 of
//    1024 in pieces of 8 pages 7.1 -> 6.6 (of 4 pages: 4 of 1024 5.7 -> 5.9),
//    30 of 518 (two KV heads, 32 pages) 15.0 -> 9.6, one of 32768 17.9 -> 10.0,
//    9 of 1432 (d 128, fp32 output) 25.2 -> 12.5;
//  * 16 pages, with more items: pieces as long as the workspace allows must
//    leave warps idle (60 ragged sequences of up to 1000 tokens, d 128, 28.2 ->
//    19.3; 40 of up to 1024, 14.4 -> 12.0), items be at most two to a CTA (64 of
//    500, d 128, 21.3 -> 15.8).  With 8 pages 16 of 2048 10.2 -> 13.6.
constexpr int kFp4TeamPages = 8, kFp4TeamItemPages = 4, kFp4TeamManyPages = 16;

template <bool BAL>
inline bool team_step(const DecodeArgs &a, int64_t items, int64_t ctas, int warps_per_cta) {
  const int longest = (a.partition_size < a.ctx_cap ? a.partition_size : a.ctx_cap) / kBlockSize;
  if (items <= ctas) return longest >= (BAL ? kFp4TeamPages : kFp4TeamItemPages);
  if (longest < kFp4TeamManyPages || a.num_kv_heads > ctas / 4) return false;
  return BAL ? page_bound(a) <= ctas * warps_per_cta * (a.partition_size / kBlockSize) : items <= 2 * ctas;
}

enum class Fp4Fit { kAlways, kLongSteps, kTeams };  // when launch_fp4_kern takes a step

template <int D, int PP, int ST, int NW, int MIN_CTAS, bool BAL, bool SPLIT, Fp4Fit FIT>
cudaError_t launch_fp4_kern(const DecodeArgs &a, unsigned int *err, cudaStream_t stream, bool *taken) {
  constexpr bool TEAM = FIT == Fp4Fit::kTeams;
  constexpr int SMEM = Fp4Ring<D, PP, ST, NW>::SMEM;
  auto kern = paged_decode_fp4_kernel<D, PP, ST, NW, MIN_CTAS, BAL, SPLIT, TEAM>;
  static std::atomic<int> occupancy[64];  // per device; 0 = not set up (races repeat it)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  int occ = occupancy[dev].load(std::memory_order_relaxed);
  if (occ == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, NW * 32, SMEM);
    if (e != cudaSuccess) return e;
    occ = occ > 0 ? occ : 1;
    occupancy[dev].store(occ, std::memory_order_relaxed);
  }
  const int64_t items = static_cast<int64_t>(a.num_seqs) * a.max_partitions * a.num_kv_heads;
  const int64_t ctas_cap = static_cast<int64_t>(device_sm_count()) * occ;
  const int64_t warps_cap = ctas_cap * NW;
  *taken = FIT == Fp4Fit::kAlways ||
           (FIT == Fp4Fit::kTeams && team_step<BAL>(a, items, ctas_cap, NW)) ||
           (FIT == Fp4Fit::kLongSteps && items >= warps_cap && page_bound(a) >= kFp4MinPagesPerWarp * warps_cap);
  if (!*taken || items == 0) return cudaSuccess;
  const int64_t workers = std::min(items, TEAM ? ctas_cap : warps_cap);
  const int64_t grid = TEAM ? workers : (workers + NW - 1) / NW;
  DecodeArgs la = a;
  la.balanced = BAL ? 1 : 0;
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(NW * 32), SMEM, stream, la, err);
}

// PP, ST, MIN_CTAS: CTAs of four warps; PP1, ST1, NW1: the one CTA per SM of
// long steps.  Short steps take few pages at once (d 64: one request of 1024
// tokens 6.8 us with four, 6.2 with two; 16 contexts of up to 2048 11.8, 11.1).
template <int D, int PP, int ST, int MIN_CTAS, int PP1, int ST1, int NW1, bool SPLIT, bool BAL>
cudaError_t launch_fp4_split(const DecodeArgs &a, unsigned int *err, cudaStream_t stream) {
  bool taken = false;
  cudaError_t e = launch_fp4_kern<D, PP, ST, 4, 1, BAL, SPLIT, Fp4Fit::kTeams>(a, err, stream, &taken);
  if (e != cudaSuccess || taken) return e;
  if constexpr (BAL) {
    e = launch_fp4_kern<D, PP1, ST1, NW1, 1, true, SPLIT, Fp4Fit::kLongSteps>(a, err, stream, &taken);
    if (e != cudaSuccess || taken) return e;
  }
  return launch_fp4_kern<D, PP, ST, 4, MIN_CTAS, BAL, SPLIT, Fp4Fit::kAlways>(a, err, stream, &taken);
}

template <int D, int PP, int ST, int MIN_CTAS, int PP1, int ST1, int NW1, bool SPLIT>
cudaError_t launch_fp4(const DecodeArgs &a, unsigned int *err, cudaStream_t stream) {
  return balanced_pieces(a) ? launch_fp4_split<D, PP, ST, MIN_CTAS, PP1, ST1, NW1, SPLIT, true>(a, err, stream)
                            : launch_fp4_split<D, PP, ST, MIN_CTAS, PP1, ST1, NW1, SPLIT, false>(a, err, stream);
}

// Merge of a row's pieces: out = sum_p o_p 2^(m_p - M) / sum_p l_p 2^(m_p - M).
// One CTA per (sequence, query head): D/4 lanes hold a piece's row, STREAMS
// streams of lanes take the pieces in turn, a stream's next two or four at
// once, so that a row costs three dependent steps (count, pieces, the streams'
// sums through shared memory), which is what bounds it.  Decode and merge, with
// the general merge kernel and with this one: one request of 1024 tokens 6.2 ->
// 4.6 us, 16 contexts of up to 2048 11.1 -> 10.0, 8 of up to 32k (d 128)
// 27.8 -> 25.8.  Up to kFp4FewRows rows per SM take 16 streams of two pieces,
// more rows 8 of four (64 ragged sequences of d 128, 1024 rows: 30.6 us, 32.5 with 16).
constexpr int kFp4FewRows = 4;

template <int D, int STREAMS>
__global__ void __launch_bounds__(STREAMS * D / 4) fp4_merge_kernel(const DecodeArgs a) {
  constexpr int LANES = D / 4, N = STREAMS == 16 ? 2 : 4;
  __shared__ float4 s_o[STREAMS][LANES];
  __shared__ float s_m[STREAMS], s_l[STREAMS];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const int P = min(a.seg_count[row], a.max_partitions);
  if (P <= 1) return;  // the decode kernel wrote the row
  const int k = threadIdx.x / LANES, x = threadIdx.x % LANES;
  const float *mp = a.m_part + row * a.max_partitions, *lp = a.l_part + row * a.max_partitions;
  const float4 *op = reinterpret_cast<const float4 *>(a.o_part + row * a.max_partitions * D) + x;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float m1, float l1, const float4 &v, float M) {
    const float f = m1 == -INFINITY ? 0.f : exp2f(m1 - M);  // a piece without valid pages
    l = fmaf(l1, f, l);
    o.x = fmaf(v.x, f, o.x);
    o.y = fmaf(v.y, f, o.y);
    o.z = fmaf(v.z, f, o.z);
    o.w = fmaf(v.w, f, o.w);
  };
  auto rescale = [&](float M) {
    const float f = m == -INFINITY ? 0.f : exp2f(m - M);
    l *= f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    m = M;
  };
  for (int p0 = k; p0 < P; p0 += N * STREAMS) {
    float m1[N], l1[N], M = m;
    float4 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = p0 + i * STREAMS;
      m1[i] = -INFINITY;
      l1[i] = 0.f;
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p < P) {
        m1[i] = mp[p];
        l1[i] = lp[p];
        v[i] = op[static_cast<int64_t>(p) * LANES];
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) M = fmaxf(M, m1[i]);
    rescale(M);
#pragma unroll
    for (int i = 0; i < N; ++i) add(m1[i], l1[i], v[i], M);
  }
  s_o[k][x] = o;
  if (x == 0) {
    s_m[k] = m;
    s_l[k] = l;
  }
  __syncthreads();
  if (k != 0) return;
  float M = m;
#pragma unroll
  for (int j = 1; j < STREAMS; ++j) M = fmaxf(M, s_m[j]);
  rescale(M);
#pragma unroll
  for (int j = 1; j < STREAMS; ++j) add(s_m[j], s_l[j], s_o[j][x], M);
  const float f = l > 0.f || l != l ? 1.f / l : 0.f;
  o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
  if (a.out_bf16)
    reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + row * D)[x] =
        make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
  else
    reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row * D)[x] = o;
}

}  // namespace

cudaError_t launch_decode_merge_fp4(const DecodeArgs &a, cudaStream_t st) {
  if (!balanced_pieces(a)) return launch_decode_reduce(a, st);  // fixed partitions
  const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.num_q_heads;
  if (rows > INT32_MAX) return cudaErrorInvalidValue;
  const bool few = rows <= kFp4FewRows * static_cast<int64_t>(device_sm_count());
  auto kern = a.head_dim == 64 ? (few ? fp4_merge_kernel<64, 16> : fp4_merge_kernel<64, 8>)
                               : (few ? fp4_merge_kernel<128, 16> : fp4_merge_kernel<128, 8>);
  return launch_pdl(kern, dim3(static_cast<unsigned>(rows)), dim3((few ? 16 : 8) * a.head_dim / 4), 0, st, a);
}

cudaError_t launch_decode_partial_fp4(const DecodeArgs &a, unsigned int *err, cudaStream_t st) {
  if (a.head_dim == 64)
    return a.out_bf16 ? launch_fp4<64, 2, 5, 4, 8, 2, 12, false>(a, err, st)
                      : launch_fp4<64, 2, 5, 4, 8, 2, 12, true>(a, err, st);
  if (a.head_dim == 128)
    return a.out_bf16 ? launch_fp4<128, 2, 3, 3, 4, 2, 12, false>(a, err, st)
                      : launch_fp4<128, 2, 3, 3, 4, 2, 12, true>(a, err, st);
  return cudaErrorInvalidValue;
}

}  // namespace photon
