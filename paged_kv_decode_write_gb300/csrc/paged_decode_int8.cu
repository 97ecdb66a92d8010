// Split-K paged decode attention over the 8-bit KV cache with one scale per block
// and KV head, head_dim 64 or 128, on the tensor cores.  Record layout in
// int8.cuh; partial / merge contract, work split and walker as the FP8 and 4-bit
// kernels' (paged_decode_mma.cuh).
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(x_j - m),  x_j = scale log2(e) s_K <q, c_j>
//
//  * A record is contiguous and in fragment order: a page is one bulk copy into
//    the warp's shared-memory ring and every fragment conflict-free 16-byte loads.
//    The lanes that hold a step's block-table entries issue its copies, ST steps
//    of PP pages ahead of the arithmetic and across item boundaries.
//  * S = K Q^T with the 16 tokens of a page as the MMA's rows and up to 8 query
//    heads as its columns; O^T = V^T P^T takes P through one movmatrix per 8 tokens.
//  * A byte b becomes the f16 number 1024 + b by a byte permute (0x64 into the high
//    byte) and the code by subtracting 1152, exactly: a permute and a half of an
//    f16x2 subtraction per pair of K codes, one logic operation more per pair of V
//    codes, whose bytes lie token by token.  The scales never touch a code: s_K
//    multiplies a page's scores, s_V its weights.
//  * q enters as f16 after an exact power-of-two scaling of its row to [1, 2), so
//    any bf16 q keeps its 8 bits down to 2^-14 of the row's largest value.
//  * Weights and their sum are kept relative to 2^m, m at most 2^6 above the
//    largest score so far.  The weights of the second product take s_V 2^(14 - E),
//    E the largest exponent of the item's s_V so far: below 2^15 whatever the
//    values' magnitude.  They enter as their f16 rounding and, in a second MMA, the
//    f16 remainder: within 2^-22 of themselves or 2^-25, and the largest is 2^8 or more.
//    (f16 alone, 2^-11, put 8 to 10 % of bf16 outputs on the other side of a rounding
//    border; the second MMA costs 1 % of ragged batches of d 128, 3 % of long steps of
//    d 64.)  The accumulators carry 2^(14 - E) to the end of the item, the sum never.
//    Sums, maxima and accumulators are fp32.
//
// What bounds it: DRAM on long steps, the issue slots close behind (with the merge, 128
// contexts of up to 32k tokens, d 64, 2.15 GB: 327 us, 6.58 TB/s where a copy reads and
// writes 6.79; 64 of up to 16k, d 128, 164 us, 0.97 of the copy rate); between, start-up,
// uneven ends and the merge (64 ragged sequences of d 128, 258 MB: 47.6 us, 0.80: the first
// page lands after 3 to 4 us, the bulk runs at the copy rate, the last warp ends 4 us after
// the median one, the merge takes 1.5); latency on short ones (one context of 1024: 4.1 us).
#include <algorithm>
#include <atomic>

#include "int8.cuh"
#include "mma_f16.cuh"
#include "paged_decode.cuh"
#include "paged_decode_mma.cuh"

namespace photon {
namespace {

// Least E: 2^(14 - E) and its inverse are normal fp32 numbers.
constexpr int kMinExp = -112;
// Base-2 distance of a new reference above the largest score.
constexpr float kSlack = 6.f;

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

constexpr uint32_t kHalf1024 = 0x64646464u;  // high byte of an f16 in [1024, 2048)
constexpr uint32_t kHalf1152 = 0x64806480u;  // 1152 twice

// The four codes of a word as f16: (byte 0, byte 1) and (byte 2, byte 3).
__device__ __forceinline__ void codes_in_order(uint32_t w, uint32_t &lo, uint32_t &hi) {
  lo = sub_f16x2(__byte_perm(w, kHalf1024, 0x4140u), kHalf1152);
  hi = sub_f16x2(__byte_perm(w, kHalf1024, 0x4342u), kHalf1152);
}

// Byte i of a and of b as f16 codes (a in the low half).
template <int I>
__device__ __forceinline__ uint32_t codes_across(uint32_t a, uint32_t b) {
  const uint32_t w = __byte_perm(a, b, 0x0400u + 0x0101u * I);
  return sub_f16x2((w & 0x00ff00ffu) | 0x64006400u, kHalf1152);
}

// Stage ring of a warp: ST steps of PP pages, whole records.
template <int D, int PP, int ST, int NW>
struct Int8Ring {
  static constexpr int REC = int8_record_bytes(D);
  static constexpr int STAGE = PP * REC;
  static constexpr int SMEM = NW * ST * (STAGE + 8);
  static_assert(32 % PP == 0, "a step lies in one block-table window");
  static_assert(ST * PP <= 32, "a bit per page of the ring");
};

// Who takes an item.
enum class Mode {
  kWarps,    // every warp has items of its own
  kTeams,    // a CTA, whose warps take a share of its pages each and meet in shared
             // memory at its end.  They walk the same items, so their barriers match; a
             // warp that gave up on a copy still walks on to them
  kCluster,  // a cluster of CTAs, the whole context of one sequence and KV head: their
             // teams' results meet in distributed shared memory, nothing is left to merge
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The float at p in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ float load_cluster(const float *p, uint32_t rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

template <int D, int PP, int ST, int NW, int MIN_CTAS, bool BAL, Mode MODE>
__global__ void __launch_bounds__(NW * 32, MIN_CTAS)
    paged_decode_int8_kernel(const DecodeArgs a, unsigned int *err) {
  using R = Int8Ring<D, PP, ST, NW>;
  constexpr bool TEAM = MODE != Mode::kWarps, CLUSTER = MODE == Mode::kCluster;
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
    if constexpr (CLUSTER) {
      w.valid = false;
    } else {
      walker_next<BAL>(w, a, lane, err, workers);
      if (w.valid) share(w);
    }
  };
  Walker prod, w;  // the producer, ST steps ahead, and the consumer
  if constexpr (CLUSTER) {
    const int pair = static_cast<int>(blockIdx.x / cluster_size());
    const int warps = static_cast<int>(cluster_size()) * NW;
    prod.s = pair / a.num_kv_heads;
    prod.h = pair - prod.s * a.num_kv_heads;
    prod.ctx = prod.tok1 = balanced_ctx(a, prod.s, err);
    const int pages = (prod.ctx + kBlockSize - 1) / kBlockSize;
    const int part = ((pages + warps - 1) / warps + PP - 1) / PP * PP;
    prod.pg0 = min(static_cast<int>(cluster_rank() * NW + warp) * part, pages);
    prod.n_pages = min(part, pages - prod.pg0);
    prod.page = prod.p = 0;
    prod.P_s = 1;
    prod.valid = true;
  } else {
    walker_start<BAL>(prod, a, lane, err, TEAM ? blockIdx.x : blockIdx.x * NW + warp, workers);
    if (prod.valid) share(prod);
  }
  w = prod;

  // Block-table window of the producer's item: lane j holds the record row of
  // page 32 k + j, `there` which of them exist with a block id in the pool;
  // the next window's ids are on their way.
  uint32_t there = 0, valid_bits = 0;
  int64_t row = 0;
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
  if (!CLUSTER && blockIdx.x == 0 && threadIdx.x == 0 && a.seg_count)  // the merge's mode
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
      row = ok ? static_cast<int64_t>(ahead) * a.num_kv_heads + prod.h : 0;
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
                    static_cast<const unsigned char *>(a.k_cache) + row * REC, REC, &bars[slot], policy);
    }
    prod.page += PP;
    return true;
  };
#pragma unroll 1
  for (int k = 0; k < ST; ++k)
    if (!issue_next(k)) break;

  bool gave_up = false;
  __shared__ float team_o[TEAM ? NW - 1 : 1][HH * 16][32];  // of warps 1 ..: accumulators,
  __shared__ float team_ml[TEAM ? NW - 1 : 1][4][32];       // references and sums; then [0]: the team's
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
      e = max(e, -126);  // 2^-e and 2^e are normal numbers; a subnormal row becomes at least 2^-7
      const float down = e == 127 ? 0x1p-127f : pow2(-e);  // 2^-e
      const float s = a.scale_log2 * pow2(e);
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
    // weights are kept relative to m_ref, no score's exceeding it; E: see above
    float m_ref[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    int E = kMinExp;

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
      float x[PP][4], sv[PP];
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        float acc[4];
#pragma unroll
        for (int hh = 0; hh < HH; ++hh) {
          const uint4 r0 = *reinterpret_cast<const uint4 *>(stage + i * REC + 1024 * hh + 16 * lane);
          const uint4 r1 = *reinterpret_cast<const uint4 *>(stage + i * REC + 1024 * hh + 512 + 16 * lane);
          const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
          for (int kt = 0; kt < 4; ++kt) {
            uint32_t a0, a1, a2, a3;
            codes_in_order(w0[kt], a0, a2);
            codes_in_order(w1[kt], a1, a3);
            if (hh == 0 && kt == 0)
              mma_f16_first(acc, a0, a1, a2, a3, qb[hh][kt][0], qb[hh][kt][1]);
            else
              mma_f16(acc, a0, a1, a2, a3, qb[hh][kt][0], qb[hh][kt][1]);
          }
        }
        const float2 sc = *reinterpret_cast<const float2 *>(stage + i * REC + int8_scale_byte(D, 0));
        // K's scale first: |k| times a q below 2 stays in range, both factors together may not
        x[i][0] = acc[0] * sc.x * sl[0];
        x[i][1] = acc[1] * sc.x * sl[1];
        x[i][2] = acc[2] * sc.x * sl[0];
        x[i][3] = acc[3] * sc.x * sl[1];
        sv[i] = sc.y;
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
            for (int n = 0; n < 2; ++n)
              if (4 * (g >> 1) + 2 * n + (g & 1) >= nv) x[i][2 * n] = x[i][2 * n + 1] = -INFINITY;
            if (nv <= 0) sv[i] = 0.f;
          }
        }
        float m0 = fmaxf(x[0][0], x[0][2]), m1 = fmaxf(x[0][1], x[0][3]);
        uint32_t top = __float_as_uint(sv[0]);
#pragma unroll
        for (int i = 1; i < PP; ++i) {
          m0 = max3(m0, x[i][0], x[i][2]);
          m1 = max3(m1, x[i][1], x[i][3]);
          top = max(top, __float_as_uint(sv[i]));
        }
        const int e_top = min(static_cast<int>(top >> 23 & 0xffu) - 127, 127);  // the same in every lane
        // A reference moves only when a score passes it or a V scale's exponent passes E.
        if (__any_sync(0xffffffffu, m0 > m_ref[0] || m1 > m_ref[1] || e_top > E)) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, d));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, d));
          }
          float alpha[2];
          const int e_new = max(E, e_top);
          const float fall = pow2(max(E - e_new, -127));  // 0 below 2^-126
          E = e_new;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float ref = fmaxf(m_ref[j] - kSlack, j ? m1 : m0) + kSlack;
            alpha[j] = exp2_approx(m_ref[j] - ref);
            m_ref[j] = ref;
            l_run[j] *= alpha[j];
            alpha[j] *= fall;
          }
#pragma unroll
          for (int hh = 0; hh < HH; ++hh)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
              o[hh][mt][0] *= alpha[0];
              o[hh][mt][1] *= alpha[1];
              o[hh][mt][2] *= alpha[0];
              o[hh][mt][3] *= alpha[1];
            }
        }
        const float down = pow2(14 - E);
        uint32_t ph[PP][2], pl[PP][2];
#pragma unroll
        for (int i = 0; i < PP; ++i) {
          const float s = sv[i] * down;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float p0 = exp2_approx(x[i][2 * n] - m_ref[0]);
            const float p1 = exp2_approx(x[i][2 * n + 1] - m_ref[1]);
            l_run[0] += p0;
            l_run[1] += p1;
            const float w0 = p0 * s, w1 = p1 * s;
            const uint32_t h = pack_half2(w0, w1);
            ph[i][n] = transpose_8x8(h);
            const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            pl[i][n] = transpose_8x8(pack_half2(w0 - r.x, w1 - r.y));
          }
        }
        // ---- O^T += V^T P^T: bytes of the same dim of two tokens make an f16 pair of the A operand
#pragma unroll
        for (int i = 0; i < PP; ++i)
#pragma unroll
          for (int hh = 0; hh < HH; ++hh) {
            const unsigned char *vp = stage + i * REC + 16 * D + 1024 * hh + 16 * lane;
            const uint4 v0 = *reinterpret_cast<const uint4 *>(vp);        // tokens 4c, 4c + 1
            const uint4 v1 = *reinterpret_cast<const uint4 *>(vp + 512);  // tokens 4c + 2, 4c + 3
            // the four weights' MMAs, then the four remainders': none waits for the one before
            uint32_t code[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint32_t x0 = t < 2 ? v0.x : v0.y, y0 = t < 2 ? v0.z : v0.w;
              const uint32_t x1 = t < 2 ? v1.x : v1.y, y1 = t < 2 ? v1.z : v1.w;
              code[t][0] = t & 1 ? codes_across<2>(x0, y0) : codes_across<0>(x0, y0);
              code[t][1] = t & 1 ? codes_across<3>(x0, y0) : codes_across<1>(x0, y0);
              code[t][2] = t & 1 ? codes_across<2>(x1, y1) : codes_across<0>(x1, y1);
              code[t][3] = t & 1 ? codes_across<3>(x1, y1) : codes_across<1>(x1, y1);
              mma_f16(o[hh][t], code[t][0], code[t][1], code[t][2], code[t][3], ph[i][0], ph[i][1]);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
              mma_f16(o[hh][t], code[t][0], code[t][1], code[t][2], code[t][3], pl[i][0], pl[i][1]);
          }
      }
      __syncwarp();  // the stage is read before the next copies overwrite it
      issue_next(c_slot);
      if (++c_slot == ST) {
        c_slot = 0;
        c_phase ^= 1u;
      }
    }

    const float up = pow2(E - 14);
#pragma unroll
    for (int i = 0; i < HH * 16; ++i) o[i / 16][i / 4 % 4][i % 4] *= up;
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
          float &y = o[i / 16][i / 4 % 4][i % 4];
          y *= f[0][i & 1];
#pragma unroll
          for (int k = 0; k < NW - 1; ++k) y = fmaf(team_o[k][i][lane], f[k + 1][i & 1], y);
        }
      }
      if constexpr (CLUSTER) {
        const uint32_t C = cluster_size();
        if (C > 1) {
          if (warp == 0) {
            __syncwarp();  // every lane has read the others' shares
#pragma unroll
            for (int i = 0; i < HH * 16; ++i) team_o[0][i][lane] = o[i / 16][i / 4 % 4][i % 4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              team_ml[0][j][lane] = m_ref[j];
              team_ml[0][2 + j][lane] = l_run[j];
            }
          }
          cluster_barrier();
          // the first CTA's warps: 4 dims of head 2c + j each, dims 64 hh + 8g + 4t ..
          for (int k = warp; cluster_rank() == 0 && k < 4 * HH; k += NW) {
            const int hh = k >> 2, t = k >> 1 & 1, j = k & 1, head = 2 * c + j;
            float M = -INFINITY, L = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
            for (uint32_t q0 = 0; q0 < C; q0 += 4) {  // the CTAs in order, four at once
              float m1[4], l1[4], x[4][4], top = M;
#pragma unroll
              for (uint32_t q = 0; q < 4; ++q) {
                const uint32_t r = min(q0 + q, C - 1);
                m1[q] = load_cluster(&team_ml[0][j][lane], r);
                l1[q] = load_cluster(&team_ml[0][2 + j][lane], r);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  x[q][i] = load_cluster(&team_o[0][16 * hh + 4 * (2 * t + (i >> 1)) + 2 * (i & 1) + j][lane], r);
                if (q0 + q >= C) m1[q] = -INFINITY;
                top = fmaxf(top, m1[q]);
              }
              const float f0 = M == -INFINITY ? 0.f : exp2_approx(M - top);
              L *= f0;
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] *= f0;
              M = top;
#pragma unroll
              for (uint32_t q = 0; q < 4; ++q) {
                if (q0 + q >= C) continue;
                const float f = m1[q] == -INFINITY ? 0.f : exp2_approx(m1[q] - M);  // a team without pages
                L = fmaf(l1[q], f, L);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = fmaf(x[q][i], f, v[i]);
              }
            }
            if (head < G) {
              const float f = L > 0.f || L != L ? 1.f / L : 0.f;
              const int64_t at = (static_cast<int64_t>(w.s) * a.num_q_heads + w.h * G + head) * D + 64 * hh + 8 * g + 4 * t;
              if (a.out_bf16)
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) =
                    make_uint2(pack_bf16(v[0] * f, v[1] * f), pack_bf16(v[2] * f, v[3] * f));
              else
                *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) =
                    make_float4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
            }
          }
          cluster_barrier();  // the others' shared memory has been read
          return;
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

// Ring depth: about 100 to 130 KB of pages on their way per SM.  That is already
// twice what the latency needs at the memory's rate, and what lies beyond it only
// queues, unevenly: the warps served last at the start finish last.  Deeper against
// these: d 128, two stages of two pages in 12 warps instead of 8: 64 contexts of up to 16k
// 176 us for 164, 64 ragged sequences 48.9 for 47.5, one of 8192 12.7 for 10.8; d 64,
// three stages instead of two in the 12 warps of long steps: 32 contexts of up to 8k
// 30.8 us for 30.4, 128 of up to 32k 327.3 for 326.7.
//
// d 64, long steps: one CTA of 12 warps per SM instead of four of 4 (the warp
// scheduler shares an SM evenly between a CTA's warps but prefers older CTAs): 32 contexts
// of up to 8k 33.2 -> 30.5 us, 128 of up to 32k 327.2 -> 326.8.  Chosen when the page
// bound -- sequences x ceil(max context / 16) x KV heads -- reaches
// kLongPagesPerWarp per warp (those 32 contexts have 72): with 36, 64 contexts of up to 2048 lose
// (20.7 -> 21.1) and 32 of up to 4096 win (20.9 -> 20.2).  d 128 takes one CTA of 8 warps always.
constexpr int64_t kLongPagesPerWarp = 64;

inline int64_t page_bound(const DecodeArgs &a) {
  return static_cast<int64_t>(a.num_seqs) * ((static_cast<int64_t>(a.ctx_cap) + kBlockSize - 1) / kBlockSize) *
         a.num_kv_heads;
}

// When items are few and long, a CTA of four warps takes each: the piece count
// of a row is bounded by the partition size (the workspace has no more slots), so
// an idle GPU does not shorten them.  Teams are used where the least piece, or an
// item without a workspace, has
//  * 8 pages, without a workspace 4, and all items fit the GPU as CTAs at once (one
//    context of 1024 in pieces of 8 pages, d 64 6.8 -> 5.1 us, d 128 9.6 -> 6.1;
//    of 2 pages 4.9 -> 5.3, d 128 6.1 -> 6.6);
//  * 16 pages, with more items: pieces as long as the workspace allows must leave
//    warps idle (16 contexts of 2048 in partitions of 512, d 64 25.5 -> 11.9 us, d 128
//    27.1 -> 19.7; 60 ragged ones of up to 1000 23.2 -> 16.5 and 32.9 -> 23.5; in partitions of 256
//    16 of 2048 15.8 -> 15.7, but d 128 18.2 -> 19.7), items without a
//    workspace at most two to a CTA.  With 8 pages 16 of 2048 lose: 11.7 -> 15.6.
// (All taken with the clusters below left out, which have most of these steps.)
constexpr int kTeamPages = 8, kTeamItemPages = 4, kTeamManyPages = 16;

template <bool BAL>
inline bool team_step(const DecodeArgs &a, int64_t items, int64_t ctas, int warps_per_cta) {
  const int longest = (a.partition_size < a.ctx_cap ? a.partition_size : a.ctx_cap) / kBlockSize;
  if (items <= ctas) return longest >= (BAL ? kTeamPages : kTeamItemPages);
  if (longest < kTeamManyPages || a.num_kv_heads > ctas / 4) return false;
  return BAL ? page_bound(a) <= ctas * warps_per_cta * (a.partition_size / kBlockSize) : items <= 2 * ctas;
}

enum class Int8Fit { kAlways, kLongSteps, kTeams };  // when launch_int8_kern takes a step

template <int D, int PP, int ST, int NW, int MIN_CTAS, bool BAL, Int8Fit FIT>
cudaError_t launch_int8_kern(const DecodeArgs &a, unsigned int *err, cudaStream_t stream, bool *taken) {
  constexpr bool TEAM = FIT == Int8Fit::kTeams;
  constexpr int SMEM = Int8Ring<D, PP, ST, NW>::SMEM;
  auto kern = paged_decode_int8_kernel<D, PP, ST, NW, MIN_CTAS, BAL, TEAM ? Mode::kTeams : Mode::kWarps>;
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
  *taken = FIT == Int8Fit::kAlways ||
           (FIT == Int8Fit::kTeams && team_step<BAL>(a, items, ctas_cap, NW)) ||
           (FIT == Int8Fit::kLongSteps && items >= warps_cap && page_bound(a) >= kLongPagesPerWarp * warps_cap);
  if (!*taken || items == 0) return cudaSuccess;
  const int64_t workers = std::min(items, TEAM ? ctas_cap : warps_cap);
  const int64_t grid = TEAM ? workers : (workers + NW - 1) / NW;
  DecodeArgs la = a;
  la.balanced = BAL ? 1 : 0;
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(NW * 32), SMEM, stream, la, err);
}

// Short steps: a cluster of up to eight CTAs takes the whole context of a sequence
// and KV head and merges in distributed shared memory: no pieces bounded by the
// partition size, no partials in memory, no second launch.  (Decode and merge ->
// cluster: one context of 1024 4.9 -> 4.1 us, d 128 6.2 -> 5.2; four of 4096 9.5 -> 7.6
// and 13.1 -> 10.0; 16 of 2048 11.7 -> 10.1 and 18.4 -> 14.7; 64 ragged ones of up to
// 256 11.6 -> 5.4 and 14.9 -> 8.2, of up to 1024 15.1 -> 13.0 and 22.4 -> 21.7; 300 of up to 700
// 37.9 -> 29.4 and 54.8 -> 45.0.)  What it costs is evenness: a warp's share follows the longest
// context.  So it is taken while no warp has more than kClusterPages pages at the
// declared longest one (16 ragged contexts of up to 4096, d 64, 16 pages, partitions of 128:
// 15.0 against 14.2; 8 of up to 16384, 32 pages: 24.6 against 21.8), and, where the clusters leave
// more than half of the SMs idle, than 16 KB (one of 8192, d 128, 8 pages: 9.9 against 9.3).
constexpr int kClusterMax = 8, kClusterPages = 16, kClusterFewBytes = 16384;

template <int D, int PP, int NW>
cudaError_t launch_int8_cluster(const DecodeArgs &a, unsigned int *err, cudaStream_t stream, bool *taken) {
  constexpr int ST = 2, SMEM = Int8Ring<D, PP, ST, NW>::SMEM;
  constexpr int MIN_CTAS = PP == 1 ? 4 : 1;
  auto kern = paged_decode_int8_kernel<D, PP, ST, NW, MIN_CTAS, false, Mode::kCluster>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(NW * 32);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // Clusters of 1, 2, 4 and 8 CTAs that the device holds at once, per device; 0 = not set up
  // (races repeat it).  Fewer than its CTAs would make: a cluster lies within one GPC.
  static std::atomic<int> resident[64][4];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (resident[dev][0].load(std::memory_order_acquire) == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 1;
    for (int i = 3; i >= 0; --i) {  // the first entry last: it says that the others are there
      attr[0].val.clusterDim.x = 1 << i;
      cfg.gridDim = dim3(1 << i);
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
      if (e != cudaSuccess) return e;
      resident[dev][i].store(std::max(n, 1), std::memory_order_release);
    }
  }
  const int64_t sms = device_sm_count(), pairs = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  const int64_t pages = (static_cast<int64_t>(a.ctx_cap) + kBlockSize - 1) / kBlockSize;
  static_assert(kClusterMax == 8, "resident has an entry for each width");
  int width = 3;  // of a cluster, log2: all resident at once, a step's pages at least per warp
  while (width > 0 && (pairs > resident[dev][width].load(std::memory_order_relaxed) || (NW * PP << width) > pages)) --width;
  const int ctas = 1 << width;
  const int64_t share = (pages + ctas * NW - 1) / (ctas * NW);
  *taken = share <= kClusterPages && (2 * pairs * ctas >= sms || share * int8_record_bytes(D) <= kClusterFewBytes + 512);
  if (!*taken || pairs == 0) return cudaSuccess;
  cfg.gridDim = dim3(static_cast<unsigned>(pairs * ctas));
  attr[0].val.clusterDim.x = ctas;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, err);
}

// The cluster's width: 8 warps per CTA while the pairs of sequence and KV head are few,
// so that a pair finds as many warps as possible; 4 where whole contexts per CTA fill
// the GPU (d 64, 512 pairs of 600 tokens: 9.7 us, 12.8 with 8 warps); in d 128 steps of one
// page and so four CTAs per SM for yet more pairs (512 pairs of 600 tokens: 17.0, 19.5 with steps of
// two; with the registers of three CTAs 21.4, but 64 ragged contexts of up to 1000 20.4 against 21.4).
template <int D>
cudaError_t launch_int8_clusters(const DecodeArgs &a, unsigned int *err, cudaStream_t stream, bool *taken) {
  const int64_t sms = device_sm_count(), pairs = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
  if constexpr (D == 64) {
    return pairs <= 3 * sms ? launch_int8_cluster<D, 2, 8>(a, err, stream, taken)
                            : launch_int8_cluster<D, 2, 4>(a, err, stream, taken);
  } else {
    return pairs <= sms       ? launch_int8_cluster<D, 2, 8>(a, err, stream, taken)
           : pairs <= 3 * sms ? launch_int8_cluster<D, 2, 4>(a, err, stream, taken)
                              : launch_int8_cluster<D, 1, 4>(a, err, stream, taken);
  }
}

// *whole: every row is written, nothing to merge.
template <int D, bool BAL>
cudaError_t launch_int8(const DecodeArgs &a, unsigned int *err, cudaStream_t stream, bool *whole) {
  cudaError_t e = launch_int8_clusters<D>(a, err, stream, whole);
  if (e != cudaSuccess || *whole) return e;
  bool taken = false;
  e = launch_int8_kern<D, 2, 2, 4, 1, BAL, Int8Fit::kTeams>(a, err, stream, &taken);
  if (e != cudaSuccess || taken) return e;
  if constexpr (D == 64) {
    if constexpr (BAL) {
      e = launch_int8_kern<D, 2, 2, 12, 1, true, Int8Fit::kLongSteps>(a, err, stream, &taken);
      if (e != cudaSuccess || taken) return e;
    }
    return launch_int8_kern<D, 2, 2, 4, 4, BAL, Int8Fit::kAlways>(a, err, stream, &taken);
  } else {
    return launch_int8_kern<D, 2, 2, 8, 1, BAL, Int8Fit::kAlways>(a, err, stream, &taken);
  }
}

template <int D>
cudaError_t dispatch_int8(const DecodeArgs &a, unsigned int *err, cudaStream_t st, bool *whole) {
  return balanced_pieces(a) ? launch_int8<D, true>(a, err, st, whole) : launch_int8<D, false>(a, err, st, whole);
}

}  // namespace

cudaError_t launch_decode_partial_int8(const DecodeArgs &a, unsigned int *err, cudaStream_t st, bool *whole) {
  *whole = false;
  if (a.head_dim == 64) return dispatch_int8<64>(a, err, st, whole);
  if (a.head_dim == 128) return dispatch_int8<128>(a, err, st, whole);
  return cudaErrorInvalidValue;
}

}  // namespace photon
