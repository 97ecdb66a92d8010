// Split-K paged decode attention over a 4-bit (E2M1) KV cache with one bf16
// scale per token and 64 head dims, head_dim 64 or 128, on the tensor cores.
// Record layout in fp4.cuh; partial / merge contract, work split and walker as
// the FP8 kernel's (paged_decode_mma.cuh).
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(x_j - m),  x_j = scale log2(e) <q, k_j>
//
//  * Records come straight from global memory into registers: every lane's
//    fragment chunk is one coalesced 16-byte load (K plane, V plane, scales),
//    so there is no shared-memory stage, barrier or fragment shuffle.  A step
//    covers PP pages.  K of the next step is loaded as soon as this step's
//    score MMAs have read their registers, V after its output MMAs.
//  * Codes convert to f16 exactly in hardware (cvt.rn.f16x2.e2m1x2).  The
//    scales never touch a code: a token's K scale multiplies its scores (per
//    64 dims), its V scale the probability that weights it.
//  * q enters as f16 after an exact power-of-two scaling of its row to
//    [1, 2), so any bf16 q keeps its 8 bits down to 2^-24 of the row's largest
//    value; the factor goes into the score scale, the scale's sign into q.
//  * P is kept relative to 2^(m + E - 13), E the largest exponent of a V scale
//    so far: p_j times its V scale then lies below 2^14 whatever the values'
//    magnitude, and rounds to f16 with relative error 2^-12 down to 2^-28 of
//    the largest.  For an fp32 output the remainder of that rounding follows
//    in a second MMA (SPLIT), for a bf16 output (half a step: 2^-9) it would
//    be lost anyway.  Sums, maxima and accumulators are fp32.
#include <atomic>
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "paged_decode.cuh"
#include "paged_decode_mma.cuh"

namespace photon {
namespace {

constexpr int kFp4Warps = 4;
// Least exponent of the V scales that P follows: p is then at most 2^103 and
// its sum over a context stays in fp32.
constexpr int kFp4MinExp = -90;

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

// 16 bytes of a record, read once: not kept in L1, first out of L2.
__device__ __forceinline__ uint4 ld_record(const unsigned char *p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.b32 {%0,%1,%2,%3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy));
  return v;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                   *reinterpret_cast<const __nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&m);
}

// One step of a warp's work: up to PP pages of one item.
struct Fp4Step {
  int s, h, p, P_s;
  int tok0, tok1;   // token of the step's first page; end of the item
  uint32_t valid;   // bit i: page i exists and its block id is in the pool
  bool first, last; // of its item
};

template <int D, int PP, bool BAL, bool SPLIT>
__global__ void __launch_bounds__(kFp4Warps * 32)
    paged_decode_fp4_kernel(const DecodeArgs a, unsigned int *err) {
  constexpr int HH = D / 64;
  constexpr int REC = fp4_record_bytes(D);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int G = a.num_q_heads / a.num_kv_heads;
  if constexpr (BAL) prefetch_tables_l2(a);
  pdl_launch_dependents();
  const uint64_t policy = l2_evict_first_policy();
  const int total_warps = gridDim.x * kFp4Warps;

  Walker w;
  walker_start<BAL>(w, a, lane, err, blockIdx.x * kFp4Warps + warp, total_warps);
  // metadata only so far; pages, q and the workspace wait for the preceding kernel
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.seg_count)  // the merge's mode
    a.seg_count[static_cast<int64_t>(a.num_seqs) * a.num_q_heads] = BAL ? 1 : 0;

  int bt_base = INT_MIN / 2, bt_reg = -1;  // lane j: block-table entry of page bt_base + j
  bool begun = false;                      // the walker's item has yielded a step
  const unsigned char *rec[PP];

  // Next step of the warp's stream into `st` and the records' addresses; an
  // item without pages is one step that writes the zero row.
  auto fetch = [&](Fp4Step &st) -> bool {
    if (w.valid && begun && w.page >= w.n_pages) {
      walker_next<BAL>(w, a, lane, err, total_warps);
      bt_base = INT_MIN / 2;
      begun = false;
    }
    if (!w.valid) return false;
    st.s = w.s;
    st.h = w.h;
    st.p = w.p;
    st.P_s = w.P_s;
    st.tok0 = (w.pg0 + w.page) * kBlockSize;
    st.tok1 = w.tok1;
    st.first = !begun;
    st.valid = 0;
    if (w.page < w.n_pages && w.page + PP - bt_base > 32) {
      bt_base = w.page;
      bt_reg = bt_base + lane < w.n_pages
                   ? a.block_tables[seq_table_row(a, w.s) * a.max_blocks_per_seq + w.pg0 + bt_base + lane]
                   : -1;
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const int blk = __shfl_sync(0xffffffffu, bt_reg, (w.page + i - bt_base) & 31);
      const bool in = w.page + i < w.n_pages;
      const bool ok = in && blk >= 0 && blk < a.num_blocks;
      bad |= in && !ok;
      st.valid |= ok ? 1u << i : 0u;
      rec[i] = static_cast<const unsigned char *>(a.k_cache) +
               (static_cast<int64_t>(ok ? blk : 0) * a.num_kv_heads + w.h) * REC + 16 * lane;
    }
    if (bad && lane == 0) atomicOr(err, PHOTON_DEVERR_BLOCK_RANGE);
    begun = true;
    w.page += PP;
    st.last = w.page >= w.n_pages;
    return true;
  };

  uint4 kr[PP][HH], vr[PP][HH], sr[PP][HH];
  auto load_k = [&](uint32_t valid) {
#pragma unroll
    for (int i = 0; i < PP; ++i)
#pragma unroll
      for (int hh = 0; hh < HH; ++hh) {
        kr[i][hh] = sr[i][hh] = make_uint4(0u, 0u, 0u, 0u);
        if (valid >> i & 1u) {
          kr[i][hh] = ld_record(rec[i] + 512 * hh, policy);
          sr[i][hh] = ld_record(rec[i] + 16 * D + 64 * hh + 16 * c - 16 * lane, policy);
        }
      }
  };
  auto load_v = [&](uint32_t valid) {
#pragma unroll
    for (int i = 0; i < PP; ++i)
#pragma unroll
      for (int hh = 0; hh < HH; ++hh) {
        vr[i][hh] = make_uint4(0u, 0u, 0u, 0u);
        if (valid >> i & 1u) vr[i][hh] = ld_record(rec[i] + 8 * D + 512 * hh, policy);
      }
  };

  Fp4Step cur, nxt;
  bool have = fetch(cur);
  if (have) {
    load_k(cur.valid);
    load_v(cur.valid);
  }

  uint32_t qa[HH][4][2];
  float o[HH][4][4];
  float m_run = -INFINITY, m_ref = -INFINITY, l_run = 0.f, sl = 0.f;
  int e_run = kFp4MinExp;

  while (have) {
    if (cur.first) {
      float f[HH][16], qm = 0.f;
#pragma unroll
      for (int hh = 0; hh < HH; ++hh)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (g < G)
            v = reinterpret_cast<const uint4 *>(
                static_cast<const __nv_bfloat16 *>(a.q) +
                (static_cast<int64_t>(cur.s) * a.num_q_heads + cur.h * G + g) * D + 64 * hh + 16 * c)[i];
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
      float down = __uint_as_float(static_cast<uint32_t>(127 - max(e, -126)) << 23);  // 2^-e
      if (e == 127) down = 0x1p-127f;
      sl = fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      if (a.scale_log2 < 0.f) down = -down;
      if (sl == 0.f) {  // all scores 0, by way of q: a masked token's -inf must stay one
        sl = 1.f;
        down = 0.f;
      }
#pragma unroll
      for (int hh = 0; hh < HH; ++hh)
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          qa[hh][kt][0] = pack_half2(f[hh][4 * kt] * down, f[hh][4 * kt + 1] * down);
          qa[hh][kt][1] = pack_half2(f[hh][4 * kt + 2] * down, f[hh][4 * kt + 3] * down);
        }
#pragma unroll
      for (int hh = 0; hh < HH; ++hh)
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) o[hh][mt][0] = o[hh][mt][1] = o[hh][mt][2] = o[hh][mt][3] = 0.f;
      m_run = m_ref = -INFINITY;
      l_run = 0.f;
      e_run = kFp4MinExp;
    }

    // ---- scores of head g: x[i][2n + j] belongs to token 4c + 2n + j of page i
    float x[PP][4];
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      float acc[HH][2][4];
#pragma unroll
      for (int hh = 0; hh < HH; ++hh)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          uint32_t kw[8];
          uint32_t(&lo)[4] = reinterpret_cast<uint32_t(&)[4]>(kw[0]);
          uint32_t(&hi)[4] = reinterpret_cast<uint32_t(&)[4]>(kw[4]);
          e2m1x8_to_f16(n ? kr[i][hh].z : kr[i][hh].x, lo);
          e2m1x8_to_f16(n ? kr[i][hh].w : kr[i][hh].y, hi);
          float(&s)[4] = acc[hh][n];
          s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
          for (int kt = 0; kt < 4; ++kt)
            mma_f16(s, qa[hh][kt][0], 0u, qa[hh][kt][1], 0u, kw[2 * kt], kw[2 * kt + 1]);
        }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint32_t s0 = n ? sr[i][0].y : sr[i][0].x;
        x[i][2 * n] = acc[0][n][0] * bf16_lo(s0);
        x[i][2 * n + 1] = acc[0][n][1] * bf16_hi(s0);
        if constexpr (HH == 2) {
          const uint32_t s1 = n ? sr[i][HH - 1].y : sr[i][HH - 1].x;
          x[i][2 * n] = fmaf(acc[HH - 1][n][0], bf16_lo(s1), x[i][2 * n]);
          x[i][2 * n + 1] = fmaf(acc[HH - 1][n][1], bf16_hi(s1), x[i][2 * n + 1]);
        }
      }
    }
    uint32_t sv[PP][HH][2];  // V scales of tokens (4c, 4c+1), (4c+2, 4c+3)
#pragma unroll
    for (int i = 0; i < PP; ++i)
#pragma unroll
      for (int hh = 0; hh < HH; ++hh) {
        sv[i][hh][0] = sr[i][hh].z;
        sv[i][hh][1] = sr[i][hh].w;
      }
    const uint32_t valid = cur.valid;
    const bool have_next = fetch(nxt);
    if (have_next) load_k(nxt.valid);

    if (valid) {  // no page of the step in the pool: nothing to add
      // tokens past the context, of absent pages: weight 0 (their bytes may hold anything)
      if (valid != (1u << PP) - 1 || cur.tok0 + PP * kBlockSize > cur.tok1) {
#pragma unroll
        for (int i = 0; i < PP; ++i) {
          const int nv = (valid >> i & 1u) ? cur.tok1 - (cur.tok0 + i * kBlockSize) : 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (4 * c + j >= nv) {
              x[i][j] = -INFINITY;
#pragma unroll
              for (int hh = 0; hh < HH; ++hh) sv[i][hh][j >> 1] &= (j & 1) ? 0x0000ffffu : 0xffff0000u;
            }
        }
      }
      float mx = x[0][0];
      uint32_t sm = sv[0][0][0];
#pragma unroll
      for (int i = 0; i < PP; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) mx = fmaxf(mx, x[i][j]);
#pragma unroll
        for (int hh = 0; hh < HH; ++hh) sm = max_bf16x2(sm, max_bf16x2(sv[i][hh][0], sv[i][hh][1]));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // exponent of the step's largest V scale (scales are not negative)
      const int es = static_cast<int>(__reduce_max_sync(0xffffffffu, max(sm & 0xffffu, sm >> 16)) >> 7) - 127;
      e_run = max(e_run, min(es, 127));
      m_run = fmaxf(m_run, mx * sl);
      const float ref = m_run + static_cast<float>(e_run - 13);
      const float alpha = exp2_approx(m_ref - ref);
      m_ref = ref;
      float ps = 0.f;
      uint32_t ph[PP][HH][2], pl[SPLIT ? PP : 1][HH][2];
#pragma unroll
      for (int i = 0; i < PP; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = exp2_approx(fmaf(x[i][2 * n], sl, -ref));
          const float p1 = exp2_approx(fmaf(x[i][2 * n + 1], sl, -ref));
          ps += p0 + p1;
#pragma unroll
          for (int hh = 0; hh < HH; ++hh) {
            const float w0 = p0 * bf16_lo(sv[i][hh][n]), w1 = p1 * bf16_hi(sv[i][hh][n]);
            ph[i][hh][n] = pack_half2(w0, w1);
            if constexpr (SPLIT) {
              const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&ph[i][hh][n]));
              pl[i][hh][n] = pack_half2(w0 - r.x, w1 - r.y);
            }
          }
        }
      l_run = fmaf(l_run, alpha, ps);
      if (__any_sync(0xffffffffu, alpha != 1.f)) {
        const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * c);
        const float a1 = __shfl_sync(0xffffffffu, alpha, 8 * c + 4);
#pragma unroll
        for (int hh = 0; hh < HH; ++hh)
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            o[hh][mt][0] *= a0;
            o[hh][mt][1] *= a1;
            o[hh][mt][2] *= a0;
            o[hh][mt][3] *= a1;
          }
      }
      // ---- O^T += V^T P^T: words of tokens 4c .. 4c+3, nibble i = dim 8g + i.
      // Pairing the same nibble of two tokens in one byte gives the f16 pairs
      // (token, token + 1) of the MMA's A operand directly.
#pragma unroll
      for (int i = 0; i < PP; ++i)
#pragma unroll
        for (int hh = 0; hh < HH; ++hh) {
          const uint4 v = vr[i][hh];
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
    if (have_next) load_v(nxt.valid);

    if (cur.last) {
      float l = l_run;
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const float l0 = __shfl_sync(0xffffffffu, l, 8 * c);
      const float l1 = __shfl_sync(0xffffffffu, l, 8 * c + 4);
      const float m0 = __shfl_sync(0xffffffffu, m_ref, 8 * c);
      const float m1 = __shfl_sync(0xffffffffu, m_ref, 8 * c + 4);
      // o[hh][mt][2r + j]: head 2c + j, dim 64 hh + 8g + 2 mt + r
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int head = 2 * c + j;
        if (head >= G) continue;
        const float lj = j ? l1 : l0;
        const int64_t qrow = static_cast<int64_t>(cur.s) * a.num_q_heads + cur.h * G + head;
        if constexpr (BAL)
          if (g == 0 && cur.p == 0) a.seg_count[qrow] = cur.P_s;
        const bool whole = cur.P_s == 1;
        const float f = whole ? (lj > 0.f || lj != lj ? 1.f / lj : 0.f) : 1.f;
        const int64_t prow = qrow * a.max_partitions + cur.p;
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
          a.m_part[prow] = j ? m1 : m0;
          a.l_part[prow] = lj;
        }
      }
    }
    cur = nxt;
    have = have_next;
  }
}

template <int D, int PP, bool BAL, bool SPLIT>
cudaError_t launch_fp4_kern(const DecodeArgs &a, unsigned int *err, cudaStream_t stream) {
  auto kern = paged_decode_fp4_kernel<D, PP, BAL, SPLIT>;
  static std::atomic<int> occupancy[64];  // per device; 0 = not looked up (races repeat it)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  int occ = occupancy[dev].load(std::memory_order_relaxed);
  if (occ == 0) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, kFp4Warps * 32, 0);
    if (e != cudaSuccess) return e;
    occ = occ > 0 ? occ : 1;
    occupancy[dev].store(occ, std::memory_order_relaxed);
  }
  const int64_t items = static_cast<int64_t>(a.num_seqs) * a.max_partitions * a.num_kv_heads;
  const int64_t warps_cap = static_cast<int64_t>(device_sm_count()) * occ * kFp4Warps;
  const int64_t warps = items < warps_cap ? items : warps_cap;
  const int grid = static_cast<int>((warps + kFp4Warps - 1) / kFp4Warps);
  if (grid == 0) return cudaSuccess;
  DecodeArgs la = a;
  la.balanced = BAL ? 1 : 0;
  return launch_pdl(kern, dim3(grid), dim3(kFp4Warps * 32), 0, stream, la, err);
}

template <int D, int PP>
cudaError_t launch_fp4(const DecodeArgs &a, unsigned int *err, cudaStream_t stream) {
  const bool bal = balanced_pieces(a);
  if (a.out_bf16)
    return bal ? launch_fp4_kern<D, PP, true, false>(a, err, stream)
               : launch_fp4_kern<D, PP, false, false>(a, err, stream);
  return bal ? launch_fp4_kern<D, PP, true, true>(a, err, stream)
             : launch_fp4_kern<D, PP, false, true>(a, err, stream);
}

}  // namespace

cudaError_t launch_decode_partial_fp4(const DecodeArgs &a, unsigned int *err, cudaStream_t st) {
  switch (a.head_dim) {
    case 64: return launch_fp4<64, 4>(a, err, st);
    case 128: return launch_fp4<128, 2>(a, err, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace photon
