// Step metadata built on the GPU: what block_meta.cpp's
// photon_build_step_metadata does on the host, from request lengths and a
// free-block stack that live in device memory (sm_103a).
//
// With nc computed and nn new tokens, sequence s holds h = ceil(nc / 16)
// blocks and needs ceil((nc + nn) / 16); three exclusive prefix sums over the
// sequences (tokens, blocks grown, blocks released) then place everything:
//   token t of sequence s (tok_s <= t < tok_{s+1}) has position nc + t - tok_s;
//   the a-th block grown overall is stack[free + R - 1 - a], R the blocks
//   released, which are pushed first, in order of sequence and row.
// Everything after the sums is one flat loop per list (tokens, grown blocks,
// released blocks), a binary search in shared memory naming the sequence, so
// long prompts and thousands of one-token sequences cost the same per entry.
//
// The kernel never lets a dependent grid start early: the decode kernels read
// block tables and context lengths before their own dependency wait.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace photon {
namespace {

constexpr int kMetaThreads = 1024;

// Last index s in [0, n) with off[s] <= x (off ascending, off[0] <= x).
__device__ __forceinline__ int owner(const int32_t *off, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ unsigned long long scan_warp(unsigned long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

__global__ void __launch_bounds__(kMetaThreads) step_metadata_kernel(const StepMetaArgs a, unsigned int *err) {
  extern __shared__ int32_t offs[];  // [3][num_seqs]: tokens, blocks grown, blocks released
  const int B = a.num_seqs;
  int32_t *tok = offs, *gro = offs + B, *rel = offs + 2 * B;
  __shared__ unsigned long long wsum[2][32];
  __shared__ int s_max, s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  if (tid == 0) s_max = s_bad = 0;
  __syncthreads();

  // ---- prefix sums (tokens in one word; grown and released blocks in another)
  unsigned long long tok_base = 0, blk_base = 0;
  for (int b0 = 0; b0 < B; b0 += kMetaThreads) {
    const int s = b0 + tid;
    unsigned long long n = 0, blk = 0;
    int ctx = 0;
    bool bad = false;
    if (s < B) {
      const int64_t nc = a.num_computed[s], nn = a.num_new[s];
      const int64_t have = (nc + kBlockSize - 1) / kBlockSize;
      const int64_t need = (nc + nn + kBlockSize - 1) / kBlockSize;
      bad = nc < 0 || nc + nn > INT32_MAX || have > a.max_blocks_per_seq ||
            (nn >= 0 && need > a.max_blocks_per_seq);
      if (!bad) {
        if (nn >= 0) {
          n = static_cast<unsigned long long>(nn);
          blk = static_cast<unsigned long long>(need - have);
          ctx = static_cast<int>(nc + nn);
        } else {
          blk = static_cast<unsigned long long>(have) << 32;
        }
      }
    }
    const unsigned long long n_in = scan_warp(n, lane), blk_in = scan_warp(blk, lane);
    if (lane == 31) {
      wsum[0][warp] = n_in;
      wsum[1][warp] = blk_in;
    }
    const int wmax = __reduce_max_sync(0xffffffffu, ctx);
    const int wbad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      if (wmax > 0) atomicMax(&s_max, wmax);
      if (wbad) s_bad = 1;
    }
    __syncthreads();
    if (warp < 2) wsum[warp][lane] = scan_warp(wsum[warp][lane], lane);
    __syncthreads();
    if (s < B) {
      const unsigned long long t = tok_base + n_in - n + (warp ? wsum[0][warp - 1] : 0);
      const unsigned long long k = blk_base + blk_in - blk + (warp ? wsum[1][warp - 1] : 0);
      tok[s] = static_cast<int32_t>(t < INT32_MAX ? t : INT32_MAX);
      gro[s] = static_cast<int32_t>(k & 0xffffffffu);
      rel[s] = static_cast<int32_t>(k >> 32);
    }
    tok_base += wsum[0][31];
    blk_base += wsum[1][31];
    __syncthreads();
  }
  const int64_t A = static_cast<int64_t>(blk_base & 0xffffffffu), R = static_cast<int64_t>(blk_base >> 32);
  const int64_t nf = *a.num_free;
  int status = PHOTON_OK;
  if (s_bad || tok_base > static_cast<unsigned long long>(a.max_tokens) || nf < 0 || nf + R > a.num_blocks)
    status = PHOTON_ERR_INVALID_ARG;
  else if (A > nf + R)
    status = PHOTON_ERR_POOL_EXHAUSTED;
  const bool ok = status == PHOTON_OK;
  const int T = ok ? static_cast<int>(tok_base) : 0;

  // ---- released blocks go on the stack, their row entries back to -1
  if (ok)
    for (int j = tid; j < R; j += kMetaThreads) {
      const int s = owner(rel, B, j);
      int32_t *entry = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq + (j - rel[s]);
      const int32_t id = *entry;
      if (id < 0 || id >= a.num_blocks) atomicOr(err, PHOTON_DEVERR_BLOCK_RANGE);
      a.free_blocks[nf + j] = id;
      *entry = -1;
    }
  __syncthreads();
  const int32_t *top = a.free_blocks + (nf + R - 1);  // the next block handed out

  // ---- grown blocks
  if (ok)
    for (int j = tid; j < A; j += kMetaThreads) {
      const int s = owner(gro, B, j);
      const int have = (a.num_computed[s] + kBlockSize - 1) / kBlockSize;
      a.block_tables[static_cast<int64_t>(s) * a.max_blocks_per_seq + have + (j - gro[s])] = __ldcg(top - j);
    }

  // ---- tokens (slots past the step's tokens: position -1, slot -1)
  for (int t = tid; t < a.max_tokens; t += kMetaThreads) {
    int s = 0, p = -1;
    int64_t slot = -1;
    if (t < T) {
      s = owner(tok, B, t);
      const int nc = a.num_computed[s];
      p = nc + (t - tok[s]);
      const int have = (nc + kBlockSize - 1) / kBlockSize, b = p / kBlockSize;
      const int32_t id = b < have ? a.block_tables[static_cast<int64_t>(s) * a.max_blocks_per_seq + b]
                                  : __ldcg(top - (gro[s] + b - have));
      if (id >= 0 && id < a.num_blocks)
        slot = static_cast<int64_t>(id) * kBlockSize + p % kBlockSize;
      else
        atomicOr(err, PHOTON_DEVERR_BLOCK_RANGE);
    }
    a.token_seq[t] = s;
    a.positions[t] = p;
    a.slot_mapping[t] = slot;
  }
  for (int s = tid; s < B; s += kMetaThreads) {
    const int nn = a.num_new[s];
    a.context_lens[s] = ok && nn >= 0 ? a.num_computed[s] + nn : 0;
  }
  if (tid == 0) {
    a.totals[0] = T;
    a.totals[1] = ok ? s_max : 0;
    a.totals[2] = static_cast<int32_t>(ok ? nf + R - A : nf);
    a.totals[3] = status;
    *a.num_free_out = a.totals[2];
    if (!ok) atomicOr(err, PHOTON_DEVERR_METADATA);
  }
  __threadfence();  // a dependent grid may read these before its own dependency wait
}

}  // namespace

cudaError_t launch_step_metadata(const StepMetaArgs &a, unsigned int *err, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(a.num_seqs) * 12;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(step_metadata_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kStepMetaMaxSeqs * 12);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(step_metadata_kernel, dim3(1), dim3(kMetaThreads), smem, st, a, err);
}

}  // namespace photon
