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
// One cluster of up to sixteen CTAs: every CTA computes all sums itself (reading
// 8 bytes per sequence) and takes its share of the flat loops, so the only
// exchange is a cluster barrier between the pushes onto the stack and the reads
// from it, and behind it one word per CTA: whether its share of the released
// rows names a block outside the pool.  The barriers are passed whatever the
// step holds, so CTAs that saw different lengths (changed under the kernel)
// still meet.  The loops' searches and loads are latency, not bandwidth:
// kMetaBatch entries of a thread run at once.
//
// The kernel never lets a dependent grid start early: the decode kernels read
// block tables and context lengths before their own dependency wait.
#include <atomic>
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace photon {
namespace {

constexpr int kMetaThreads = 1024;

constexpr int kMetaMaxCtas = 16;  // of a cluster; 8 where the GPU has no room for one of 16
constexpr int kMetaBatch = 4;

// The last index s in [0, n) with off[s] <= x (off ascending, off[0] <= x).
__device__ __forceinline__ int owner(const int32_t *off, int n, int x) {
  int s = 0;
  for (int step = n > 1 ? 1 << (31 - __clz(n - 1)) : 0; step > 0; step >>= 1)
    if (s + step < n && off[s + step] <= x) s += step;
  return s;
}

// The same for a warp's 32 ascending x, none owned before `from`: the next 32
// starts are one load, a lane finds its own among them by shuffles, and a
// warp inside one sequence (long prompts) needs neither.
__device__ __forceinline__ int warp_owner(const int32_t *off, int n, int x, int from, int lane) {
  int s = -1;
  for (;; from += 32) {
    const int next = from + 1 + lane < n ? off[from + 1 + lane] : INT_MAX;
    const int v0 = __shfl_sync(0xffffffffu, next, 0);  // every lane takes part, found or not
    if (__all_sync(0xffffffffu, s >= 0 || x < v0)) return s >= 0 ? s : from;
    int pos = 0;  // starts at or before x in the window
#pragma unroll
    for (int step = 16; step > 0; step >>= 1)
      if (__shfl_sync(0xffffffffu, next, pos + step - 1) <= x) pos += step;
    const bool past = __shfl_sync(0xffffffffu, next, 31) <= x;
    if (s < 0 && !past) s = from + pos;
    if (__all_sync(0xffffffffu, s >= 0)) return s;
  }
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

// A word of the same place in another CTA's shared memory.
__device__ __forceinline__ int cluster_load(const int *mine, int cta) {
  unsigned at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(mine)), "r"(cta));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ unsigned long long scan_warp(unsigned long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Lengths of sequence s: new tokens, blocks grown (low word) or released (high
// word), context; false for lengths that the step must refuse.
__device__ __forceinline__ bool step_lengths(const StepMetaArgs &a, int s, unsigned long long &n,
                                             unsigned long long &blk, int &ctx) {
  const int64_t nc = a.num_computed[s], nn = a.num_new[s];
  const int64_t have = (nc + kBlockSize - 1) / kBlockSize;
  const int64_t need = (nc + nn + kBlockSize - 1) / kBlockSize;
  n = blk = 0;
  ctx = 0;
  if (nc < 0 || nc + nn > INT32_MAX || have > a.max_blocks_per_seq ||
      (nn >= 0 && need > a.max_blocks_per_seq))
    return false;
  if (nn >= 0) {
    n = static_cast<unsigned long long>(nn);
    blk = static_cast<unsigned long long>(need - have);
    ctx = static_cast<int>(nc + nn);
  } else {
    blk = static_cast<unsigned long long>(have) << 32;
  }
  return true;
}

__global__ void __launch_bounds__(kMetaThreads) step_metadata_kernel(const StepMetaArgs a, unsigned int *err) {
  extern __shared__ int32_t offs[];  // [3][num_seqs]: tokens, blocks grown, blocks released
  constexpr int N = kMetaBatch;
  const int B = a.num_seqs;
  int32_t *tok = offs, *gro = offs + B, *rel = offs + 2 * B;
  __shared__ unsigned long long wsum[2][32];
  __shared__ int s_max, s_bad, s_foreign;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int warps = static_cast<int>(blockDim.x >> 5);
  const int gtid = blockIdx.x * blockDim.x + tid, threads = gridDim.x * blockDim.x;
  pdl_wait();
  if (tid == 0) s_max = s_bad = s_foreign = 0;
  __syncthreads();

  // ---- prefix sums (tokens in one word; grown and released blocks in
  // another), each thread `per` neighbouring sequences
  const int per = (B + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
  const int first = min(tid * per, B), last = min(first + per, B);
  unsigned long long n_sum = 0, blk_sum = 0;
  int ctx_max = 0;
  bool bad = false;
  for (int s = first; s < last; ++s) {
    unsigned long long n, blk;
    int ctx;
    bad |= !step_lengths(a, s, n, blk, ctx);
    n_sum += n;
    blk_sum += blk;
    ctx_max = max(ctx_max, ctx);
  }
  const int64_t nf = *a.num_free;
  const unsigned long long n_in = scan_warp(n_sum, lane), blk_in = scan_warp(blk_sum, lane);
  if (lane == 31) {
    wsum[0][warp] = n_in;
    wsum[1][warp] = blk_in;
  }
  ctx_max = __reduce_max_sync(0xffffffffu, ctx_max);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    if (ctx_max > 0) atomicMax(&s_max, ctx_max);
    if (bad) s_bad = 1;
  }
  __syncthreads();
  if (warp < 2) wsum[warp][lane] = scan_warp(lane < warps ? wsum[warp][lane] : 0ull, lane);
  __syncthreads();
  unsigned long long at_n = n_in - n_sum + (warp ? wsum[0][warp - 1] : 0);
  unsigned long long at_blk = blk_in - blk_sum + (warp ? wsum[1][warp - 1] : 0);
  for (int s = first; s < last; ++s) {
    tok[s] = static_cast<int32_t>(at_n < INT32_MAX ? at_n : INT32_MAX);
    gro[s] = static_cast<int32_t>(at_blk & 0xffffffffu);
    rel[s] = static_cast<int32_t>(at_blk >> 32);
    unsigned long long n, blk;
    int ctx;
    step_lengths(a, s, n, blk, ctx);
    at_n += n;
    at_blk += blk;
  }
  const unsigned long long total = wsum[0][31];
  const int64_t A = static_cast<int64_t>(wsum[1][31] & 0xffffffffu), R = static_cast<int64_t>(wsum[1][31] >> 32);
  int status = PHOTON_OK;
  if (s_bad || total > static_cast<unsigned long long>(a.max_tokens) || nf < 0 || nf + R > a.num_blocks)
    status = PHOTON_ERR_INVALID_ARG;
  else if (A > nf + R)
    status = PHOTON_ERR_POOL_EXHAUSTED;
  __syncthreads();  // the sums

  // ---- released blocks go above the stack, cells that nothing holds yet, and
  // their row entries back to -1; a block from outside the pool refuses the step,
  // and the entries return from those cells
  const bool sound = status != PHOTON_ERR_INVALID_ARG, fits = status == PHOTON_OK;
  if (sound)
    for (int j = gtid; j < R; j += threads) {
      const int s = owner(rel, B, j);
      int32_t *entry = a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq + (j - rel[s]);
      const int32_t id = *entry;
      if (id < 0 || id >= a.num_blocks) s_foreign = 1;
      a.free_blocks[nf + j] = id;
      if (fits) *entry = -1;
    }
  // the stack is complete, and every CTA has read the lengths' sums and the count
  if (gridDim.x > 1) cluster_sync(); else __syncthreads();
  bool foreign = false;
  if (sound && R > 0)
    foreign = gridDim.x > 1 ? __any_sync(0xffffffffu, lane < static_cast<int>(gridDim.x) &&
                                                          cluster_load(&s_foreign, lane) != 0)
                            : s_foreign != 0;
  if (gridDim.x > 1) cluster_arrive();  // this CTA's reads are done; waited for at the end
  if (foreign) status = PHOTON_ERR_INVALID_ARG;
  const bool ok = status == PHOTON_OK;
  const int T = ok ? static_cast<int>(total) : 0;
  if (foreign && fits)
    for (int j = gtid; j < R; j += threads) {  // the thread's own cells
      const int s = owner(rel, B, j);
      a.block_tables[static_cast<int64_t>(s) * a.max_blocks_per_seq + (j - rel[s])] = a.free_blocks[nf + j];
    }
  const int32_t *top = a.free_blocks + (nf + R - 1);  // the next block handed out

  // ---- grown blocks
  if (ok)
    for (int j = gtid; j < A; j += threads) {
      const int s = owner(gro, B, j);
      const int have = (a.num_computed[s] + kBlockSize - 1) / kBlockSize;
      a.block_tables[static_cast<int64_t>(s) * a.max_blocks_per_seq + have + (j - gro[s])] = __ldcg(top - j);
    }

  // ---- tokens, a span of up to 32 N neighbours per warp
  const int turns = min(N, (T + threads - 1) / threads);
  for (int64_t base = static_cast<int64_t>(gtid >> 5) * (32 * turns); base < T;
       base += static_cast<int64_t>(threads) * turns) {
    int x[N], s[N], nc[N], p[N];
    int from = owner(tok, B, static_cast<int>(base));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = static_cast<int>(min(base + 32 * i + lane, static_cast<int64_t>(T - 1)));
      s[i] = from;
      if (i >= turns) continue;
      s[i] = warp_owner(tok, B, x[i], from, lane);
      from = __shfl_sync(0xffffffffu, s[i], 31);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) nc[i] = i < turns ? a.num_computed[s[i]] : 0;
    int32_t id[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      id[i] = -1;
      p[i] = 0;
      if (i >= turns) continue;  // s[i] need not own x[i]: its row may not reach that far, nor the stack
      p[i] = nc[i] + (x[i] - tok[s[i]]);
      const int have = (nc[i] + kBlockSize - 1) / kBlockSize, b = p[i] / kBlockSize;
      id[i] = __ldcg(b < have ? a.block_tables + static_cast<int64_t>(s[i]) * a.max_blocks_per_seq + b
                              : top - (gro[s[i]] + b - have));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t t = base + 32 * i + lane;
      if (i >= turns || t >= T) continue;
      const bool valid = id[i] >= 0 && id[i] < a.num_blocks;
      if (!valid) atomicOr(err, PHOTON_DEVERR_BLOCK_RANGE);
      a.token_seq[t] = s[i];
      a.positions[t] = p[i];
      a.slot_mapping[t] = valid ? static_cast<int64_t>(id[i]) * kBlockSize + p[i] % kBlockSize : -1;
    }
  }
  // slots past the step's tokens
  for (int64_t t = static_cast<int64_t>(T) + gtid; t < a.max_tokens; t += threads) {
    a.token_seq[t] = 0;
    a.positions[t] = -1;
    a.slot_mapping[t] = -1;
  }
  for (int s = gtid; s < B; s += threads) {
    const int nn = a.num_new[s];
    a.context_lens[s] = ok && nn >= 0 ? a.num_computed[s] + nn : 0;
  }
  if (gtid == 0) {
    const int32_t left = static_cast<int32_t>(ok ? nf + R - A : nf);
    a.totals[0] = T;
    a.totals[1] = ok ? s_max : 0;
    a.totals[2] = left;
    a.totals[3] = status;
    *a.num_free_out = left;
    if (!ok) atomicOr(err, PHOTON_DEVERR_METADATA | (foreign ? PHOTON_DEVERR_BLOCK_RANGE : 0u));
  }
  if (gridDim.x > 1) cluster_wait();  // no CTA leaves while another may read its word
  __threadfence();  // a dependent grid may read these before its own dependency wait
}

}  // namespace

namespace {

// The largest cluster of this kernel that the current device can hold (16, else
// the portable 8), and the kernel's shared memory allowance; looked up once per device.
cudaError_t max_cluster(int *ctas) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  *ctas = known[dev].load(std::memory_order_relaxed);
  if (*ctas) return cudaSuccess;
  e = cudaFuncSetAttribute(step_metadata_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStepMetaMaxSeqs * 12);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(step_metadata_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kMetaMaxCtas);
  cfg.blockDim = dim3(kMetaThreads);
  cfg.dynamicSmemBytes = kStepMetaMaxSeqs * 12;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kMetaMaxCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, step_metadata_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();  // no answer: the portable size
    clusters = 0;
  }
  *ctas = clusters > 0 ? kMetaMaxCtas : 8;
  known[dev].store(*ctas, std::memory_order_relaxed);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_step_metadata(const StepMetaArgs &a, unsigned int *err, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(a.num_seqs) * 12;
  // A CTA for every 2048 entries of the longer list (65536 tokens of 2048
  // sequences: 71 us with one CTA, 12.0 with eight, 9.1 with sixteen, 9.7 with the word per CTA); up to 256
  // entries, 256 threads start and meet sooner than 1024 (4.6 us for 64 sequences, 5.0).
  const int64_t entries = a.max_tokens > a.num_seqs ? a.max_tokens : a.num_seqs;
  int most = 0;
  const cudaError_t e = max_cluster(&most);
  if (e != cudaSuccess) return e;
  unsigned ctas = 1;
  while (ctas * int64_t{2048} < entries && ctas < static_cast<unsigned>(most)) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(entries <= 256 ? 256 : kMetaThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, step_metadata_kernel, a, err);
}

}  // namespace photon
