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
// tokens of one block, next to each other in the call.  A warp takes one run's K or
// V of one head, 16 rows by offset, with one reduction for m; of runs of one token,
// several heads at once.  A CTA walks tiles of tokens and takes the runs that begin in
// them, all heads, over one (cos, sin) table per tile.
//
// Two runs of one block in a call would race for its scale. Nothing orders them; where a
// tile's 32 tokens, or those of a call of at most 256, show them, an error bit does.
//
// What bounds it: latency at 16 (d 64) or 8 (d 128) warps per SM, whose rows fill the
// registers, and an uneven last round of tiles; neither memory nor the issue slots (active half
// of the time).  16384 tokens of 8 x 64, bf16, take 16.4 us for 50 MB (7.4 at the copy rate;
// 13.4 without the rotation): 1024 tiles over 304 CTAs, so some CTAs walk four where 3.4 would do.
// 65536 tokens, 13.5 tiles a CTA, 52.8 us, 0.56 of the copy rate; 8192 of 8 x 128 18.1 us; 64 tokens
// of a decode step 3.9 us, two dependent loads and a launch.  Of a run's 2 x heads units a warp
// takes whole ones: with one KV head two warps of a CTA work (16384 tokens of 1 x 64 10.2 us, 1 x 128 18.4,
// where 4 heads take 11.3 and 20.5).  The read is bound by DRAM, two thirds of it
// writes: 32768 tokens of 8 x 128 34.2 us, 0.87 of the copy rate.
#include <climits>

#include "int8.cuh"
#include "norm_rope.cuh"

namespace photon {
namespace {

constexpr int kInt8Warps = 8;
constexpr int kInt8MaxTile = 16;                       // tokens of a CTA
constexpr int kInt8TableRows = kInt8MaxTile + kBlockSize - 1;  // its last run may pass the tile's end
static_assert(32 * kInt8Warps == kNormThreads, "query tiles run in the same CTAs");

constexpr float kCodeMagic = 12582912.f + 128.f;  // fma(y, r, this): low byte = rne(y r) + 128

// Codes + 128 of eight values, value i in byte i.
__device__ __forceinline__ uint2 codes8(const float2 (&y)[4], float r) {
  const float2 rr = make_float2(r, r), magic = make_float2(kCodeMagic, kCodeMagic);
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __ffma2_rn(y[i], rr, magic);
    b[i] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x0040u);
  }
  return make_uint2(__byte_perm(b[0], b[1], 0x5410u), __byte_perm(b[2], b[3], 0x5410u));
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

// A run of several tokens as a warp sees it: lane o (0 .. 15) holds the token of row
// o, as an index into the tile's tokens (-1: not written).
struct Run {
  int block;
  uint32_t written;  // a bit per row
  int src, any;      // any: the first token
};

// fl(m / 127) in fp32's normal range: a product, its exact residual, one
// correction (equal to the division for every mantissa; tests/test_int8_host.py).
__device__ __forceinline__ float div127(float m) {
  constexpr float kInv = 1.f / 127.f;
  const float q = __fmul_rn(m, kInv);
  return __fmaf_rn(__fmaf_rn(-127.f, q, m), kInv, q);
}

// A row's scale after a write whose largest magnitude is m, and what follows from it.
struct Scale {
  float value, inv, ratio;  // ratio: for the codes of kept rows, where `grows`
  bool some, grows;
};
__device__ __forceinline__ Scale new_scale(float m, float old) {
  Scale s;
  const float quo = div127(m), want = quo < kInt8Least ? 0.f : quo;
  const bool finite = m <= 3.4028234663852886e38f;
  s.grows = finite && want > old;
  s.value = !finite ? __uint_as_float(0x7fffffffu) : s.grows ? fmaxf(want, 2.f * old) : old;
  s.some = s.value > 0.f;
  s.inv = s.some ? __frcp_rn(s.value) : 0.f;
  s.ratio = __fmul_rn(old, s.inv);
  s.grows = s.grows && old > 0.f;
  return s;
}

__device__ __forceinline__ float max_abs_row(const LaneRow &y) {
  float m = max_abs3(y.a[0].x, y.a[0].y, y.b[0].x);
  m = max_abs3(m, y.b[0].y, y.a[1].x);
  m = max_abs3(m, y.a[1].y, y.b[1].x);
  m = max_abs3(m, y.b[1].y, y.a[2].x);
  m = max_abs3(m, y.a[2].y, y.b[2].x);
  m = max_abs3(m, y.b[2].y, y.a[3].x);
  m = max_abs3(m, y.a[3].y, y.b[3].x);
  return max_abs3(m, y.b[3].y, 0.f);
}

constexpr uint2 kZeroCodes = {0x80808080u, 0x80808080u};

template <typename Tag, int D, bool NORM>
struct Write8 {
  using T = typename Tag::T;
  using R = RopeRow<D>;
  static constexpr int RPP = 32 / R::LPR, PASSES = kBlockSize / RPP;  // rows of a pass
  static_assert(RPP == 8 || RPP == 4, "head_dim 64 or 128");

  // Unit u of a run is K (0) or V (1) of head (or heads) u / 2.  Every eighth unit is a
  // warp's: the two take turns, K's rotation costs what would leave V's warps waiting.
  __device__ __forceinline__ static int which(int u) { return (u ^ (u >> 3)) & 1; }

  __device__ __forceinline__ static unsigned char *record(const NormRopeArgs &a, int block, int h) {
    return static_cast<unsigned char *>(a.k_cache) +
           (static_cast<int64_t>(block) * a.num_kv_heads + h) * int8_record_bytes(D);
  }
  template <int WHICH>
  __device__ __forceinline__ static int byte_of(int row, int e) {
    return WHICH ? int8_v_byte(D, row, e) : int8_k_byte(row, e);
  }

  // Norm (NORM) and rotation of a K row, V as it is.
  template <int WHICH>
  __device__ __forceinline__ static void prepare(const NormRopeArgs &a, LaneRow &y, const RowLoad<T> &weight, int w,
                                                 const float *row) {
    if constexpr (!WHICH) {
      const bool gptj = a.rope_style == PHOTON_ROPE_GPTJ, rotate = a.rope_style != PHOTON_ROPE_NONE;
      const RowAt<D> at{row, w};
      if constexpr (NORM) {
        norm_rope_row<T, D>(y, weight, a.eps, rotate, at, gptj);
      } else if (rotate) {
        rotate_row(y, at, gptj);
      }
    }
  }

  // A lane's 16 codes of a row that the call does not write.
  template <int WHICH>
  __device__ __forceinline__ static void keep_row(unsigned char *rec, int row, int w, bool anew, float ratio) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint2 *at = reinterpret_cast<uint2 *>(rec + byte_of<WHICH>(row, 8 * w + half * R::HALF));
      if (anew) {
        *at = kZeroCodes;
      } else {
        float c[8];
        codes_to_f32(*at, c);
        const float2 f[4] = {make_float2(c[0], c[1]), make_float2(c[2], c[3]), make_float2(c[4], c[5]),
                             make_float2(c[6], c[7])};
        *at = codes8(f, ratio);
      }
    }
  }

  // ---- a run of several tokens: K (V: WHICH 1) of one head is a warp's unit of
  // work, 16 rows by offset.  A lane holds 16 dims of one row per pass, rows 0, 1, 4,
  // 5, 2, 3, 6, 7 and those + 8 in the order of the warp's row groups, so that the V
  // bytes of half a warp fill whole 32-byte sectors; everything but a lane's first
  // addresses is a constant.  All rows stay in registers, in fp32, from the scale to
  // the codes: taking them twice from shared memory, with the registers of 24 warps
  // per SM instead of 16, measured 16.1 -> 19.7 us (16384 tokens, 8 heads of 64).

  // Row of pass p: that of pass 0 and this.
  __device__ __forceinline__ static constexpr int row_step(int p) { return RPP == 8 ? 8 * p : 2 * (p & 1) + 8 * (p >> 1); }
  __device__ __forceinline__ static int first_row(int lane) {
    const int i = lane / R::LPR;
    return (i & 1) | ((i >> 1) & 2) | ((i << 1) & 4);
  }
  __device__ __forceinline__ static constexpr uint32_t rows(int p) {
    return RPP == 8 ? 0xffu << (8 * p) : 0x33u << row_step(p);
  }
  // Bytes of pass p and half `half` of the dims past those of pass 0, dims 8w.
  template <int WHICH>
  __device__ __forceinline__ static constexpr int byte_step(int p, int half) {
    return WHICH ? 32 * (row_step(p) >> 3) + 512 * (row_step(p) >> 1 & 1) + half * (D == 64 ? 256 : 1024)
                 : 256 * (row_step(p) >> 3) + 512 * (row_step(p) >> 1 & 1) + half * (D == 64 ? 32 : 1024);
  }

  struct Unit {
    RowLoad<T> raw[PASSES];
    float old;  // the block's scale so far
  };

  // Starts unit u's loads.  Rows that are not written take the run's first token:
  // their values go nowhere.
  __device__ __forceinline__ static void load(Unit &unit, const NormRopeArgs &a, const Run &run, int t0, int u,
                                              int lane) {
    const T *x = static_cast<const T *>(which(u) ? a.v : a.k) +
                 (static_cast<int64_t>(t0) * a.num_kv_heads + (u >> 1)) * D + 8 * (lane % R::LPR);
    const int token = a.num_kv_heads * D;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if (!(run.written & rows(p))) continue;
      const int src = __shfl_sync(0xffffffffu, run.src, first_row(lane) + row_step(p));
      unit.raw[p].load(x + static_cast<int64_t>(src < 0 ? run.any : src) * token, R::HALF);
    }
    unit.old = run.written & 1u
                   ? 0.f
                   : *reinterpret_cast<const float *>(record(a, run.block, u >> 1) + int8_scale_byte(D, which(u)));
  }

  template <int WHICH>
  __device__ __forceinline__ static void write(const NormRopeArgs &a, const Run &run, int h, int lane,
                                               LaneRow (&y)[PASSES], float old, const float (*cs)[R::STRIDE]) {
    const int w = lane % R::LPR, row0 = first_row(lane);
    const bool anew = run.written & 1u;
    float m = 0.f;
    RowLoad<T> weight;
    if (NORM && !WHICH) weight = load_weights<T>(a.k_weight, w, R::HALF);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if (!(run.written & rows(p))) continue;
      const int src = WHICH ? 0 : __shfl_sync(0xffffffffu, run.src, row0 + row_step(p));
      prepare<WHICH>(a, y[p], weight, w, cs[src < 0 ? run.any : src]);
      const float top = max_abs_row(y[p]);
      if (run.written >> (row0 + row_step(p)) & 1u) m = max_abs3(m, top, 0.f);
      asm volatile("" ::: "memory");  // the next pass's table chunks are not fetched early: they would spill
    }
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));  // a NaN's bits are the largest
    const Scale s = new_scale(m, old);
    unsigned char *rec = record(a, run.block, h);
    if (lane == 0) *reinterpret_cast<float *>(rec + int8_scale_byte(D, WHICH)) = s.value;
    unsigned char *at = rec + byte_of<WHICH>(row0, 8 * w);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if (!(run.written & rows(p))) continue;
      const uint2 lo = s.some ? codes8(y[p].a, s.inv) : kZeroCodes, hi = s.some ? codes8(y[p].b, s.inv) : kZeroCodes;
      if (run.written >> (row0 + row_step(p)) & 1u) {
        *reinterpret_cast<uint2 *>(at + byte_step<WHICH>(p, 0)) = lo;
        *reinterpret_cast<uint2 *>(at + byte_step<WHICH>(p, 1)) = hi;
      }
    }
    if (run.written == 0xffffu || !(anew || s.grows)) return;
#pragma unroll 1
    for (int row = lane / R::LPR; row < kBlockSize; row += RPP)
      if (!(run.written >> row & 1u)) keep_row<WHICH>(rec, row, w, anew, s.ratio);
  }

  // ---- a run of one token: K or V of as many heads as the warp has row groups, one
  // row each.  (As runs of several, 28 of 32 lanes would have no work: 2048 tokens
  // of a decode step, 8 heads of 64, 17.0 us.)
  struct Single {
    RowLoad<T> raw;
    float old;
  };
  __device__ __forceinline__ static int groups(const NormRopeArgs &a) { return (a.num_kv_heads + RPP - 1) / RPP; }

  // token: its index in the call.  Heads past the last take the last one's row.
  __device__ __forceinline__ static void load_single(Single &s, const NormRopeArgs &a, int64_t token, int block, int off,
                                                     int u, int lane) {
    const int h = min((u >> 1) * RPP + lane / R::LPR, a.num_kv_heads - 1);
    s.raw.load(static_cast<const T *>(which(u) ? a.v : a.k) + (token * a.num_kv_heads + h) * D + 8 * (lane % R::LPR),
               R::HALF);
    s.old = off == 0 ? 0.f : *reinterpret_cast<const float *>(record(a, block, h) + int8_scale_byte(D, which(u)));
  }

  template <int WHICH>
  __device__ __forceinline__ static void write_single(const NormRopeArgs &a, const Single &in, int block, int off,
                                                      int group, int lane, const float *row) {
    const int w = lane % R::LPR, h = group * RPP + lane / R::LPR;
    RowLoad<T> weight;
    if (NORM && !WHICH) weight = load_weights<T>(a.k_weight, w, R::HALF);
    LaneRow y;
    widen_row(in.raw, y);
    prepare<WHICH>(a, y, weight, w, row);
    float m = max_abs_row(y);
#pragma unroll
    for (int o = R::LPR / 2; o > 0; o >>= 1) m = max_abs3(m, __shfl_xor_sync(0xffffffffu, m, o), 0.f);
    if (h < a.num_kv_heads) {
      const Scale s = new_scale(m, in.old);
      unsigned char *rec = record(a, block, h);
      if (w == 0) *reinterpret_cast<float *>(rec + int8_scale_byte(D, WHICH)) = s.value;
      unsigned char *at = rec + byte_of<WHICH>(off, 8 * w);
      *reinterpret_cast<uint2 *>(at) = s.some ? codes8(y.a, s.inv) : kZeroCodes;
      *reinterpret_cast<uint2 *>(at + byte_step<WHICH>(0, 1)) = s.some ? codes8(y.b, s.inv) : kZeroCodes;
      if (off == 0 || s.grows)
#pragma unroll 1
        for (int i = 0; i < kBlockSize; ++i)
          if (i != off) keep_row<WHICH>(rec, i, w, off == 0, s.ratio);
    }
    __syncwarp();
  }
};

// CTAs per SM that the write's registers allow.
constexpr int int8_write_ctas(int head_dim) { return head_dim == 64 ? 2 : 1; }

// The first kv_ctas CTAs walk the tiles of tokens, the others take a query tile
// each.  A tile's slots and positions are loaded one tile ahead, a unit's rows and
// scale one unit ahead, across runs and tiles.
template <typename Tag, int D, bool NORM>
__global__ void __launch_bounds__(kNormThreads, int8_write_ctas(D))
    kv_cache_write_int8_kernel(const __grid_constant__ NormRopeArgs a, int kv_ctas, int tiles, unsigned int *err) {
  using R = RopeRow<D>;
  using W = Write8<Tag, D, NORM>;
  __shared__ __align__(16) float cs[2][kInt8TableRows][R::STRIDE];  // of this tile and the next
  pdl_wait();
  pdl_launch_dependents();
  if constexpr (NORM) {
    if (static_cast<int>(blockIdx.x) >= kv_ctas) {
      norm_rope_q_tile<Tag, D>(a, blockIdx.x - kv_ctas, cs[0]);
      return;
    }
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int units = 2 * a.num_kv_heads;  // K and V of every head, over the warps
  const bool rotate = a.rope_style != PHOTON_ROPE_NONE;
  // The open tile: lane i looks at token t0 - 1 + i.  A run's length is at most a
  // block's 16, so the runs that begin in a tile of 16 end within the 32 tokens.
  // singles, leaders: where runs of one, of several tokens begin.
  int tile = static_cast<int>(blockIdx.x) - kv_ctas, t0 = 0, block = 0, off = 0, pos = 0, first = 0, last = 0;
  uint32_t joined = 0, rising = 0, leaders = 0, singles = 0;
  int64_t slot1 = -1;  // of the next tile
  int pos1 = 0;
  auto fetch = [&](int k) {
    const int64_t t = (static_cast<int64_t>(k) << a.tile_log2) - 1 + lane;
    const bool in = k < tiles && t >= 0 && t < a.num_tokens;
    slot1 = in ? a.slot_mapping[t] : -1;
    pos1 = in && rotate ? a.positions[t] : 0;
  };
  // tokens that follow lane i in its run
  auto follow = [&](int i) { return min(__ffs(~(joined >> (i + 1))) - 1, kBlockSize - 1); };
  Run run;
  auto take_run = [&]() {
    const int i = __ffs(leaders) - 1, n = follow(i);
    leaders &= leaders - 1;
    run.block = __shfl_sync(0xffffffffu, block, i);
    run.any = i - 1;
    const int o = __shfl_sync(0xffffffffu, off, i);
    const uint32_t rest = ((1u << n) - 1) << (i + 1);
    if ((rising & rest) == rest) {  // offsets in order: the rule
      run.written = ((2u << n) - 1) << o;
      run.src = lane >= o && lane <= o + n ? i - 1 + lane - o : -1;
    } else {  // the last token of those with a row's slot
      run.written = 0;
      run.src = -1;
      for (int j = 0; j <= n; ++j) {
        const int at = __shfl_sync(0xffffffffu, off, i + j);
        if (lane == at) run.src = i - 1 + j;
        run.written |= 1u << at;
      }
    }
  };
  typename W::Unit unit{};
  // `unit` holds the warp's first unit of the open tile's runs of several tokens; else,
  // as its first row, that of the runs of one token
  bool have = false;
  auto load_single = [&](int j) {  // the warp's j-th unit of the runs of one token
    typename W::Single s;
    const int n = 2 * W::groups(a);
    uint32_t left = singles;
    for (; j >= n; j -= n) left &= left - 1;
    const int i = __ffs(left) - 1;
    W::load_single(s, a, static_cast<int64_t>(t0) - 1 + i, __shfl_sync(0xffffffffu, block, i),
                   __shfl_sync(0xffffffffu, off, i), j, lane);
    return s;
  };
  // Opens the CTA's next tile in which a run begins, the same in every warp, and
  // starts the warp's first loads there.
  auto next_tile = [&]() -> bool {
    for (tile += kv_ctas; tile < tiles; tile += kv_ctas) {
      int64_t slot = slot1;
      pos = pos1;
      fetch(tile + kv_ctas);
      t0 = tile << a.tile_log2;
      const bool own = lane >= 1 && lane <= 1 << a.tile_log2;
      if (slot >= a.num_slots) {
        if (warp == 0 && own) atomicOr(err, PHOTON_DEVERR_SLOT_RANGE);
        slot = -1;
      }
      const bool live = slot >= 0;
      block = live ? static_cast<int>(slot >> 4) : -1;
      off = static_cast<int>(slot) & (kBlockSize - 1);
      const int before = __shfl_up_sync(0xffffffffu, block, 1);
      const bool same = lane > 0 && live && before == block;
      if (warp == 0) {  // a block's second run in the window
        const uint32_t alike = __match_any_sync(0xffffffffu, block);
        if (live && !same && (alike & ((1u << lane) - 1))) atomicOr(err, PHOTON_DEVERR_BLOCK_ORDER);
      }
      joined = __ballot_sync(0xffffffffu, same);
      const int off_before = __shfl_up_sync(0xffffffffu, off, 1);
      rising = __ballot_sync(0xffffffffu, off_before + 1 == off);
      leaders = __ballot_sync(0xffffffffu, own && live && !same);
      if (!leaders) continue;
      first = __ffs(leaders) - 1;  // the tile's runs cover lanes first .. last
      last = 31 - __clz(leaders);
      last += follow(last);
      singles = leaders & ~(joined >> 1);
      leaders &= ~singles;
      have = leaders && warp < units;
      if (have) {
        take_run();
        W::load(unit, a, run, t0, warp, lane);
      } else if (warp < __popc(singles) * 2 * W::groups(a)) {
        const typename W::Single s = load_single(warp);
        unit.raw[0] = s.raw;
        unit.old = s.old;
      }
      return true;
    }
    return false;
  };
  fetch(blockIdx.x);
  // a short call's tokens, one per thread: its blocks' second runs are found wherever they are
  const bool all_seen = a.num_tokens <= kNormThreads;
  const int64_t my_slot = all_seen && static_cast<int>(threadIdx.x) < a.num_tokens ? a.slot_mapping[threadIdx.x] : -1;
  if (!next_tile()) return;
  if (all_seen) {
    for (int i = 1; i <= 1 << a.tile_log2; ++i) {
      const int b = __shfl_sync(0xffffffffu, block, i), end = i + __ffs(~(joined >> (i + 1))) - 1;
      // (a run that reaches the window's end repeats slots)
      if (b >= 0 && my_slot >> 4 == b && end < 31 && static_cast<int>(threadIdx.x) > t0 - 1 + end)
        atomicOr(err, PHOTON_DEVERR_BLOCK_ORDER);
    }
  }
  for (int buf = 0;; buf ^= 1) {
    if (rotate) {
      rope_table_rows<D>(cs[buf] + (first - 1), last + 1 - first, a.turns, a.rope_style == PHOTON_ROPE_GPTJ,
                         [&](int t) { return __shfl_sync(0xffffffffu, pos, first + t); });
      __syncthreads();  // the table of the tile before last is free: its readers passed the barrier since
    }
    const int n1 = 2 * W::groups(a);
    for (int j = warp; j < __popc(singles) * n1; j += kInt8Warps) {
      typename W::Single s{unit.raw[0], unit.old};
      if (j != warp || have) s = load_single(j);
      uint32_t left = singles;
      int u = j;
      for (; u >= n1; u -= n1) left &= left - 1;
      const int i = __ffs(left) - 1;
      const int b = __shfl_sync(0xffffffffu, block, i), o = __shfl_sync(0xffffffffu, off, i);
      if (W::which(u))
        W::template write_single<1>(a, s, b, o, u >> 1, lane, cs[buf][i - 1]);
      else
        W::template write_single<0>(a, s, b, o, u >> 1, lane, cs[buf][i - 1]);
    }
    bool more = true;  // there is another tile
    if (!have) {
      more = next_tile();
    } else {
      for (int u = warp;;) {
        LaneRow y[W::PASSES];
#pragma unroll
        for (int p = 0; p < W::PASSES; ++p) widen_row(unit.raw[p], y[p]);
        const float old = unit.old;
        const Run now = run;
        const int u0 = u;
        bool open = true;
        u += kInt8Warps;
        if (u >= units) {
          u = warp;
          if (leaders)
            take_run();
          else
            open = false;
        }
        if (open)
          W::load(unit, a, run, t0, u, lane);
        else
          more = next_tile();
        if (W::which(u0))
          W::template write<1>(a, now, u0 >> 1, lane, y, old, cs[buf]);
        else
          W::template write<0>(a, now, u0 >> 1, lane, y, old, cs[buf]);
        if (!open) break;
      }
    }
    if (!more) return;
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
cudaError_t launch_write(NormRopeArgs a, bool norm, unsigned int *err, cudaStream_t st) {
  // tokens per tile: as few as leave no whole tile more than there are resident CTAs, up to 16
  // (777 fp32 tokens of 4 x 128: 5.3 us, 8.6 with a quarter of them in a tile, three tiles to a
  // CTA).  A ragged tile beyond them is walked second by one CTA; counted too, it would double
  // all tiles: 1217 tokens of 8 x 128, singles 8.2 -> 12.7 us, a prompt 6.0 -> 7.2, though 609
  // singles of 8 x 64 4.7 -> 4.3.
  const int64_t room = static_cast<int64_t>(device_sm_count()) * int8_write_ctas(D);
  a.tile_log2 = 0;
  while ((1 << a.tile_log2) < kInt8MaxTile && (static_cast<int64_t>(a.num_tokens) >> a.tile_log2) > room) ++a.tile_log2;
  const int64_t tiles = (static_cast<int64_t>(a.num_tokens) + (1 << a.tile_log2) - 1) >> a.tile_log2;
  const int64_t kv_ctas = tiles < room ? tiles : room, ctas = kv_ctas + a.q_tiles;
  if (ctas == 0) return cudaSuccess;
  if (ctas > INT32_MAX || tiles + kv_ctas > INT32_MAX) return cudaErrorInvalidValue;
  auto kern = norm ? kv_cache_write_int8_kernel<Tag, D, true> : kv_cache_write_int8_kernel<Tag, D, false>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kNormThreads), 0, st, a,
                    static_cast<int>(kv_ctas), static_cast<int>(tiles), err);
}

}  // namespace

// Query rows from which they get a launch of their own, in the bf16 / fp32 write's
// kernel, whose registers leave 32 warps per SM to this one's 16 (d 64) or 8 (d 128).  d 64:
// 524288 rows, with 16384 tokens, 44.8 -> 42.9 us, 262144 24.4 against 24.5; d 128: 131072 rows,
// with 8192 tokens, 44.1 -> 37.2, 65536 18.3 against 19.0.
constexpr int64_t query_rows_apart(int head_dim) { return head_dim == 64 ? 524288 : 131072; }

cudaError_t launch_kv_cache_write_int8(NormRopeArgs a, bool norm, photon_dtype in_dt, int head_dim,
                                       unsigned int *err, cudaStream_t st) {
  if (static_cast<int64_t>(a.num_q_tokens) * a.num_q_heads >= query_rows_apart(head_dim)) {
    NormRopeArgs q = a;
    q.num_tokens = 0;
    const cudaError_t e = launch_qk_norm_rope_write(q, in_dt, head_dim, err, st);
    if (e != cudaSuccess) return e;
    a.num_q_tokens = 0;
  }
  a.q_tile_log2 = norm_tile_log2(a.num_q_tokens, 3);
  a.q_tiles = static_cast<int>((static_cast<int64_t>(a.num_q_tokens) + (1 << a.q_tile_log2) - 1) >> a.q_tile_log2);
  if (head_dim == 64)
    return in_dt == PHOTON_BF16 ? launch_write<BF16Tag, 64>(a, norm, err, st) : launch_write<F32Tag, 64>(a, norm, err, st);
  return in_dt == PHOTON_BF16 ? launch_write<BF16Tag, 128>(a, norm, err, st) : launch_write<F32Tag, 128>(a, norm, err, st);
}

cudaError_t launch_kv_cache_read_int8(const CacheReadArgs &a, photon_dtype out_dt, unsigned int *err,
                                      cudaStream_t st) {
  if (a.num_tokens == 0) return cudaSuccess;
  return out_dt == PHOTON_BF16 ? launch_read<BF16Tag>(a, err, st) : launch_read<F32Tag>(a, err, st);
}

}  // namespace photon
