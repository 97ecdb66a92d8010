// Rows of head_dim values spread over head_dim / 16 neighbouring lanes: lane w
// of a row holds dims 8w .. 8w + 7 (x0) and those + D/2 (x1), so that both
// halves of every rotation pair, of either style, are in one lane.  Shared by
// the writes that normalise, rotate or quantise rows.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace photon {

// A lane's 16 values of a row as loaded.
template <typename T>
struct RowLoad {
  static constexpr int N = sizeof(T) / 2;
  uint4 lo[N], hi[N];
  __device__ __forceinline__ void load(const T *src, int half) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      lo[i] = reinterpret_cast<const uint4 *>(src)[i];
      hi[i] = reinterpret_cast<const uint4 *>(src + half)[i];
    }
  }
  __device__ __forceinline__ void store(T *dst, int half) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      reinterpret_cast<uint4 *>(dst)[i] = lo[i];
      reinterpret_cast<uint4 *>(dst + half)[i] = hi[i];
    }
  }
  __device__ __forceinline__ static void widen(const uint4 (&r)[N], float (&x)[8]) {
    if constexpr (N == 1) {
      Unpack<BF16Tag>::run(r[0], x);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[4 * i] = __uint_as_float(r[i].x);
        x[4 * i + 1] = __uint_as_float(r[i].y);
        x[4 * i + 2] = __uint_as_float(r[i].z);
        x[4 * i + 3] = __uint_as_float(r[i].w);
      }
    }
  }
};

// Eight values to the storage type, one rounding each.
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
  uint4 w;
  uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  *reinterpret_cast<uint4 *>(p) = w;
}

}  // namespace photon
