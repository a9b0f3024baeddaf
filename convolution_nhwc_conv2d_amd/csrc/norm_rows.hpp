// Rows of channels held by the threads of a workgroup: what layer norm and the
// root-mean-square norm share.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

#include "seq_common.hpp"

namespace cnhwc {
namespace seq {

__device__ __forceinline__ int64_t row_offset(int64_t row, int32_t l, const int64_t (&s)[2]) {
  if (l == 1) return row * s[0];
  const int64_t n = row / l;
  return n * s[0] + (row - n * l) * s[1];
}

// Sum over the TPR threads of a row, in every one of them.  Rows of more than
// one wavefront own the whole workgroup; `slot` alternates between calls so one
// barrier per call is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*red)[16], int slot) {
  if constexpr (TPR <= 64) {
    return group_sum<TPR>(v);
  } else {
    v = group_sum<64>(v);
    if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[slot][0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) s += red[slot][i];
    return s;
  }
}

// Two sums at once.
template <int TPR>
__device__ __forceinline__ void row_sums(float& v, float& w, float (*red)[2][16], int slot) {
  v = group_sum<(TPR < 64 ? TPR : 64)>(v);
  w = group_sum<(TPR < 64 ? TPR : 64)>(w);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) {
      red[slot][0][threadIdx.x >> 6] = v;
      red[slot][1][threadIdx.x >> 6] = w;
    }
    __syncthreads();
    v = red[slot][0][0], w = red[slot][1][0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) v += red[slot][0][i], w += red[slot][1][i];
  }
}

// The largest over the TPR threads of a row, in every one of them.
template <int TPR>
__device__ __forceinline__ float row_max(float v, float (*red)[16], int slot) {
  v = group_max<(TPR < 64 ? TPR : 64)>(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[slot][0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) v = __builtin_fmaxf(v, red[slot][i]);
  }
  return v;
}

// Calls f with the smallest register tile that holds `vecs` vectors, of at
// most REGS elements per thread (WIDE with 1024 threads, which share the
// registers of four times as many wavefronts); false if there is none.
template <int NV, int TPR>
struct Tile {
  static constexpr int nv = NV, tpr = TPR;
};
template <int VE, int REGS, int WIDE, typename F>
bool with_tile(int64_t vecs, F&& f) {
  if (vecs <= 8) { f(Tile<1, 8>{}); return true; }
  if (vecs <= 16) { f(Tile<1, 16>{}); return true; }
  if (vecs <= 32) { f(Tile<1, 32>{}); return true; }
  if (vecs <= 64) { f(Tile<1, 64>{}); return true; }
  if (vecs <= 128) { f(Tile<2, 64>{}); return true; }
  if (vecs <= 256) { f(Tile<1, 256>{}); return true; }
  if (vecs <= 512) { f(Tile<2, 256>{}); return true; }
  if (vecs <= 1024) { f(Tile<4, 256>{}); return true; }
  if constexpr (VE * 8 <= REGS) {
    if (vecs <= 2048) { f(Tile<8, 256>{}); return true; }
  }
  if constexpr (VE * 2 <= WIDE) {
    if (vecs <= 2048) { f(Tile<2, 1024>{}); return true; }
  }
  if constexpr (VE * 4 <= WIDE) {
    if (vecs <= 4096) { f(Tile<4, 1024>{}); return true; }
  }
  if constexpr (VE * 8 <= WIDE) {
    if (vecs <= 8192) { f(Tile<8, 1024>{}); return true; }
  }
  return false;
}

}  // namespace seq
}  // namespace cnhwc
