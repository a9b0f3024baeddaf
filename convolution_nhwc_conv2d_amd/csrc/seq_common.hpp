// Device helpers shared by the sequence kernels: element types, vector loads and
// stores, sums across lanes, and the scalar functions.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>
#include <type_traits>

#include "cnhwc_seq.h"

namespace cnhwc {
namespace seq {

template <int DT> struct ElemOf { using T = uint16_t; };
template <> struct ElemOf<CNHWC_F32> { using T = float; };
template <int DT> using Elem = typename ElemOf<DT>::T;

template <int DT>
__device__ __forceinline__ float to_f(Elem<DT> v) {
  if constexpr (DT == CNHWC_F32) return v;
  else if constexpr (DT == CNHWC_BF16) return __builtin_bit_cast(float, uint32_t(v) << 16);
  else return static_cast<float>(__builtin_bit_cast(_Float16, v));
}

// Round to nearest even; the 16-bit forms are single conversion instructions.
template <int DT>
__device__ __forceinline__ Elem<DT> from_f(float v) {
  if constexpr (DT == CNHWC_F32) return v;
  else if constexpr (DT == CNHWC_BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  else return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

// V consecutive elements: 16, 8 or 4 aligned bytes, or V is 1.
template <int DT, int V>
struct Pack { Elem<DT> e[V]; };
template <int DT, int V>
using PackBits = std::conditional_t<V * sizeof(Elem<DT>) == 16, uint4,
                                    std::conditional_t<V * sizeof(Elem<DT>) == 8, uint2, uint32_t>>;

template <int DT, int V>
__device__ __forceinline__ Pack<DT, V> load_pack(const Elem<DT>* p) {
  Pack<DT, V> r;
  if constexpr (V == 1) {
    r.e[0] = *p;
  } else {
    r = __builtin_bit_cast(Pack<DT, V>, *reinterpret_cast<const PackBits<DT, V>*>(p));
  }
  return r;
}

template <int DT, int V>
__device__ __forceinline__ void store_pack(Elem<DT>* p, const Pack<DT, V>& v) {
  if constexpr (V == 1) {
    *p = v.e[0];
  } else {
    *reinterpret_cast<PackBits<DT, V>*>(p) = __builtin_bit_cast(PackBits<DT, V>, v);
  }
}

// A parameter of dtype DT or fp32 (the choice is uniform over the launch).
template <int DT>
__device__ __forceinline__ float load_param(const void* p, int64_t i, bool f32) {
  if constexpr (DT == CNHWC_F32) return static_cast<const float*>(p)[i];
  else return f32 ? static_cast<const float*>(p)[i] : to_f<DT>(static_cast<const uint16_t*>(p)[i]);
}

// V consecutive parameters; vectors of V * sizeof(element of DT) = 16 bytes (32
// where they are fp32 beside a 16-bit DT), 16-byte aligned.
template <int DT, int V>
__device__ __forceinline__ void load_params(const void* p, int64_t i, bool f32, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = load_param<DT>(p, i, f32);
  } else {
    if (DT == CNHWC_F32 || f32) {
#pragma unroll
      for (int k = 0; k < V; k += 4) {
        const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + k);
        v[k] = f.x, v[k + 1] = f.y, v[k + 2] = f.z, v[k + 3] = f.w;
      }
    } else {
      const Pack<DT, V> r = load_pack<DT, V>(static_cast<const Elem<DT>*>(p) + i);
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = to_f<DT>(r.e[k]);
    }
  }
}

template <int DT>
__device__ __forceinline__ void store_param(void* p, int64_t i, bool f32, float v) {
  if constexpr (DT == CNHWC_F32) {
    static_cast<float*>(p)[i] = v;
  } else {
    if (f32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = from_f<DT>(v);
  }
}

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// ---------------------------------------------------------------- lanes

// v moved by a row-local lane permutation (every lane of the pattern is live).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kQuadReverse = 0x1B;  // lanes 1032, 2301, 3210 of a quad
constexpr int kHalfMirror = 0x141, kRowMirror = 0x140;    // reversed 8 or 16 lanes
constexpr int kRor8 = 0x128, kRor4 = 0x124;               // rows of 16 rotated
constexpr int kQuadBcast = 0x55;                          // times j: lane j of each quad

__device__ __forceinline__ float add_row_pairs(float v) {  // rows 0+1 and 2+3, in every lane
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return __builtin_bit_cast(float, uint32_t(r[0])) + __builtin_bit_cast(float, uint32_t(r[1]));
}
__device__ __forceinline__ float add_halves(float v) {  // lower and upper 32 lanes, in every lane
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, uint32_t(r[0])) + __builtin_bit_cast(float, uint32_t(r[1]));
}

// Sum over groups of G consecutive lanes, the same bits in each of them.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr (G >= 2) v += dpp<kQuadXor1>(v);
  if constexpr (G >= 4) v += dpp<kQuadXor2>(v);
  if constexpr (G >= 8) v += dpp<kHalfMirror>(v);
  if constexpr (G >= 16) v += dpp<kRowMirror>(v);
  if constexpr (G >= 32) v = add_row_pairs(v);
  if constexpr (G >= 64) v = add_halves(v);
  return v;
}

__device__ __forceinline__ float max_row_pairs(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return __builtin_fmaxf(__builtin_bit_cast(float, uint32_t(r[0])), __builtin_bit_cast(float, uint32_t(r[1])));
}
__device__ __forceinline__ float max_halves(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_fmaxf(__builtin_bit_cast(float, uint32_t(r[0])), __builtin_bit_cast(float, uint32_t(r[1])));
}

// The largest over groups of G consecutive lanes, in each of them; NaN is passed over.
template <int G>
__device__ __forceinline__ float group_max(float v) {
  if constexpr (G >= 2) v = __builtin_fmaxf(v, dpp<kQuadXor1>(v));
  if constexpr (G >= 4) v = __builtin_fmaxf(v, dpp<kQuadXor2>(v));
  if constexpr (G >= 8) v = __builtin_fmaxf(v, dpp<kHalfMirror>(v));
  if constexpr (G >= 16) v = __builtin_fmaxf(v, dpp<kRowMirror>(v));
  if constexpr (G >= 32) v = max_row_pairs(v);
  if constexpr (G >= 64) v = max_halves(v);
  return v;
}

// ---------------------------------------------------------------- functions

// e^x for x from -110 (where it is 0) to 88; the product with log2(e) is carried
// in two terms, so the relative error stays near one unit of the last place
// instead of growing with |x|.
__device__ __forceinline__ float exp_near(float x) {
  constexpr float hi = 1.44269502f, lo = 1.92596299e-8f;  // log2(e) = hi + lo
  const float t = x * hi;
  const float r = __builtin_fmaf(x, lo, __builtin_fmaf(x, hi, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, r * 0.693147181f, e);
}

// The same below -110 too (0, for minus infinity as well); NaN stays NaN.
__device__ __forceinline__ float exp_full(float x) { return exp_near(x < -110.0f ? -110.0f : x); }

// 1 / v for ordinary v: the hardware's estimate and one Newton step.
__device__ __forceinline__ float rcp_full(float v) {
  const float r = __builtin_amdgcn_rcpf(v);
  return __builtin_fmaf(r, __builtin_fmaf(-v, r, 1.0f), r);
}

// 1 / (1 + e^-x), from e = e^-|x| in (0, 1] (below 0: e / (1 + e)), so nothing
// overflows and the result falls to 0 with e: silu and its slope, which multiply
// it by x, are 0 for any finite x below -88.  (Held at a smallest value instead,
// it gave silu(-1e35) = -1.8.)  |x| is held at 110 by a minimum, one instruction
// where exp_full's comparison takes two (32 x 512 x 2048 channels x 16 fp32 229 us,
// 233); that makes 1 of a NaN, which the product with x brings back.
__device__ __forceinline__ float sigmoid(float x) {
  const float e = exp_near(-__builtin_fminf(__builtin_fabsf(x), 110.0f));
  const float inv = rcp_full(1.0f + e);
  return x < 0.0f ? e * inv : inv;
}

// The same beside 16-bit activations: the plain product and the hardware's
// exponential and reciprocal, 2^-22 of the value and what a change of x by 2^-24 of
// itself makes.  16-bit results round that away.  The fp32 ones that a gate's
// sigmoid enters (gradients of a, skip, delta_bias and the state; the
// convolution's sums) keep their digits as well: against 64 bits the
// gradients of 4 x 512 x 256 channels are off by 1.4e-7 to 2.3e-7 of their norm with this
// form and 1.3e-7 to 2.2e-7 with the one above, 2.5e-7 to 3.1e-7 and 1.4e-7 to 2.5e-7 where
// all gates stand about -10.  The form above would cost 8 x 2048 x 2048 x 16 backward
// 714 us for 698, 1 x 16384 x 2048 x 16 forward 289 for 279.
template <int DT>
__device__ __forceinline__ float sigmoid_for(float x) {
  if constexpr (DT == CNHWC_F32) return sigmoid(x);
  else return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x| in (0, 1], and its
// derivative s = 1 / (1 + e^-x).  log(1 + e) is taken of the rounded w = 1 + e
// and corrected by what the rounding left out, (e - (w - 1)) / w: within 2^-21.9
// of the value over all x down to -87, where it becomes 0 (measured; the
// logarithm alone would lose every digit of a small e).
__device__ __forceinline__ float softplus(float x, float& s) {
  const float e = exp_full(-__builtin_fabsf(x));
  const float w = 1.0f + e;
  const float inv = rcp_full(w);
  const float left = e - (w - 1.0f);
  s = x < 0.0f ? e * inv : inv;
  return (x > 0.0f ? x : 0.0f) + __builtin_fmaf(__builtin_amdgcn_logf(w), 0.693147181f, left * inv);
}
// The value alone: 1 / w scales only the correction there, the estimate is enough.
__device__ __forceinline__ float softplus(float x) {
  const float e = exp_full(-__builtin_fabsf(x));
  const float w = 1.0f + e;
  const float left = e - (w - 1.0f);
  return (x > 0.0f ? x : 0.0f) +
         __builtin_fmaf(__builtin_amdgcn_logf(w), 0.693147181f, left * __builtin_amdgcn_rcpf(w));
}

// Valid positions of sequence n.
__device__ __forceinline__ int32_t valid_len(const int32_t* lengths, int64_t n, int32_t l) {
  if (!lengths) return l;
  const int32_t v = lengths[n];
  return v < 0 ? 0 : (v > l ? l : v);
}

// ---------------------------------------------------------------- partial sums

// Up to three outputs side by side in the rows of partial sums; those with a
// NULL pointer are skipped.
struct SumOut {
  void* p[3];
  int64_t n[3];
};

// part: `parts` rows of n[0] + n[1] + n[2] fp32 partial sums.  The outputs = the
// sums over the rows, in a fixed order, rounded once: 16 columns by 16 row
// groups to a workgroup, so a few thousand columns fill the device.
template <int DT>
__global__ __launch_bounds__(256) void sum_parts_kernel(const float* __restrict__ part, int64_t parts, SumOut out,
                                                        bool f32) {
  __shared__ float sum[16][17];
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int64_t c = int64_t(blockIdx.x) * 16 + col, width = out.n[0] + out.n[1] + out.n[2];
  float v = 0.0f;
  if (c < width) {
#pragma unroll 8
    for (int64_t r = grp; r < parts; r += 16) v += part[r * width + c];
  }
  sum[grp][col] = v;
  __syncthreads();
  if (grp != 0 || c >= width) return;
#pragma unroll
  for (int k = 1; k < 16; ++k) v += sum[k][col];
  int64_t at = c;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (at >= 0 && at < out.n[i] && out.p[i]) store_param<DT>(out.p[i], at, f32, v);
    at -= out.n[i];
  }
}

template <int DT>
void sum_parts(const float* part, int64_t parts, const SumOut& out, bool f32, hipStream_t st) {
  const int64_t width = out.n[0] + out.n[1] + out.n[2];
  hipLaunchKernelGGL((sum_parts_kernel<DT>), dim3(unsigned((width + 15) / 16)), dim3(256), 0, st, part, parts, out,
                     f32);
}

}  // namespace seq
}  // namespace cnhwc
