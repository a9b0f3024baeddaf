// Rotary positions for gfx950: the first R channels of every head turn in pairs,
//   (a, b) -> scale (a cos - b sin, a sin + b cos),  angle = position * frequency[i],
// the pair being the channels i and i + R/2 (half) or 2i and 2i + 1 (interleaved);
// the channels from R on go through unchanged.  The gradient is the same turn backwards.
//
// The angle is a product in 64 bits, taken to turns and reduced to an eighth of a
// turn there: at position 10^6 the product in 32 bits would be off by 0.03 rad.  Sine and
// cosine are their Taylor series on [-pi/4, pi/4] (remainders 2e-9 and 1e-10).  A
// thread turns the same pairs of several heads, so it computes them once for these.
//
// Bound by memory, every element read and written once (4 x 4096 x 32 x 128 bf16: 50 us,
// 5.4 TB/s); a token's call by its launch.
#include <hip/hip_runtime.h>

#include "internal.hpp"
#include "seq_common.hpp"
#include "seq_host.hpp"

namespace cnhwc {
namespace seq {
namespace {

struct RotGeo {
  int64_t tokens;
  int32_t l, h, half, units, pair_units;  // units of a head: pairs, then what stays
  int32_t head_lanes;                      // threads that share a token's heads
  int64_t xs[3], os[3], ps[2];             // element strides: sequence, position, head
  int64_t offset;
  float scale, sign;
};

// cos and sin of 2 pi t.
__device__ __forceinline__ void turn(double t, float& c, float& s) {
  const double quarter = __builtin_rint(4.0 * t);
  const float a = float(__builtin_fma(quarter, -0.25, t)) * 6.28318530717958647692f;
  const int k = int(int64_t(quarter) & 3);
  const float q = a * a;
  float sp = __builtin_fmaf(q, 2.75573192e-6f, -1.98412698e-4f);
  sp = __builtin_fmaf(q, sp, 8.33333333e-3f);
  sp = __builtin_fmaf(q, sp, -0.166666667f);
  sp = __builtin_fmaf(q * a, sp, a);
  float cp = __builtin_fmaf(q, -2.75573192e-7f, 2.48015873e-5f);
  cp = __builtin_fmaf(q, cp, -1.38888889e-3f);
  cp = __builtin_fmaf(q, cp, 4.16666667e-2f);
  cp = __builtin_fmaf(q, cp, -0.5f);
  cp = __builtin_fmaf(q, cp, 1.0f);
  const float x = k & 1 ? sp : cp, y = k & 1 ? cp : sp;
  c = k == 1 || k == 2 ? -x : x;
  s = k & 2 ? -y : y;
}

// Heads whose loads are issued together (4 x 4096 x 32 x 128 bf16: 1 56 us, 2 45, 3 48, 4 52),
// and heads that share a thread's angles: of two vectors 2 (43 us, 4 44, 8 50; f32 with 16 heads
// 41, 43, 49), of one 4 (interleaved, 2 heads 50 us, 4 46, 8 48), of single elements, with
// an angle for each pair, 8 (4 x 2048 x 32 x 100 bf16: 2 40 us, 4 27, 8 24).  These with three
// sets of inputs in turn, which stay in the cache in part.
constexpr int kBatch = 2;
constexpr int heads_of(int ve, bool interleaved) { return ve == 1 ? 8 : interleaved ? 4 : 2; }

// Elements of a unit: VE pairs in two vectors (half), VE / 2 pairs in one
// (interleaved), one vector of what stays; with VE 1 a pair or an element.
template <int DT, int VE, bool INTERLEAVED>
__global__ __launch_bounds__(256) void rotary_kernel(const Elem<DT>* x, const double* __restrict__ freqs,
                                                     const int32_t* __restrict__ positions, Elem<DT>* out, RotGeo g) {
  constexpr bool kTwo = !INTERLEAVED || VE == 1;            // a unit has two vectors
  constexpr int kPairs = INTERLEAVED && VE > 1 ? VE / 2 : VE;
  const int64_t all = g.tokens * g.head_lanes * g.units;
  for (int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x; id < all; id += int64_t(gridDim.x) * 256) {
    const int64_t row = id / g.units;
    const int32_t unit = int32_t(id - row * g.units);
    const int64_t token = row / g.head_lanes;
    const int32_t h0 = int32_t(row - token * g.head_lanes);
    const int64_t n = token / g.l, t = token - n * g.l;
    const Elem<DT>* xr = x + n * g.xs[0] + t * g.xs[1];
    Elem<DT>* yr = out + n * g.os[0] + t * g.os[1];
    if (unit < g.pair_units) {
      const int32_t i0 = unit * kPairs;
      const int32_t c0 = INTERLEAVED ? 2 * i0 : i0, c1 = INTERLEAVED ? 2 * i0 + 1 : g.half + i0;
      const double at = double(g.offset + (positions ? int64_t(positions[n * g.ps[0] + t * g.ps[1]]) : t)) * g.sign;
      float cs[kPairs], sn[kPairs];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        turn(at * (freqs[i0 + i] * 0.15915494309189533577), cs[i], sn[i]);
        cs[i] *= g.scale, sn[i] *= g.scale;
      }
      for (int64_t h = h0; h < g.h; h += int64_t(kBatch) * g.head_lanes) {
        Pack<DT, VE> a[kBatch], b[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int64_t hh = h + int64_t(j) * g.head_lanes;
          if (hh >= g.h) continue;
          a[j] = load_pack<DT, VE>(xr + hh * g.xs[2] + c0);
          if constexpr (kTwo) b[j] = load_pack<DT, VE>(xr + hh * g.xs[2] + c1);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int64_t hh = h + int64_t(j) * g.head_lanes;
          if (hh >= g.h) continue;
#pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            Elem<DT>& ea = kTwo ? a[j].e[kTwo ? i : 0] : a[j].e[kTwo ? 0 : 2 * i];
            Elem<DT>& eb = kTwo ? b[j].e[kTwo ? i : 0] : a[j].e[kTwo ? 0 : 2 * i + 1];
            const float fa = to_f<DT>(ea), fb = to_f<DT>(eb);
            ea = from_f<DT>(__builtin_fmaf(fa, cs[i], -(fb * sn[i])));
            eb = from_f<DT>(__builtin_fmaf(fa, sn[i], fb * cs[i]));
          }
          store_pack<DT, VE>(yr + hh * g.os[2] + c0, a[j]);
          if constexpr (kTwo) store_pack<DT, VE>(yr + hh * g.os[2] + c1, b[j]);
        }
      }
    } else if (x != out) {
      const int32_t c = 2 * g.half + (unit - g.pair_units) * VE;
      for (int64_t h = h0; h < g.h; h += g.head_lanes)
        store_pack<DT, VE>(yr + h * g.os[2] + c, load_pack<DT, VE>(xr + h * g.xs[2] + c));
    }
  }
}

// ---------------------------------------------------------------- host

bool strides3_ok(const cnhwc_rotary_desc_t& d, const int64_t (&s)[3]) {
  constexpr int64_t kMax = 1ll << 60;
  const int64_t ext[3] = {d.n, d.l, d.h};
  int64_t end = d.d;
  for (int i = 0; i < 3; ++i) {
    if (ext[i] == 1) continue;
    if (s[i] < 0 || s[i] > kMax / ext[i]) return false;
    end += (ext[i] - 1) * s[i];
  }
  return end <= kMax;
}

// No two rows of a strided output meet: each stride passes what lies within it.
bool apart(const cnhwc_rotary_desc_t& d, const int64_t (&s)[3]) {
  int64_t ext[3] = {d.n, d.l, d.h}, st[3] = {s[0], s[1], s[2]}, inner = d.d;
  for (int i = 0; i < 3; ++i)  // a dimension of one row strides nowhere
    if (ext[i] == 1) st[i] = 0;
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[j] < st[i]) {
        const int64_t a = st[i], b = ext[i];
        st[i] = st[j], ext[i] = ext[j], st[j] = a, ext[j] = b;
      }
  for (int i = 0; i < 3; ++i) {
    if (ext[i] == 1) continue;
    if (st[i] < inner) return false;
    inner += (ext[i] - 1) * st[i];
  }
  return true;
}

uint64_t span3(const cnhwc_rotary_desc_t& d, const int64_t (&s)[3]) {
  return uint64_t((d.n > 1 ? (d.n - 1) * s[0] : 0) + (d.l > 1 ? (d.l - 1) * s[1] : 0) +
                  (d.h > 1 ? (d.h - 1) * s[2] : 0) + d.d);
}

bool vectors(const cnhwc_rotary_desc_t& d, const int64_t (&s)[3], const void* p) {
  const int64_t v = 16 / int64_t(dtype_size(d.dtype));
  return aligned(p, 16) && d.d % v == 0 && (d.interleaved ? d.r : d.r / 2) % v == 0 && (d.n == 1 || s[0] % v == 0) &&
         (d.l == 1 || s[1] % v == 0) && (d.h == 1 || s[2] % v == 0);
}

template <int DT, int VE>
hipError_t rotary_t(const cnhwc_rotary_desc_t& d, RotGeo g, const void* x, const double* freqs,
                    const int32_t* positions, void* out, hipStream_t st) {
  using E = Elem<DT>;
  const int32_t pairs = d.interleaved && VE > 1 ? VE / 2 : VE;
  g.pair_units = g.half / pairs;
  g.units = g.pair_units + (d.d - d.r) / VE;
  g.head_lanes = int32_t(ceil_div(int64_t(g.h), int64_t(heads_of(VE, d.interleaved))));
  const dim3 grid = grid_of(ceil_div(g.tokens * g.units * g.head_lanes, int64_t(256)));
  if (d.interleaved)
    hipLaunchKernelGGL((rotary_kernel<DT, VE, true>), grid, dim3(256), 0, st, static_cast<const E*>(x), freqs,
                       positions, static_cast<E*>(out), g);
  else
    hipLaunchKernelGGL((rotary_kernel<DT, VE, false>), grid, dim3(256), 0, st, static_cast<const E*>(x), freqs,
                       positions, static_cast<E*>(out), g);
  return hipGetLastError();
}

}  // namespace
}  // namespace seq
}  // namespace cnhwc

using namespace cnhwc;
using namespace cnhwc::seq;

extern "C" cnhwc_status_t cnhwc_rotary(const cnhwc_rotary_desc_t* desc, const void* x, const double* freqs,
                                       const int32_t* positions, void* out, void* hip_stream) {
  if (!desc || !dtype_ok(desc->dtype) || desc->reserved != 0) return CNHWC_ERR_INVALID_ARGUMENT;
  const cnhwc_rotary_desc_t& d = *desc;
  if ((d.interleaved | 1) != 1 || (d.inverse | 1) != 1) return CNHWC_ERR_INVALID_ARGUMENT;
  if (!extent_ok(d.n) || !extent_ok(d.l) || !extent_ok(d.h) || d.d < 1 || d.r < 0 || d.r % 2 != 0 || d.r > d.d)
    return CNHWC_ERR_INVALID_ARGUMENT;
  if (!strides3_ok(d, d.x_stride) || !strides3_ok(d, d.out_stride)) return CNHWC_ERR_INVALID_ARGUMENT;
  if (positions && !strides_ok(d.n, d.l, 1, d.position_stride)) return CNHWC_ERR_INVALID_ARGUMENT;
  if (d.offset < -(1ll << 40) || d.offset > (1ll << 40)) return CNHWC_ERR_INVALID_ARGUMENT;
  if (static_cast<unsigned __int128>(d.n) * uint64_t(d.l) * uint64_t(d.h) * uint64_t(d.d) >= (1ull << 60))
    return CNHWC_ERR_UNSUPPORTED;
  const uint64_t es = dtype_size(d.dtype);
  Buffers bf;
  if (x == out) {  // in place
    for (int i = 0; i < 3; ++i)
      if ((i == 0 ? d.n : i == 1 ? d.l : d.h) > 1 && d.x_stride[i] != d.out_stride[i]) return CNHWC_ERR_INVALID_ARGUMENT;
  } else {
    bf.in(x, span3(d, d.x_stride) * es, es, true);
  }
  if (!apart(d, d.out_stride)) return CNHWC_ERR_INVALID_ARGUMENT;
  bf.in(freqs, uint64_t(d.r) / 2 * 8, 8, d.r > 0);
  bf.in(positions, positions ? span(d.n, d.l, 1, d.position_stride) * 4 : 0, 4, false);
  bf.out(out, span3(d, d.out_stride) * es, es, true);
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  RotGeo g{};
  g.tokens = d.n * d.l;
  g.l = int32_t(d.l), g.h = int32_t(d.h), g.half = d.r / 2;
  for (int i = 0; i < 3; ++i) g.xs[i] = d.x_stride[i], g.os[i] = d.out_stride[i];
  for (int i = 0; i < 2; ++i) g.ps[i] = d.position_stride[i];
  g.offset = d.offset;
  g.scale = d.scale;
  g.sign = d.inverse ? -1.0f : 1.0f;
  const bool vec = vectors(d, d.x_stride, x) && vectors(d, d.out_stride, out);
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  hipError_t e;
  if (d.dtype == CNHWC_F32)
    e = vec ? rotary_t<CNHWC_F32, 4>(d, g, x, freqs, positions, out, s)
            : rotary_t<CNHWC_F32, 1>(d, g, x, freqs, positions, out, s);
  else if (d.dtype == CNHWC_F16)
    e = vec ? rotary_t<CNHWC_F16, 8>(d, g, x, freqs, positions, out, s)
            : rotary_t<CNHWC_F16, 1>(d, g, x, freqs, positions, out, s);
  else
    e = vec ? rotary_t<CNHWC_BF16, 8>(d, g, x, freqs, positions, out, s)
            : rotary_t<CNHWC_BF16, 1>(d, g, x, freqs, positions, out, s);
  return e == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
}
