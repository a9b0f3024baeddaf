// Root-mean-square norm over the channels, for gfx950: forward with the
// residual's addition, the same into 8 bits with scales, and backward.
//
// Forward, per row of C channels: z = x + residual, rstd = 1 / sqrt(mean z^2 + eps),
// y = z rstd w, and z itself, rounded, as the residual of the next layer.  y comes
// from the sum before that rounding.  In 8 bits y goes out as e4m3 with a scale for
// the row or for each group of 32, 64 or 128 channels, max |y| / 448: the maximum of
// a group is a few lane permutations, because a lane's vector lies in one group
// and a group's lanes are neighbours.
//
// Backward, with xh = z rstd and g = dy w:
//   dz = rstd (g - xh mean(g xh)) + dsum,  dw = sum_rows dy xh,
// dsum being the gradient that reaches z past the norm.  The rows are walked as in
// layer norm's: each workgroup sums dw of its rows in registers and leaves one
// fp32 row, and a second kernel adds those in a fixed order.
//
// Every tensor moves once: the row is held in fp32 registers (tiles of norm_rows.hpp).
// Rows that are not whole 16-byte vectors go element by element, rows wider than
// the largest tile are read again from the cache.
//
// Bound by memory: 4 x 4096 x 4096 bf16 with the residual 99 us (5.4 TB/s), the same in 8
// bits by groups of 128 93 us (5.1 TB/s), 8 x 2048 x 2048 backward 56 us (4.8 TB/s); a
// token's row by its launch (kernel 2.1 us).  Rows off 16 bytes by their single elements:
// 16384 x 613 bf16 with the residual 36 us (2.2 TB/s), in 8 bits 43, backward 29.
#include <hip/hip_runtime.h>

#include <cfloat>

#include "internal.hpp"
#include "norm_rows.hpp"
#include "seq_common.hpp"
#include "seq_host.hpp"

namespace cnhwc {
namespace seq {
namespace {

constexpr float kQ8Max = 448.0f;       // e4m3's largest value
constexpr float kScaleMin = 0x1p-100f; // its inverse is finite, and so is 448 times that

struct RmsGeo {
  int64_t rows;
  int32_t l, c, group;  // group: channels to a scale (0: the row)
  int64_t xs[2], rs[2], dys[2];  // element strides: sequence, position; rs: residual, or dsum
  float eps, inv_c;
  bool w_f32;
};

template <int DT>
struct RmsFwd {
  const Elem<DT>* x;
  const Elem<DT>* residual;  // may be sum
  const void* w;
  Elem<DT>* sum;
  Elem<DT>* y;   // or
  uint8_t* q;    // with
  float* scale;
  float* rstd;
};

// V values over a scale in e4m3, round to nearest even.
template <int V>
__device__ __forceinline__ void store_q8(uint8_t* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = uint8_t(__builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[0], 0, false));
  } else {
    uint32_t r[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      int u = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
      r[i] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], u, true));
    }
    if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(r[0], r[1]);
    else *reinterpret_cast<uint32_t*>(p) = r[0];
  }
}

// v / scale to the last digit, so that an element in 8 bits is the nearest one but for
// what v itself is off: the product with the inverse and what it leaves.  (An infinite
// scale makes NaN of everything, as the product does.)
__device__ __forceinline__ float over(float v, float scale, float inv) {
  const float q = v * inv;
  return __builtin_fmaf(__builtin_fmaf(-q, scale, v), inv, q);
}

__device__ __forceinline__ float scale_of(float largest) {
  const float s = largest / kQ8Max;
  return s < kScaleMin ? kScaleMin : s;
}

// The largest over the lanes that hold a group of g.group channels.
template <int VE>
__device__ __forceinline__ float lanes_max(float v, int32_t group) {
  v = group_max<32 / VE>(v);
  if (group >= 64) v = __builtin_fmaxf(v, __shfl_xor(v, 32 / VE));
  if (group >= 128) v = __builtin_fmaxf(v, __shfl_xor(v, 64 / VE));
  return v;
}

template <int DT, int VE, int NV, int TPR, bool Q8>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void rms_fwd_kernel(RmsFwd<DT> io, RmsGeo g) {
  constexpr int kThreads = TPR > 256 ? TPR : 256;
  __shared__ float red[2][16];
  const int t = threadIdx.x % TPR;
  // w stays in registers where it is short, else each row takes it from the cache again
  constexpr bool kHold = NV * VE <= 16;
  float wf[kHold ? NV : 1][VE];
  auto params = [&](int32_t c0, float (&wv)[VE]) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < VE; ++e) wv[e] = 1.0f;
    if (io.w && c0 < g.c) load_params<DT, VE>(io.w, c0, g.w_f32, wv);
  };
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < NV; ++i) params((i * TPR + t) * VE, wf[i]);
  }
  int slot = 0;
  // every thread of a workgroup walks the same number of rows (barriers inside)
  for (int64_t row0 = int64_t(blockIdx.x) * (kThreads / TPR); row0 < g.rows;
       row0 += int64_t(gridDim.x) * (kThreads / TPR), slot ^= 1) {
    const int64_t row = row0 + threadIdx.x / TPR;
    const bool live = row < g.rows;  // whole groups of TPR threads
    const Elem<DT>* xr = io.x + (live ? row_offset(row, g.l, g.xs) : 0);
    Pack<DT, VE> p[NV];
    float z[NV * VE];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t c0 = (i * TPR + t) * VE;
      if (live && c0 < g.c) p[i] = load_pack<DT, VE>(xr + c0);
      else p[i] = Pack<DT, VE>{};
    }
    if (io.residual) {
      const Elem<DT>* rr = io.residual + (live ? row_offset(row, g.l, g.rs) : 0);
      Pack<DT, VE> r[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int32_t c0 = (i * TPR + t) * VE;
        if (live && c0 < g.c) r[i] = load_pack<DT, VE>(rr + c0);
        else r[i] = Pack<DT, VE>{};
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) z[i * VE + e] = to_f<DT>(p[i].e[e]) + to_f<DT>(r[i].e[e]);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) z[i * VE + e] = to_f<DT>(p[i].e[e]);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV * VE; ++i) s = __builtin_fmaf(z[i], z[i], s);
    if (io.sum && live) {
      Elem<DT>* sr = io.sum + row * g.c;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int32_t c0 = (i * TPR + t) * VE;
        if (c0 >= g.c) continue;
        Pack<DT, VE> o;
#pragma unroll
        for (int e = 0; e < VE; ++e) o.e[e] = from_f<DT>(z[i * VE + e]);
        store_pack<DT, VE>(sr + c0, o);
      }
    }
    const float ms = row_sum<TPR>(s, red, Q8 ? 0 : slot) * g.inv_c;
    const float rstd = 1.0f / __builtin_sqrtf(ms + g.eps);
    if (io.rstd && t == 0 && live) io.rstd[row] = rstd;
    if constexpr (!Q8) {
      if (!live) continue;
      Elem<DT>* yr = io.y + row * g.c;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int32_t c0 = (i * TPR + t) * VE;
        if (c0 >= g.c) continue;
        if constexpr (!kHold) {
          int32_t at = c0;
          asm volatile("" : "+v"(at));  // not to be held over the rows
          params(at, wf[0]);
        }
        Pack<DT, VE> o;
#pragma unroll
        for (int e = 0; e < VE; ++e) o.e[e] = from_f<DT>(z[i * VE + e] * rstd * wf[kHold ? i : 0][e]);
        store_pack<DT, VE>(yr + c0, o);
      }
    } else {
      float largest = 0.0f, of[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int32_t c0 = (i * TPR + t) * VE;
        if constexpr (!kHold) {
          int32_t at = c0;
          asm volatile("" : "+v"(at));
          params(at, wf[0]);
        }
        of[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          z[i * VE + e] = z[i * VE + e] * rstd * wf[kHold ? i : 0][e];
          of[i] = __builtin_fmaxf(of[i], c0 < g.c ? __builtin_fabsf(z[i * VE + e]) : 0.0f);
        }
        largest = __builtin_fmaxf(largest, of[i]);
      }
      if (g.group) {
        if constexpr (VE > 1) {
#pragma unroll
          for (int i = 0; i < NV; ++i) of[i] = lanes_max<VE>(of[i], g.group);
        }
      } else {
        largest = row_max<TPR>(largest, red, 1);
#pragma unroll
        for (int i = 0; i < NV; ++i) of[i] = largest;
      }
      // without groups one barrier follows the sum's (in row_max); with them this one does
      if constexpr (TPR > 64) {
        if (g.group) __syncthreads();
      }
      if (!live) continue;
      uint8_t* qr = io.q + row * g.c;
      const int shift = g.group ? __builtin_ctz(g.group) : 31;
      const int32_t groups = g.group ? g.c >> shift : 1, inside = g.group ? g.group - 1 : 0x7fffffff;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int32_t c0 = (i * TPR + t) * VE;
        if (c0 >= g.c) continue;
        const float scale = scale_of(of[i]), inv = 1.0f / scale;
        float v[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) v[e] = over(z[i * VE + e], scale, inv);
        store_q8<VE>(qr + c0, v);
        if ((c0 & inside) == 0) io.scale[row * groups + (c0 >> shift)] = scale;
      }
    }
  }
}

// Rows wider than the register tiles, and groups of rows that are not whole
// vectors: a row at a time, read again from the cache.  The sum goes out last,
// so it may lie on the residual.
template <int DT, bool Q8>
__global__ __launch_bounds__(1024) void rms_fwd_wide_kernel(RmsFwd<DT> io, RmsGeo g) {
  __shared__ float red[2][16];
  for (int64_t row = blockIdx.x; row < g.rows; row += gridDim.x) {
    const Elem<DT>* xr = io.x + row_offset(row, g.l, g.xs);
    const Elem<DT>* rr = io.residual ? io.residual + row_offset(row, g.l, g.rs) : nullptr;
    auto at = [&](int64_t c) { return to_f<DT>(xr[c]) + (rr ? to_f<DT>(rr[c]) : 0.0f); };
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < g.c; c += 1024) s = __builtin_fmaf(at(c), at(c), s);
    const float rstd = 1.0f / __builtin_sqrtf(row_sum<1024>(s, red, 0) * g.inv_c + g.eps);
    if (io.rstd && threadIdx.x == 0) io.rstd[row] = rstd;
    auto y_at = [&](int64_t c, float z) { return z * rstd * (io.w ? load_param<DT>(io.w, c, g.w_f32) : 1.0f); };
    // one wavefront to a group, or all of them to the row
    const int32_t span = g.group ? g.group : g.c;
    const int32_t first = g.group ? threadIdx.x >> 6 : 0, next = g.group ? 16 : 1;
    const int32_t lane = g.group ? threadIdx.x & 63 : threadIdx.x, lanes = g.group ? 64 : 1024;
    const int32_t groups = g.c / span;
    for (int32_t k = first; k < groups; k += next) {
      const int64_t c0 = int64_t(k) * span;
      float inv = 1.0f, scale = 1.0f;
      if constexpr (Q8) {
        float largest = 0.0f;
        for (int32_t c = lane; c < span; c += lanes)
          largest = __builtin_fmaxf(largest, __builtin_fabsf(y_at(c0 + c, at(c0 + c))));
        scale = scale_of(g.group ? group_max<64>(largest) : row_max<1024>(largest, red, 1));
        inv = 1.0f / scale;
        if (lane == 0) io.scale[row * groups + k] = scale;
      }
      for (int32_t c = lane; c < span; c += lanes) {
        const float z = at(c0 + c), v = y_at(c0 + c, z);
        if constexpr (Q8) {
          const float one[1] = {over(v, scale, inv)};
          store_q8<1>(io.q + row * g.c + c0 + c, one);
        } else {
          io.y[row * g.c + c0 + c] = from_f<DT>(v);
        }
        if (io.sum) io.sum[row * g.c + c0 + c] = from_f<DT>(z);
      }
    }
    __syncthreads();  // red[0] again
  }
}

// ---------------------------------------------------------------- backward

// part: [gridDim.x][C] partial sums of dw (NULL: not wanted).
template <int DT, int VE, int NV, int TPR>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void rms_bwd_kernel(
    const Elem<DT>* __restrict__ dy, const Elem<DT>* __restrict__ dsum, const Elem<DT>* __restrict__ x,
    const float* __restrict__ rstd, const void* __restrict__ w, Elem<DT>* __restrict__ dx,
    float* __restrict__ part, RmsGeo g) {
  constexpr int kThreads = TPR > 256 ? TPR : 256;
  constexpr int kGroups = kThreads / TPR;
  __shared__ float red[2][16];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  float wf[NV * VE], dw[NV * VE];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int32_t c0 = (i * TPR + t) * VE;
    float wv[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) wv[e] = 1.0f;
    if (w && c0 < g.c) load_params<DT, VE>(w, c0, g.w_f32, wv);
#pragma unroll
    for (int e = 0; e < VE; ++e) wf[i * VE + e] = wv[e], dw[i * VE + e] = 0.0f;
  }
  const int64_t step = int64_t(gridDim.x) * kGroups;
  // small tiles have the next row's loads under way meanwhile
  constexpr bool kAhead = NV * VE <= 8 && TPR <= 256;
  Pack<DT, VE> px[NV], pg[NV], ps[NV];
  float rs = 0.0f;
  auto load = [&](int64_t row) __attribute__((always_inline)) {
    const bool ok = row < g.rows;
    const Elem<DT>* xr = x + (ok ? row_offset(row, g.l, g.xs) : 0);
    const Elem<DT>* gr = dy + (ok ? row_offset(row, g.l, g.dys) : 0);
    const Elem<DT>* sr = dsum + (ok && dsum ? row_offset(row, g.l, g.rs) : 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t c0 = (i * TPR + t) * VE;
      Pack<DT, VE> a{}, b{}, c{};
      if (ok && c0 < g.c) {
        a = load_pack<DT, VE>(xr + c0);
        b = load_pack<DT, VE>(gr + c0);
        if (dsum) c = load_pack<DT, VE>(sr + c0);
      }
      px[i] = a, pg[i] = b, ps[i] = c;
    }
    rs = ok ? rstd[row] : 0.0f;
  };
  int slot = 0;
  // a workgroup-wide row takes part in barriers: its row index is uniform there
  int64_t row = int64_t(blockIdx.x) * kGroups + grp;
  if constexpr (kAhead) load(row);
  for (; row < g.rows; row += step, slot ^= 1) {
    if constexpr (!kAhead) load(row);
    float xh[NV * VE], v[NV * VE], ds[kAhead ? NV * VE : 1], s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = (i * TPR + t) * VE < g.c;  // 0 past the row, whatever the statistics
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int k = i * VE + e;
        const float d = to_f<DT>(pg[i].e[e]);
        xh[k] = in ? to_f<DT>(px[i].e[e]) * rs : 0.0f;
        v[k] = d * wf[k];
        s = __builtin_fmaf(v[k], xh[k], s);
        dw[k] = __builtin_fmaf(d, xh[k], dw[k]);
        if constexpr (kAhead) ds[k] = to_f<DT>(ps[i].e[e]);
      }
    }
    const float r = rs;
    if constexpr (kAhead) load(row + step);
    s = row_sum<TPR>(s, red, slot) * g.inv_c;
    Elem<DT>* dr = dx + row * g.c;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t c0 = (i * TPR + t) * VE;
      if (c0 >= g.c) continue;
      Pack<DT, VE> o;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int k = i * VE + e;
        float past = 0.0f;
        if (dsum) {
          if constexpr (kAhead) past = ds[k];
          else past = to_f<DT>(ps[i].e[e]);
        }
        o.e[e] = from_f<DT>(__builtin_fmaf(r, v[k] - xh[k] * s, past));
      }
      store_pack<DT, VE>(dr + c0, o);
    }
  }
  if (!part) return;
  float* pw = part + int64_t(blockIdx.x) * g.c;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int32_t c = (i * TPR + t) * VE + e;
        if (c < g.c) pw[c] = dw[i * VE + e];
      }
  } else {
    // the workgroup's row groups, added in order
    constexpr int kCols = NV * VE * TPR;
    __shared__ float sum[kGroups][kCols];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) sum[grp][(i * TPR + t) * VE + e] = dw[i * VE + e];
    __syncthreads();
    for (int c = threadIdx.x; c < g.c; c += kThreads) {
      float v = sum[0][c];
#pragma unroll
      for (int k = 1; k < kGroups; ++k) v += sum[k][c];
      pw[c] = v;
    }
  }
}

// Rows wider than the register tiles: dx alone, two passes over the row.
template <int DT>
__global__ __launch_bounds__(1024) void rms_bwd_wide_kernel(
    const Elem<DT>* __restrict__ dy, const Elem<DT>* __restrict__ dsum, const Elem<DT>* __restrict__ x,
    const float* __restrict__ rstd, const void* __restrict__ w, Elem<DT>* __restrict__ dx, RmsGeo g) {
  __shared__ float red[2][16];
  int slot = 0;
  for (int64_t row = blockIdx.x; row < g.rows; row += gridDim.x, slot ^= 1) {
    const Elem<DT>* xr = x + row_offset(row, g.l, g.xs);
    const Elem<DT>* gr = dy + row_offset(row, g.l, g.dys);
    const Elem<DT>* sr = dsum ? dsum + row_offset(row, g.l, g.rs) : nullptr;
    const float rs = rstd[row];
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < g.c; c += 1024) {
      const float v = to_f<DT>(gr[c]) * (w ? load_param<DT>(w, c, g.w_f32) : 1.0f);
      s = __builtin_fmaf(v, to_f<DT>(xr[c]) * rs, s);
    }
    s = row_sum<1024>(s, red, slot) * g.inv_c;
    Elem<DT>* dr = dx + row * g.c;
    for (int64_t c = threadIdx.x; c < g.c; c += 1024) {
      const float v = to_f<DT>(gr[c]) * (w ? load_param<DT>(w, c, g.w_f32) : 1.0f);
      dr[c] = from_f<DT>(__builtin_fmaf(rs, v - to_f<DT>(xr[c]) * rs * s, sr ? to_f<DT>(sr[c]) : 0.0f));
    }
  }
}

// ... and its dw: 256 channels by rows r, r + gridDim.y, ... per workgroup.
template <int DT>
__global__ __launch_bounds__(256) void rms_bwd_cols_kernel(const Elem<DT>* __restrict__ dy,
                                                           const Elem<DT>* __restrict__ x,
                                                           const float* __restrict__ rstd, float* __restrict__ part,
                                                           RmsGeo g) {
  const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (c >= g.c) return;
  float dw = 0.0f;
  for (int64_t row = blockIdx.y; row < g.rows; row += gridDim.y)
    dw = __builtin_fmaf(to_f<DT>(dy[row_offset(row, g.l, g.dys) + c]),
                        to_f<DT>(x[row_offset(row, g.l, g.xs) + c]) * rstd[row], dw);
  part[int64_t(blockIdx.y) * g.c + c] = dw;
}

// ---------------------------------------------------------------- host

RmsGeo geo_of(const cnhwc_rms_norm_desc_t& d, bool more, bool bwd) {
  RmsGeo g{};
  g.rows = d.n * d.l;
  g.l = int32_t(d.l);
  g.c = int32_t(d.c);
  g.group = d.group;
  for (int i = 0; i < 2; ++i) {
    g.xs[i] = d.x_stride[i];
    g.rs[i] = d.residual_stride[i];
    g.dys[i] = d.dy_stride[i];
  }
  // rows at one stride throughout: no division of the row index
  auto one = [&](const int64_t (&s)[2]) { return d.n == 1 || s[0] == d.l * s[1]; };
  if (d.l > 1 && one(d.x_stride) && (!more || one(d.residual_stride)) && (!bwd || one(d.dy_stride))) {
    g.l = 1;
    g.xs[0] = d.x_stride[1];
    g.rs[0] = d.residual_stride[1];
    g.dys[0] = d.dy_stride[1];
  }
  g.eps = d.eps;
  g.inv_c = float(1.0 / double(d.c));
  g.w_f32 = d.w_dtype == CNHWC_F32;
  return g;
}

// 16-byte vectors: every row starts on one and holds a whole number of them.
bool vectors(const cnhwc_rms_norm_desc_t& d, const int64_t (&s)[2], const void* p) {
  const int64_t v = 16 / int64_t(dtype_size(d.dtype));
  return !p || (aligned(p, 16) && d.c % v == 0 && (d.n == 1 || s[0] % v == 0) && (d.l == 1 || s[1] % v == 0));
}

// Most workgroups of the forward pass, so that w is taken up a few times only (16384 x 4096
// bf16 with the residual: 1024 workgroups 100 us, 2048 111, 8192 99, 65536 98; in 8 bits 93, 96,
// 93, 97), and the elements that a thread holds.
constexpr int64_t kFwdBlocks = 8192;
constexpr int kFwdRegs = 64, kFwdWide = 32, kBwdRegs = 32, kBwdWide = 16;

template <int DT, int VE, bool Q8>
hipError_t rms_fwd_t(const RmsGeo& g, const RmsFwd<DT>& io, hipStream_t st) {
  bool held = false;
  if (!(Q8 && VE == 1 && g.group))  // a group's lanes hold vectors
    held = with_tile<VE, kFwdRegs, kFwdWide>(ceil_div(g.c, VE), [&](auto tile) {
      constexpr int NV = decltype(tile)::nv, TPR = decltype(tile)::tpr;
      constexpr int threads = TPR > 256 ? TPR : 256;
      const int64_t blocks = ceil_div(g.rows, threads / TPR);
      hipLaunchKernelGGL((rms_fwd_kernel<DT, VE, NV, TPR, Q8>),
                         dim3(unsigned(blocks < kFwdBlocks ? blocks : kFwdBlocks)), dim3(threads), 0, st, io, g);
    });
  if (!held) hipLaunchKernelGGL((rms_fwd_wide_kernel<DT, Q8>), grid_of(g.rows), dim3(1024), 0, st, io, g);
  return hipGetLastError();
}

// Workgroups of the backward pass (rows of partial sums), a function of the shape only: as
// many as find their places at once, and no fewer rows than four each.  Measured with
// 512, 768 and 1024: one vector to a thread, 16384 x 2048 bf16 54, 55, 58 us (256: 86), 65536 x 512
// 49, 53, 54, 16384 x 1024 f32 50, 52, 54; two, 16384 x 4096 bf16 111, 109, 114, 8192 x 2424 f16 50, 43,
// 42; four, 8192 x 8192 bf16 117, 139, 132; elements, 16384 x 613 40, 32, 28; a workgroup of more than
// 256 threads, 2048 x 16384 80 each, 64 with 256 (one sweep).
int64_t bwd_groups(const cnhwc_rms_norm_desc_t& d, bool vec) {
  const int64_t rows = d.n * d.l;
  const int64_t ve = vec ? 16 / int64_t(dtype_size(d.dtype)) : 1;
  int64_t per = 1, cap = 64;  // thread groups per workgroup; the wide form's row groups
  auto pick = [&](auto tile) {
    constexpr int TPR = decltype(tile)::tpr, NV = decltype(tile)::nv;
    per = TPR > 256 ? 1 : 256 / TPR;
    cap = TPR > 256 ? 256 : ve == 1 ? 1024 : NV == 2 ? 768 : 512;
  };
  if (ve == 8) with_tile<8, kBwdRegs, kBwdWide>(ceil_div(d.c, 8), pick);
  else if (ve == 4) with_tile<4, kBwdRegs, kBwdWide>(ceil_div(d.c, 4), pick);
  else with_tile<1, kBwdRegs, kBwdWide>(d.c, pick);
  const int64_t want = ceil_div(rows, per * 4);
  return want < cap ? want : cap;
}

template <int DT, int VE>
hipError_t rms_bwd_t(const cnhwc_rms_norm_desc_t& d, const RmsGeo& g, const void* dy, const void* dsum, const void* x,
                     const float* rstd, const void* w, void* dx, void* dw, float* part, hipStream_t st) {
  using E = Elem<DT>;
  const int64_t groups = bwd_groups(d, VE > 1);
  float* pt = dw ? part : nullptr;
  const E *pdy = static_cast<const E*>(dy), *pds = static_cast<const E*>(dsum), *px = static_cast<const E*>(x);
  const bool held = with_tile<VE, kBwdRegs, kBwdWide>(ceil_div(g.c, VE), [&](auto tile) {
    constexpr int NV = decltype(tile)::nv, TPR = decltype(tile)::tpr;
    hipLaunchKernelGGL((rms_bwd_kernel<DT, VE, NV, TPR>), dim3(unsigned(groups)), dim3(TPR > 256 ? TPR : 256), 0, st,
                       pdy, pds, px, rstd, w, static_cast<E*>(dx), pt, g);
  });
  if (!held) {
    hipLaunchKernelGGL((rms_bwd_wide_kernel<DT>), grid_of(g.rows), dim3(1024), 0, st, pdy, pds, px, rstd, w,
                       static_cast<E*>(dx), g);
    if (dw)
      hipLaunchKernelGGL((rms_bwd_cols_kernel<DT>), dim3(unsigned(ceil_div(g.c, 256)), unsigned(groups)), dim3(256),
                         0, st, pdy, px, rstd, part, g);
  }
  if (dw) sum_parts<DT>(part, groups, SumOut{{dw, nullptr, nullptr}, {g.c, 0, 0}}, g.w_f32, st);
  return hipGetLastError();
}

cnhwc_status_t check_desc(const cnhwc_rms_norm_desc_t* d, bool more, bool bwd, bool q8) {
  if (!d || !dtype_ok(d->dtype)) return CNHWC_ERR_INVALID_ARGUMENT;
  if (d->w_dtype != d->dtype && d->w_dtype != CNHWC_F32) return CNHWC_ERR_INVALID_ARGUMENT;
  if (!extent_ok(d->n) || !extent_ok(d->l) || !extent_ok(d->c) || !(d->eps >= 0.0f)) return CNHWC_ERR_INVALID_ARGUMENT;
  if (!strides_ok(d->n, d->l, d->c, d->x_stride)) return CNHWC_ERR_INVALID_ARGUMENT;
  if (more && !strides_ok(d->n, d->l, d->c, d->residual_stride)) return CNHWC_ERR_INVALID_ARGUMENT;
  if (bwd && !strides_ok(d->n, d->l, d->c, d->dy_stride)) return CNHWC_ERR_INVALID_ARGUMENT;
  if (d->group != 0) {
    if (!q8 || d->group < 0 || d->c % d->group != 0) return CNHWC_ERR_INVALID_ARGUMENT;
    if (d->group != 32 && d->group != 64 && d->group != 128) return CNHWC_ERR_UNSUPPORTED;
  }
  // the reduction's grid, and 64-bit offsets
  if (d->c > (1ll << 26) || !dense_ok(d->n, d->l, d->c)) return CNHWC_ERR_UNSUPPORTED;
  return CNHWC_OK;
}

template <int DT, int VE>
hipError_t rms_fwd_q(bool q8, const RmsGeo& g, const void* x, const void* residual, const void* w, void* out,
                     float* scale, void* sum, float* rstd, hipStream_t st) {
  using E = Elem<DT>;
  RmsFwd<DT> io{};
  io.x = static_cast<const E*>(x);
  io.residual = static_cast<const E*>(residual);
  io.w = w;
  io.sum = static_cast<E*>(sum);
  io.rstd = rstd;
  if (q8) {
    io.q = static_cast<uint8_t*>(out);
    io.scale = scale;
    return rms_fwd_t<DT, VE, true>(g, io, st);
  }
  io.y = static_cast<E*>(out);
  return rms_fwd_t<DT, VE, false>(g, io, st);
}

cnhwc_status_t forward(const cnhwc_rms_norm_desc_t* desc, bool q8, const void* x, const void* residual, const void* w,
                       void* out, float* scale, void* sum, float* rstd, void* hip_stream) {
  cnhwc_status_t st = check_desc(desc, residual != nullptr, false, q8);
  if (st != CNHWC_OK) return st;
  const cnhwc_rms_norm_desc_t& d = *desc;
  const uint64_t es = dtype_size(d.dtype), ws = dtype_size(d.w_dtype);
  const uint64_t rows = uint64_t(d.n) * d.l;
  Buffers bf;
  bf.in(x, span(d.n, d.l, d.c, d.x_stride) * es, es, true);
  bf.in(w, d.c * ws, ws, false);
  if (sum && sum == residual) {  // in place: the same element goes where it came from
    if ((d.l > 1 && d.residual_stride[1] != d.c) || (d.n > 1 && d.residual_stride[0] != d.l * d.c))
      return CNHWC_ERR_INVALID_ARGUMENT;
  } else {
    bf.in(residual, span(d.n, d.l, d.c, d.residual_stride) * es, es, sum != nullptr);
  }
  bf.out(sum, rows * d.c * es, es, false);
  bf.out(out, rows * d.c * (q8 ? 1 : es), q8 ? 1 : es, true);
  if (q8) bf.out(scale, rows * (d.group ? d.c / d.group : 1) * 4, 4, true);
  bf.out(rstd, rows * 4, 4, false);
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  const RmsGeo g = geo_of(d, residual != nullptr, false);
  const bool vec = vectors(d, d.x_stride, x) && vectors(d, d.residual_stride, residual) && aligned(w, 16) &&
                   aligned(sum, 16) && aligned(out, q8 ? 8 : 16);
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  hipError_t e;
  if (d.dtype == CNHWC_F32)
    e = vec ? rms_fwd_q<CNHWC_F32, 4>(q8, g, x, residual, w, out, scale, sum, rstd, s)
            : rms_fwd_q<CNHWC_F32, 1>(q8, g, x, residual, w, out, scale, sum, rstd, s);
  else if (d.dtype == CNHWC_F16)
    e = vec ? rms_fwd_q<CNHWC_F16, 8>(q8, g, x, residual, w, out, scale, sum, rstd, s)
            : rms_fwd_q<CNHWC_F16, 1>(q8, g, x, residual, w, out, scale, sum, rstd, s);
  else
    e = vec ? rms_fwd_q<CNHWC_BF16, 8>(q8, g, x, residual, w, out, scale, sum, rstd, s)
            : rms_fwd_q<CNHWC_BF16, 1>(q8, g, x, residual, w, out, scale, sum, rstd, s);
  return e == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
}

}  // namespace
}  // namespace seq
}  // namespace cnhwc

using namespace cnhwc;
using namespace cnhwc::seq;

extern "C" cnhwc_status_t cnhwc_rms_norm_fwd(const cnhwc_rms_norm_desc_t* desc, const void* x, const void* residual,
                                             const void* w, void* y, void* sum, float* rstd, void* hip_stream) {
  return forward(desc, false, x, residual, w, y, nullptr, sum, rstd, hip_stream);
}

extern "C" cnhwc_status_t cnhwc_rms_norm_fwd_q8(const cnhwc_rms_norm_desc_t* desc, const void* x,
                                                const void* residual, const void* w, void* q, float* scale, void* sum,
                                                float* rstd, void* hip_stream) {
  return forward(desc, true, x, residual, w, q, scale, sum, rstd, hip_stream);
}

extern "C" cnhwc_status_t cnhwc_rms_norm_bwd_workspace(const cnhwc_rms_norm_desc_t* desc, int32_t param_grads,
                                                       uint64_t* bytes) {
  const cnhwc_status_t st = check_desc(desc, false, true, false);
  if (st != CNHWC_OK) return st;
  if (!bytes) return CNHWC_ERR_INVALID_ARGUMENT;
  // enough for the vector and the element form alike: which one runs also
  // depends on the pointers
  const int64_t a = bwd_groups(*desc, true), b = bwd_groups(*desc, false);
  *bytes = param_grads ? uint64_t(a > b ? a : b) * uint64_t(desc->c) * 4 : 0;
  return CNHWC_OK;
}

extern "C" cnhwc_status_t cnhwc_rms_norm_bwd(const cnhwc_rms_norm_desc_t* desc, const void* dy, const void* dsum,
                                             const void* x, const float* rstd, const void* w, void* dx, void* dw,
                                             void* workspace, uint64_t workspace_bytes, void* hip_stream) {
  cnhwc_status_t st = check_desc(desc, dsum != nullptr, true, false);
  if (st != CNHWC_OK) return st;
  const cnhwc_rms_norm_desc_t& d = *desc;
  uint64_t need = 0;
  st = cnhwc_rms_norm_bwd_workspace(desc, dw != nullptr, &need);
  if (st != CNHWC_OK) return st;
  const uint64_t es = dtype_size(d.dtype), ws = dtype_size(d.w_dtype);
  const uint64_t rows = uint64_t(d.n) * d.l;
  Buffers bf;
  bf.in(dy, span(d.n, d.l, d.c, d.dy_stride) * es, es, true);
  if (dsum) bf.in(dsum, span(d.n, d.l, d.c, d.residual_stride) * es, es, true);
  bf.in(x, span(d.n, d.l, d.c, d.x_stride) * es, es, true);
  bf.in(rstd, rows * 4, 4, true);
  bf.in(w, d.c * ws, ws, dw != nullptr);
  bf.out(dx, rows * d.c * es, es, true);
  bf.out(dw, d.c * ws, ws, false);
  if (need) {
    if (workspace_bytes < need) return CNHWC_ERR_WORKSPACE_TOO_SMALL;
    bf.out(workspace, need, 16, true);
  }
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  const RmsGeo g = geo_of(d, dsum != nullptr, true);
  const bool vec = vectors(d, d.x_stride, x) && vectors(d, d.dy_stride, dy) && vectors(d, d.residual_stride, dsum) &&
                   aligned(w, 16) && aligned(dx, 16);
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  float* part = static_cast<float*>(workspace);
  hipError_t e;
  if (d.dtype == CNHWC_F32)
    e = vec ? rms_bwd_t<CNHWC_F32, 4>(d, g, dy, dsum, x, rstd, w, dx, dw, part, s)
            : rms_bwd_t<CNHWC_F32, 1>(d, g, dy, dsum, x, rstd, w, dx, dw, part, s);
  else if (d.dtype == CNHWC_F16)
    e = vec ? rms_bwd_t<CNHWC_F16, 8>(d, g, dy, dsum, x, rstd, w, dx, dw, part, s)
            : rms_bwd_t<CNHWC_F16, 1>(d, g, dy, dsum, x, rstd, w, dx, dw, part, s);
  else
    e = vec ? rms_bwd_t<CNHWC_BF16, 8>(d, g, dy, dsum, x, rstd, w, dx, dw, part, s)
            : rms_bwd_t<CNHWC_BF16, 1>(d, g, dy, dsum, x, rstd, w, dx, dw, part, s);
  return e == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
}
