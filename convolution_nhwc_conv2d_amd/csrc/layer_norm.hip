// Layer norm over the channels, forward and backward, for gfx950.
//
// Forward, per row of C channels: mean = sum x / C, var = sum (x - mean)^2 / C,
// y = (x - mean) rstd w + b.  The row stays in registers as it was loaded, so
// the variance is the two-pass one (no cancellation) at the traffic of one
// pass: x read once, y written once.  The mean of a row of one constant is that
// constant: what the product with 1 / C has rounded is put back, and for fp32
// rows what the sum has rounded too (mean_of, put_right below).
//
// Backward, with xh = (x - mean) rstd and g = dy w:
//   dx = rstd (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy.
// The workgroups are few and walk over the rows, so each thread keeps the dw
// and db sums of its own channels in registers; a workgroup writes one fp32
// row of partial sums, and a second kernel adds those rows in a fixed order.
//
// Both are bound by memory: 32768 x 4096 bf16 forward 99 us, 5.4 TB/s; backward
// of 65536 x 2048 bf16 157 us, 5.1 TB/s, of 16384 x 2048 55 us, 3.7 TB/s (52 where the
// inputs come back every third call; a copy reaches 4.8 to 5.0 TB/s on this card).
// A row is held by TPR threads, NV vectors each: few threads for narrow rows
// (several rows to a wavefront), one wavefront up to 64 * NV vectors, a workgroup
// beyond.  Rows whose address or length is not a
// multiple of 16 bytes go element by element; rows wider than the largest
// register tile are re-read from the cache.
#include <hip/hip_runtime.h>

#include <cfloat>

#include "internal.hpp"
#include "seq_common.hpp"
#include "seq_host.hpp"

namespace cnhwc {
namespace seq {
namespace {

struct LnGeo {
  int64_t rows;
  int32_t l, c;
  int64_t xs[2], dys[2];  // element strides: sequence, position
  float eps, inv_c;
  bool w_f32;
};

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

__device__ __forceinline__ float if_finite(float v) { return __builtin_fabsf(v) <= FLT_MAX ? v : 0.0f; }

// sum / C: the product with 1 / C, and what that leaves of the sum (exact).  A
// row with an infinity keeps it as its mean.
__device__ __forceinline__ float mean_of(float sum, const LnGeo& g) {
  const float m = sum * g.inv_c;
  return __builtin_fmaf(if_finite(__builtin_fmaf(-float(g.c), m, sum)), g.inv_c, m);
}

// The variance from the sum of (x - m)^2.  fp32: the sum of x - m beside it says
// how far the rounded sum of the row has moved m, which matters where the row
// hardly varies (3000.1 throughout: up to 80 units of the last place, 0.02 of a
// distance whose scale is sqrt(eps)); m moves back, and m's own distance
// leaves the variance.  Rows of 16-bit elements of one constant have an exact
// sum up to thousands of channels, and the second sum costs 65536 x 512 f16 5% (23.2 to
// 24.4 us; 25088 x 512 f32 16.2 with and without), so they go without.
template <int DT>
__device__ __forceinline__ float put_right(float left, float squares, float& m, const LnGeo& g) {
  if constexpr (DT != CNHWC_F32) return squares * g.inv_c;
  const float dm = if_finite(left * g.inv_c);
  const float var = __builtin_fmaf(-dm, dm, squares * g.inv_c);
  m += dm;
  return var < 0.0f ? 0.0f : var;  // a NaN stays
}

template <int DT, int VE, int NV, int TPR>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void ln_fwd_kernel(
    const Elem<DT>* __restrict__ x, const void* __restrict__ w, const void* __restrict__ b,
    Elem<DT>* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out, LnGeo g) {
  constexpr int kThreads = TPR > 256 ? TPR : 256;
  __shared__ float red[2][2][16];
  const int t = threadIdx.x % TPR;
  // w and b stay in registers where they are few, else each row takes them from
  // the cache again
  constexpr bool kHold = NV * VE <= 16;
  float wf[kHold ? NV : 1][VE], bf[kHold ? NV : 1][VE];
  auto params = [&](int32_t c0, float (&wv)[VE], float (&bv)[VE]) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < VE; ++e) wv[e] = 1.0f, bv[e] = 0.0f;
    if (w && c0 < g.c) load_params<DT, VE>(w, c0, g.w_f32, wv);
    if (b && c0 < g.c) load_params<DT, VE>(b, c0, g.w_f32, bv);
  };
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < NV; ++i) params((i * TPR + t) * VE, wf[i], bf[i]);
  }
  // every thread of a workgroup walks the same number of rows (barriers inside)
  for (int64_t row0 = int64_t(blockIdx.x) * (kThreads / TPR); row0 < g.rows;
       row0 += int64_t(gridDim.x) * (kThreads / TPR)) {
    const int64_t row = row0 + threadIdx.x / TPR;
    const bool live = row < g.rows;  // whole groups of TPR threads
    const Elem<DT>* xr = x + (live ? row_offset(row, g.l, g.xs) : 0);
    Pack<DT, VE> p[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t c0 = (i * TPR + t) * VE;
      if (live && c0 < g.c) p[i] = load_pack<DT, VE>(xr + c0);
      else p[i] = Pack<DT, VE>{};
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) s += to_f<DT>(p[i].e[e]);
    float mean = mean_of(row_sum<TPR>(s, red[0], 0), g);
    float q = 0.0f, left = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * TPR + t) * VE >= g.c) continue;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float d = to_f<DT>(p[i].e[e]) - mean;
        q = __builtin_fmaf(d, d, q);
        if constexpr (DT == CNHWC_F32) left += d;
      }
    }
    if constexpr (DT == CNHWC_F32) row_sums<TPR>(left, q, red, 1);
    else q = row_sum<TPR>(q, red[1], 0);
    const float var = put_right<DT>(left, q, mean, g);
    const float rstd = 1.0f / __builtin_sqrtf(var + g.eps);
    if (!live) continue;
    Elem<DT>* yr = y + row * g.c;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t c0 = (i * TPR + t) * VE;
      if (c0 >= g.c) continue;
      if constexpr (!kHold) {
        int32_t at = c0;
        asm volatile("" : "+v"(at));  // not to be held over the rows
        params(at, wf[0], bf[0]);
      }
      Pack<DT, VE> o;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float v = (to_f<DT>(p[i].e[e]) - mean) * rstd;
        o.e[e] = from_f<DT>(__builtin_fmaf(v, wf[kHold ? i : 0][e], bf[kHold ? i : 0][e]));
      }
      store_pack<DT, VE>(yr + c0, o);
    }
    if (mean_out && t == 0) {
      mean_out[row] = mean;
      rstd_out[row] = rstd;
    }
  }
}

// Rows wider than the register tiles: three passes over a row, the last two from the cache.
template <int DT>
__global__ __launch_bounds__(1024) void ln_fwd_wide_kernel(
    const Elem<DT>* __restrict__ x, const void* __restrict__ w, const void* __restrict__ b,
    Elem<DT>* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out, LnGeo g) {
  __shared__ float red[2][2][16];
  for (int64_t row = blockIdx.x; row < g.rows; row += gridDim.x) {
    const Elem<DT>* xr = x + row_offset(row, g.l, g.xs);
    float s = 0.0f, q = 0.0f, left = 0.0f;
    for (int64_t c = threadIdx.x; c < g.c; c += 1024) s += to_f<DT>(xr[c]);
    float mean = mean_of(row_sum<1024>(s, red[0], 0), g);
    for (int64_t c = threadIdx.x; c < g.c; c += 1024) {
      const float d = to_f<DT>(xr[c]) - mean;
      q = __builtin_fmaf(d, d, q);
      if constexpr (DT == CNHWC_F32) left += d;
    }
    if constexpr (DT == CNHWC_F32) row_sums<1024>(left, q, red, 1);
    else q = row_sum<1024>(q, red[1], 0);
    const float rstd = 1.0f / __builtin_sqrtf(put_right<DT>(left, q, mean, g) + g.eps);
    Elem<DT>* yr = y + row * g.c;
    for (int64_t c = threadIdx.x; c < g.c; c += 1024) {
      float v = (to_f<DT>(xr[c]) - mean) * rstd;
      if (w) v = __builtin_fmaf(v, load_param<DT>(w, c, g.w_f32), b ? load_param<DT>(b, c, g.w_f32) : 0.0f);
      yr[c] = from_f<DT>(v);
    }
    if (mean_out && threadIdx.x == 0) {
      mean_out[row] = mean;
      rstd_out[row] = rstd;
    }
  }
}

// ---------------------------------------------------------------- backward

// part: [gridDim.x][2][C] partial sums of dw and db (NULL: not wanted).
template <int DT, int VE, int NV, int TPR>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void ln_bwd_kernel(
    const Elem<DT>* __restrict__ dy, const Elem<DT>* __restrict__ x, const float* __restrict__ mean,
    const float* __restrict__ rstd, const void* __restrict__ w, Elem<DT>* __restrict__ dx,
    float* __restrict__ part, LnGeo g) {
  constexpr int kThreads = TPR > 256 ? TPR : 256;
  constexpr int kGroups = kThreads / TPR;
  __shared__ float red[2][2][16];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  float wf[NV * VE], dw[NV * VE], db[NV * VE];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int32_t c0 = (i * TPR + t) * VE;
    float wv[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) wv[e] = 1.0f;
    if (w && c0 < g.c) load_params<DT, VE>(w, c0, g.w_f32, wv);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      wf[i * VE + e] = wv[e];
      dw[i * VE + e] = db[i * VE + e] = 0.0f;
    }
  }
  const int64_t step = int64_t(gridDim.x) * kGroups;
  // small tiles keep g and xh, and the next row's loads are under way meanwhile
  constexpr bool kAhead = NV * VE <= 8 && TPR <= 256;
  Pack<DT, VE> px[NV], pg[NV];
  float mu = 0.0f, rs = 0.0f;
  auto load = [&](int64_t row) __attribute__((always_inline)) {
    const bool ok = row < g.rows;
    const Elem<DT>* xr = x + (ok ? row_offset(row, g.l, g.xs) : 0);
    const Elem<DT>* gr = dy + (ok ? row_offset(row, g.l, g.dys) : 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t c0 = (i * TPR + t) * VE;
      Pack<DT, VE> a{}, b{};
      if (ok && c0 < g.c) {
        a = load_pack<DT, VE>(xr + c0);
        b = load_pack<DT, VE>(gr + c0);
      }
      px[i] = a;
      pg[i] = b;
    }
    mu = ok ? mean[row] : 0.0f;
    rs = ok ? rstd[row] : 0.0f;
  };
  int slot = 0;
  // a workgroup-wide row takes part in barriers: its row index is uniform there
  int64_t row = int64_t(blockIdx.x) * kGroups + grp;
  if constexpr (kAhead) load(row);
  for (; row < g.rows; row += step, slot ^= 1) {
    if constexpr (!kAhead) load(row);
    // g and xh of an element, from the row as it was loaded (0 past the row,
    // whatever the statistics)
    auto terms = [&](int i, int e, float& v, float& xh) __attribute__((always_inline)) {
      v = to_f<DT>(pg[i].e[e]) * wf[i * VE + e];
      xh = !kAhead || (i * TPR + t) * VE < g.c ? (to_f<DT>(px[i].e[e]) - mu) * rs : 0.0f;
    };
    float xh[kAhead ? NV * VE : 1], v[kAhead ? NV * VE : 1], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!kAhead && (i * TPR + t) * VE >= g.c) continue;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int k = i * VE + e, h = kAhead ? k : 0;
        terms(i, e, v[h], xh[h]);
        const float d = to_f<DT>(pg[i].e[e]);
        s1 += v[h];
        s2 = __builtin_fmaf(v[h], xh[h], s2);
        dw[k] = __builtin_fmaf(d, xh[h], dw[k]);
        db[k] += d;
      }
    }
    const float r = rs;
    if constexpr (kAhead) load(row + step);
    row_sums<TPR>(s1, s2, red, slot);
    if constexpr (!kAhead) asm volatile("" : "+v"(mu), "+v"(rs));  // made again, not held
    s1 *= g.inv_c;
    s2 *= g.inv_c;
    Elem<DT>* dr = dx + row * g.c;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t c0 = (i * TPR + t) * VE;
      if (c0 >= g.c) continue;
      Pack<DT, VE> o;
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int h = kAhead ? i * VE + e : 0;
        if constexpr (!kAhead) terms(i, e, v[0], xh[0]);
        o.e[e] = from_f<DT>(r * (v[h] - s1 - xh[h] * s2));
      }
      store_pack<DT, VE>(dr + c0, o);
    }
  }
  if (!part) return;
  float* pw = part + int64_t(blockIdx.x) * 2 * g.c;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int32_t c = (i * TPR + t) * VE + e;
        if (c < g.c) {
          pw[c] = dw[i * VE + e];
          pw[g.c + c] = db[i * VE + e];
        }
      }
  } else {
    // the workgroup's row groups, added in order
    constexpr int kCols = NV * VE * TPR;
    __shared__ float sum[kGroups][kCols];
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e)
          sum[grp][(i * TPR + t) * VE + e] = which ? db[i * VE + e] : dw[i * VE + e];
      __syncthreads();
      for (int c = threadIdx.x; c < g.c; c += kThreads) {
        float v = sum[0][c];
#pragma unroll
        for (int k = 1; k < kGroups; ++k) v += sum[k][c];
        pw[which * int64_t(g.c) + c] = v;
      }
    }
  }
}

// Rows wider than the register tiles: dx alone, two passes over the row.
template <int DT>
__global__ __launch_bounds__(1024) void ln_bwd_wide_kernel(
    const Elem<DT>* __restrict__ dy, const Elem<DT>* __restrict__ x, const float* __restrict__ mean,
    const float* __restrict__ rstd, const void* __restrict__ w, Elem<DT>* __restrict__ dx, LnGeo g) {
  __shared__ float red[2][16];
  for (int64_t row = blockIdx.x; row < g.rows; row += gridDim.x) {
    const Elem<DT>* xr = x + row_offset(row, g.l, g.xs);
    const Elem<DT>* gr = dy + row_offset(row, g.l, g.dys);
    const float mu = mean[row], rs = rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < g.c; c += 1024) {
      const float v = to_f<DT>(gr[c]) * (w ? load_param<DT>(w, c, g.w_f32) : 1.0f);
      s1 += v;
      s2 = __builtin_fmaf(v, (to_f<DT>(xr[c]) - mu) * rs, s2);
    }
    s1 = row_sum<1024>(s1, red, 0) * g.inv_c;
    s2 = row_sum<1024>(s2, red, 1) * g.inv_c;
    Elem<DT>* dr = dx + row * g.c;
    for (int64_t c = threadIdx.x; c < g.c; c += 1024) {
      const float v = to_f<DT>(gr[c]) * (w ? load_param<DT>(w, c, g.w_f32) : 1.0f);
      dr[c] = from_f<DT>(rs * (v - s1 - (to_f<DT>(xr[c]) - mu) * rs * s2));
    }
  }
}

// ... and its dw, db: 256 channels by rows r, r + gridDim.y, ... per workgroup.
template <int DT>
__global__ __launch_bounds__(256) void ln_bwd_cols_kernel(
    const Elem<DT>* __restrict__ dy, const Elem<DT>* __restrict__ x, const float* __restrict__ mean,
    const float* __restrict__ rstd, float* __restrict__ part, LnGeo g) {
  const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (c >= g.c) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = blockIdx.y; row < g.rows; row += gridDim.y) {
    const float d = to_f<DT>(dy[row_offset(row, g.l, g.dys) + c]);
    dw = __builtin_fmaf(d, (to_f<DT>(x[row_offset(row, g.l, g.xs) + c]) - mean[row]) * rstd[row], dw);
    db += d;
  }
  float* pw = part + int64_t(blockIdx.y) * 2 * g.c;
  pw[c] = dw;
  pw[g.c + c] = db;
}

// ---------------------------------------------------------------- host

LnGeo geo_of(const cnhwc_layer_norm_desc_t& d, bool bwd) {
  LnGeo g{};
  g.rows = d.n * d.l;
  g.l = int32_t(d.l);
  g.c = int32_t(d.c);
  for (int i = 0; i < 2; ++i) {
    g.xs[i] = d.x_stride[i];
    g.dys[i] = d.dy_stride[i];
  }
  // rows at one stride throughout: no division of the row index
  if (d.l > 1 && (d.n == 1 || (d.x_stride[0] == d.l * d.x_stride[1] &&
                               (!bwd || d.dy_stride[0] == d.l * d.dy_stride[1])))) {
    g.l = 1;
    g.xs[0] = d.x_stride[1];
    g.dys[0] = d.dy_stride[1];
  }
  g.eps = d.eps;
  g.inv_c = float(1.0 / double(d.c));
  g.w_f32 = d.w_dtype == CNHWC_F32;
  return g;
}

// 16-byte vectors: every row starts on one and holds a whole number of them.
bool vectors(const cnhwc_layer_norm_desc_t& d, const int64_t (&s)[2], const void* p) {
  const int64_t v = 16 / int64_t(dtype_size(d.dtype));
  return aligned(p, 16) && d.c % v == 0 && (d.n == 1 || s[0] % v == 0) && (d.l == 1 || s[1] % v == 0);
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

// The forward pass keeps the row as it was loaded; the backward pass also w and
// two sums for every channel, in 32 bits.
// Most workgroups of the forward pass, a few for every place on the device, so
// that w and b are taken up a few times only (32768 x 4096 bf16: 1024
// workgroups 104 us, 8192 98, 65536 117; 65536 x 2048: 154, 98, 111).
constexpr int64_t kFwdBlocks = 8192;
constexpr int kFwdRegs = 64, kFwdWide = 64, kBwdRegs = 32, kBwdWide = 16;

template <int DT, int VE>
hipError_t ln_fwd_t(const LnGeo& g, const void* x, const void* w, const void* b, void* y, float* mean,
                    float* rstd, hipStream_t st) {
  using E = Elem<DT>;
  const bool held = with_tile<VE, kFwdRegs, kFwdWide>(ceil_div(g.c, VE), [&](auto tile) {
    constexpr int NV = decltype(tile)::nv, TPR = decltype(tile)::tpr;
    constexpr int threads = TPR > 256 ? TPR : 256;
    const int64_t blocks = ceil_div(g.rows, threads / TPR);
    hipLaunchKernelGGL((ln_fwd_kernel<DT, VE, NV, TPR>), dim3(unsigned(blocks < kFwdBlocks ? blocks : kFwdBlocks)),
                       dim3(threads), 0, st, static_cast<const E*>(x), w, b, static_cast<E*>(y), mean, rstd, g);
  });
  if (!held)
    hipLaunchKernelGGL((ln_fwd_wide_kernel<DT>), grid_of(g.rows), dim3(1024), 0, st,
                       static_cast<const E*>(x), w, b, static_cast<E*>(y), mean, rstd, g);
  return hipGetLastError();
}

// Workgroups of the backward pass (rows of partial sums): at least four rows
// for each thread group, at most two workgroups of 256 threads for each of the
// 256 compute units.  A function of the shape only.
int64_t bwd_groups(const cnhwc_layer_norm_desc_t& d, bool vec) {
  const int64_t rows = d.n * d.l;
  const int64_t ve = vec ? 16 / int64_t(dtype_size(d.dtype)) : 1;
  int64_t per = 1, cap = 64;  // thread groups per workgroup; the wide form's row groups
  auto pick = [&](auto tile) {
    constexpr int TPR = decltype(tile)::tpr;
    per = TPR > 256 ? 1 : 256 / TPR;
    cap = TPR > 256 ? 256 : 1024;
  };
  if (ve == 8) with_tile<8, kBwdRegs, kBwdWide>(ceil_div(d.c, 8), pick);
  else if (ve == 4) with_tile<4, kBwdRegs, kBwdWide>(ceil_div(d.c, 4), pick);
  else with_tile<1, kBwdRegs, kBwdWide>(d.c, pick);
  const int64_t want = ceil_div(rows, per * 4);
  return want < cap ? want : cap;
}

template <int DT, int VE>
hipError_t ln_bwd_t(const cnhwc_layer_norm_desc_t& d, const LnGeo& g, const void* dy, const void* x,
                    const float* mean, const float* rstd, const void* w, void* dx, void* dw, void* db,
                    float* part, hipStream_t st) {
  using E = Elem<DT>;
  const int64_t groups = bwd_groups(d, VE > 1);
  float* pt = dw ? part : nullptr;
  const bool held = with_tile<VE, kBwdRegs, kBwdWide>(ceil_div(g.c, VE), [&](auto tile) {
    constexpr int NV = decltype(tile)::nv, TPR = decltype(tile)::tpr;
    hipLaunchKernelGGL((ln_bwd_kernel<DT, VE, NV, TPR>), dim3(unsigned(groups)), dim3(TPR > 256 ? TPR : 256), 0,
                       st, static_cast<const E*>(dy), static_cast<const E*>(x), mean, rstd, w,
                       static_cast<E*>(dx), pt, g);
  });
  if (!held) {
    hipLaunchKernelGGL((ln_bwd_wide_kernel<DT>), grid_of(g.rows), dim3(1024), 0, st,
                       static_cast<const E*>(dy), static_cast<const E*>(x), mean, rstd, w, static_cast<E*>(dx), g);
    if (dw)
      hipLaunchKernelGGL((ln_bwd_cols_kernel<DT>), dim3(unsigned(ceil_div(g.c, 256)), unsigned(groups)), dim3(256),
                         0, st, static_cast<const E*>(dy), static_cast<const E*>(x), mean, rstd, part, g);
  }
  if (dw)
    sum_parts<DT>(part, groups, SumOut{{dw, db, nullptr}, {g.c, g.c, 0}}, g.w_f32, st);
  return hipGetLastError();
}

cnhwc_status_t check_desc(const cnhwc_layer_norm_desc_t* d, bool bwd) {
  if (!d || !dtype_ok(d->dtype) || d->reserved != 0) return CNHWC_ERR_INVALID_ARGUMENT;
  if (d->w_dtype != d->dtype && d->w_dtype != CNHWC_F32) return CNHWC_ERR_INVALID_ARGUMENT;
  if (!extent_ok(d->n) || !extent_ok(d->l) || !extent_ok(d->c) || !(d->eps >= 0.0f)) return CNHWC_ERR_INVALID_ARGUMENT;
  if (!strides_ok(d->n, d->l, d->c, d->x_stride)) return CNHWC_ERR_INVALID_ARGUMENT;
  if (bwd && !strides_ok(d->n, d->l, d->c, d->dy_stride)) return CNHWC_ERR_INVALID_ARGUMENT;
  // the reduction's grid, and 64-bit offsets
  if (d->c > (1ll << 26) || !dense_ok(d->n, d->l, d->c)) return CNHWC_ERR_UNSUPPORTED;
  return CNHWC_OK;
}

}  // namespace
}  // namespace seq
}  // namespace cnhwc

using namespace cnhwc;
using namespace cnhwc::seq;

extern "C" cnhwc_status_t cnhwc_layer_norm_fwd(const cnhwc_layer_norm_desc_t* desc, const void* x, const void* w,
                                               const void* b, void* y, float* mean, float* rstd,
                                               void* hip_stream) {
  cnhwc_status_t st = check_desc(desc, false);
  if (st != CNHWC_OK) return st;
  const cnhwc_layer_norm_desc_t& d = *desc;
  const uint64_t es = dtype_size(d.dtype), ws = dtype_size(d.w_dtype);
  const uint64_t rows = uint64_t(d.n) * d.l;
  Buffers bf;
  bf.in(x, span(d.n, d.l, d.c, d.x_stride) * es, es, true);
  bf.in(w, d.c * ws, ws, b != nullptr);
  bf.in(b, d.c * ws, ws, false);
  bf.out(y, rows * d.c * es, es, true);
  bf.out(mean, rows * 4, 4, rstd != nullptr);
  bf.out(rstd, rows * 4, 4, mean != nullptr);
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  const LnGeo g = geo_of(d, false);
  const bool vec = vectors(d, d.x_stride, x) && aligned(w, 16) && aligned(b, 16) && aligned(y, 16);
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  hipError_t e;
  if (d.dtype == CNHWC_F32)
    e = vec ? ln_fwd_t<CNHWC_F32, 4>(g, x, w, b, y, mean, rstd, s)
            : ln_fwd_t<CNHWC_F32, 1>(g, x, w, b, y, mean, rstd, s);
  else if (d.dtype == CNHWC_F16)
    e = vec ? ln_fwd_t<CNHWC_F16, 8>(g, x, w, b, y, mean, rstd, s)
            : ln_fwd_t<CNHWC_F16, 1>(g, x, w, b, y, mean, rstd, s);
  else
    e = vec ? ln_fwd_t<CNHWC_BF16, 8>(g, x, w, b, y, mean, rstd, s)
            : ln_fwd_t<CNHWC_BF16, 1>(g, x, w, b, y, mean, rstd, s);
  return e == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
}

extern "C" cnhwc_status_t cnhwc_layer_norm_bwd_workspace(const cnhwc_layer_norm_desc_t* desc, int32_t param_grads,
                                                         uint64_t* bytes) {
  const cnhwc_status_t st = check_desc(desc, true);
  if (st != CNHWC_OK) return st;
  if (!bytes) return CNHWC_ERR_INVALID_ARGUMENT;
  // enough for the vector and the element form alike: which one runs also
  // depends on the pointers
  const int64_t a = bwd_groups(*desc, true), b = bwd_groups(*desc, false);
  *bytes = param_grads ? uint64_t(a > b ? a : b) * 2 * uint64_t(desc->c) * 4 : 0;
  return CNHWC_OK;
}

extern "C" cnhwc_status_t cnhwc_layer_norm_bwd(const cnhwc_layer_norm_desc_t* desc, const void* dy, const void* x,
                                               const float* mean, const float* rstd, const void* w, void* dx,
                                               void* dw, void* db, void* workspace, uint64_t workspace_bytes,
                                               void* hip_stream) {
  cnhwc_status_t st = check_desc(desc, true);
  if (st != CNHWC_OK) return st;
  const cnhwc_layer_norm_desc_t& d = *desc;
  if ((dw == nullptr) != (db == nullptr)) return CNHWC_ERR_INVALID_ARGUMENT;
  uint64_t need = 0;
  st = cnhwc_layer_norm_bwd_workspace(desc, dw != nullptr, &need);
  if (st != CNHWC_OK) return st;
  const uint64_t es = dtype_size(d.dtype), ws = dtype_size(d.w_dtype);
  const uint64_t rows = uint64_t(d.n) * d.l;
  Buffers bf;
  bf.in(dy, span(d.n, d.l, d.c, d.dy_stride) * es, es, true);
  bf.in(x, span(d.n, d.l, d.c, d.x_stride) * es, es, true);
  bf.in(mean, rows * 4, 4, true);
  bf.in(rstd, rows * 4, 4, true);
  bf.in(w, d.c * ws, ws, dw != nullptr);
  bf.out(dx, rows * d.c * es, es, true);
  bf.out(dw, d.c * ws, ws, false);
  bf.out(db, d.c * ws, ws, false);
  if (need) {
    if (workspace_bytes < need) return CNHWC_ERR_WORKSPACE_TOO_SMALL;
    bf.out(workspace, need, 16, true);
  }
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  const LnGeo g = geo_of(d, true);
  const bool vec = vectors(d, d.x_stride, x) && vectors(d, d.dy_stride, dy) && aligned(w, 16) && aligned(dx, 16);
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  float* part = static_cast<float*>(workspace);
  hipError_t e;
  if (d.dtype == CNHWC_F32)
    e = vec ? ln_bwd_t<CNHWC_F32, 4>(d, g, dy, x, mean, rstd, w, dx, dw, db, part, s)
            : ln_bwd_t<CNHWC_F32, 1>(d, g, dy, x, mean, rstd, w, dx, dw, db, part, s);
  else if (d.dtype == CNHWC_F16)
    e = vec ? ln_bwd_t<CNHWC_F16, 8>(d, g, dy, x, mean, rstd, w, dx, dw, db, part, s)
            : ln_bwd_t<CNHWC_F16, 1>(d, g, dy, x, mean, rstd, w, dx, dw, db, part, s);
  else
    e = vec ? ln_bwd_t<CNHWC_BF16, 8>(d, g, dy, x, mean, rstd, w, dx, dw, db, part, s)
            : ln_bwd_t<CNHWC_BF16, 1>(d, g, dy, x, mean, rstd, w, dx, dw, db, part, s);
  return e == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
}
