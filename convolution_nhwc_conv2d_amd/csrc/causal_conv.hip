// Short causal (depthwise) convolution, forward, backward and single tokens,
// for gfx950.
//
// With X = K-1 rows of state followed by the valid rows of x:
//   pre[t,c] = bias[c] + sum_k w[c,k] X[t+k,c],  y = act(pre)
// and backward, with dpre = dy act'(pre) (0 outside the valid positions):
//   dX[j,c] = sum_k w[c,k] dpre[j-k,c],  dw[c,k] = sum_t dpre[t,c] X[t+k,c],
//   dbias[c] = sum_t dpre[t,c];
// the first K-1 rows of dX are the state's gradient, the others x's, and the
// gradient of the state that the forward pass left is added to the last K-1.
//
// A few operations per element, so memory is the bound: a thread owns 16 bytes
// of channels (two channels in the backward pass) over a run of positions and slides a register window along it,
// so each row is loaded once per run (plus the K-1 rows before it, which the
// neighbouring run has just brought into the cache).  The weights stay in
// registers.  The backward pass recomputes pre from x instead of reading a
// saved copy, sums dw and dbias in registers over the run, adds the runs of a
// workgroup through LDS, and leaves one row of partial sums per workgroup to a
// second kernel, which adds them in a fixed order.
//
// Measured, bf16: 4 x 4096 x 4096 forward 59 us, 4.6 TB/s (52 us where the inputs
// come back every third call and are partly in the cache); backward 114 us, 3.5
// TB/s (a copy: 4.8 to 5.0), the vector pipes busy 70% of it.  Backward of five
// f16 sequences of 2047 x 2048 with 4260 valid positions 33 us: the runs that
// hold valid rows are 2.4 wavefronts a SIMD, each 28 rows one after the other
// and three of its neighbour's; the pipes are busy 37%.  In both every row asks
// whether it is valid, its own run's, a state's: the batch of four rows goes
// through as several short pieces.
#include <hip/hip_runtime.h>

#include <climits>

#include "internal.hpp"
#include "seq_common.hpp"
#include "seq_host.hpp"

namespace cnhwc {
namespace seq {
namespace {

struct ConvGeo {
  int32_t l, c, act;
  int32_t vecs;      // channel vectors
  int32_t run;       // positions per thread, a multiple of kBatch
  int64_t runs;      // runs per sequence (forward), workgroups per sequence (backward)
  int64_t xs[2], dys[2];
};

constexpr int kBatch = 4;  // rows loaded together

// w[c0..c0+V)[K] and bias as floats.
template <int DT, int V, int K>
struct Taps {
  float w[V][K], b[V];
  __device__ __forceinline__ void load(const Elem<DT>* __restrict__ wp, const Elem<DT>* __restrict__ bp, int64_t c0) {
    if constexpr (V == 1) {
#pragma unroll
      for (int k = 0; k < K; ++k) w[0][k] = to_f<DT>(wp[c0 * K + k]);
      b[0] = bp ? to_f<DT>(bp[c0]) : 0.0f;
    } else {
      Pack<DT, V> p[K];  // K vectors hold the V * K weights
#pragma unroll
      for (int i = 0; i < K; ++i) p[i] = load_pack<DT, V>(wp + c0 * K + i * V);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < K; ++k) w[v][k] = to_f<DT>(p[(v * K + k) / V].e[(v * K + k) % V]);
      const Pack<DT, V> pb = bp ? load_pack<DT, V>(bp + c0) : Pack<DT, V>{};
#pragma unroll
      for (int v = 0; v < V; ++v) b[v] = to_f<DT>(pb.e[v]);
    }
  }
};

// Row r of a sequence: x for 0 <= r < len, the state before it, zeros elsewhere.
template <int DT, int V, int K>
__device__ __forceinline__ Pack<DT, V> load_row(const Elem<DT>* __restrict__ x, const Elem<DT>* __restrict__ state,
                                                int64_t xs1, int32_t c, int64_t r, int32_t len) {
  if (r >= 0 && r < len) return load_pack<DT, V>(x + r * xs1);
  if (r < 0 && r >= -(K - 1) && state) return load_pack<DT, V>(state + (r + K - 1) * int64_t(c));
  return Pack<DT, V>{};
}

// kBatch rows from r on, all of them rows of x where the fast path holds.
template <int DT, int V, int K>
__device__ __forceinline__ void load_rows(Pack<DT, V> (&p)[kBatch], const Elem<DT>* __restrict__ x,
                                          const Elem<DT>* __restrict__ state, int64_t xs1, int32_t c, int64_t r,
                                          int32_t len) {
  if (r >= 0 && r + kBatch <= len) {
    const Elem<DT>* row = x + r * xs1;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) p[i] = load_pack<DT, V>(row + i * xs1);
  } else {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) p[i] = load_row<DT, V, K>(x, state, xs1, c, r + i, len);
  }
}

template <int DT, int V, int K>
__global__ __launch_bounds__(256) void conv_fwd_kernel(
    const Elem<DT>* __restrict__ x, const Elem<DT>* __restrict__ wp, const Elem<DT>* __restrict__ bp,
    const Elem<DT>* __restrict__ state, const int32_t* __restrict__ lengths, Elem<DT>* __restrict__ y,
    Elem<DT>* __restrict__ state_out, ConvGeo g, int64_t total) {
  for (int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x; id < total; id += int64_t(gridDim.x) * 256) {
    const int64_t run_id = id / g.vecs;
    const int64_t c0 = (id - run_id * g.vecs) * V;
    const int64_t n = run_id / g.runs;
    const int32_t t0 = int32_t((run_id - n * g.runs) * g.run);
    const int32_t len = valid_len(lengths, n, g.l);
    const Elem<DT>* xn = x + n * g.xs[0] + c0;
    const Elem<DT>* sn = state ? state + n * (K - 1) * int64_t(g.c) + c0 : nullptr;
    Elem<DT>* yn = y + n * g.l * int64_t(g.c) + c0;
    Taps<DT, V, K> tap;
    tap.load(wp, bp, c0);
    float win[K][V];  // the K newest rows, win[K-1] the newest
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      const Pack<DT, V> p = load_row<DT, V, K>(xn, sn, g.xs[1], g.c, int64_t(t0) - (K - 1) + k, len);
#pragma unroll
      for (int v = 0; v < V; ++v) win[k + 1][v] = to_f<DT>(p.e[v]);
    }
    const int32_t end = t0 + g.run < g.l ? t0 + g.run : g.l;
    const int32_t live = end < len ? end : len;
    Pack<DT, V> p[kBatch], next[kBatch];
    load_rows<DT, V, K>(p, xn, sn, g.xs[1], g.c, t0, len);
    for (int32_t tb = t0; tb < live; tb += kBatch) {
      load_rows<DT, V, K>(next, xn, sn, g.xs[1], g.c, tb + kBatch, tb + kBatch < live ? len : 0);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int32_t t = tb + i;
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
#pragma unroll
          for (int v = 0; v < V; ++v) win[k][v] = win[k + 1][v];
        Pack<DT, V> o;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          win[K - 1][v] = to_f<DT>(p[i].e[v]);
          float a = tap.b[v];
#pragma unroll
          for (int k = 0; k < K; ++k) a = __builtin_fmaf(tap.w[v][k], win[k][v], a);
          if (g.act == CNHWC_ACT_SILU) a *= sigmoid_for<DT>(a);
          o.e[v] = from_f<DT>(a);
        }
        if (t < live) store_pack<DT, V>(yn + t * int64_t(g.c), o);
        p[i] = next[i];
      }
    }
    for (int32_t t = t0 > len ? t0 : len; t < end; ++t) store_pack<DT, V>(yn + t * int64_t(g.c), Pack<DT, V>{});
    if (K > 1 && state_out && t0 == 0) {
      Elem<DT>* so = state_out + n * (K - 1) * int64_t(g.c) + c0;
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const int64_t r = int64_t(len) + j - (K - 1);
        store_pack<DT, V>(so + j * int64_t(g.c), load_row<DT, V, K>(xn, sn, g.xs[1], g.c, r, len));
      }
    }
  }
}

// One token per sequence; state_out may be state.
template <int DT, int V, int K>
__global__ __launch_bounds__(256) void conv_step_kernel(
    const Elem<DT>* __restrict__ x, const Elem<DT>* state, const Elem<DT>* __restrict__ wp,
    const Elem<DT>* __restrict__ bp, Elem<DT>* __restrict__ y, Elem<DT>* state_out, ConvGeo g, int64_t total) {
  for (int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x; id < total; id += int64_t(gridDim.x) * 256) {
    const int64_t n = id / g.vecs;
    const int64_t c0 = (id - n * g.vecs) * V;
    const int64_t so = n * (K - 1) * int64_t(g.c) + c0;
    Taps<DT, V, K> tap;
    tap.load(wp, bp, c0);
    Pack<DT, V> row[K];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) row[k] = load_pack<DT, V>(state + so + k * int64_t(g.c));
    row[K - 1] = load_pack<DT, V>(x + n * g.xs[0] + c0);
    Pack<DT, V> o;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float a = tap.b[v];
#pragma unroll
      for (int k = 0; k < K; ++k) a = __builtin_fmaf(tap.w[v][k], to_f<DT>(row[k].e[v]), a);
      if (g.act == CNHWC_ACT_SILU) a *= sigmoid_for<DT>(a);
      o.e[v] = from_f<DT>(a);
    }
    store_pack<DT, V>(y + n * int64_t(g.c) + c0, o);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) store_pack<DT, V>(state_out + so + k * int64_t(g.c), row[k + 1]);
  }
}

// A workgroup: 32 channel vectors by 8 runs of positions of one sequence, over
// the L + K - 1 rows j of dX.  part: per workgroup column of 32 vectors and per
// (sequence, workgroup along it) one row [C*K | C] of dw and dbias sums.
// first_block: the launch's first workgroup among all of the pass.
constexpr int kLanes = 32, kRunsPerBlock = 8;

template <int DT, int V, int K>
__global__ __launch_bounds__(256) void conv_bwd_kernel(
    const Elem<DT>* __restrict__ dy, const Elem<DT>* __restrict__ dfin, const Elem<DT>* __restrict__ x,
    const Elem<DT>* __restrict__ wp, const Elem<DT>* __restrict__ bp, const Elem<DT>* __restrict__ state,
    const int32_t* __restrict__ lengths, Elem<DT>* __restrict__ dx, Elem<DT>* __restrict__ dstate,
    float* __restrict__ part, ConvGeo g, int64_t col_blocks, int64_t first_block) {
  const int64_t block = first_block + blockIdx.x, row_id = block / col_blocks, col = block - row_id * col_blocks;
  const int32_t vec = int32_t(col) * kLanes + int32_t(threadIdx.x & (kLanes - 1));
  const int64_t n = row_id / g.runs;
  const int64_t j0 = ((row_id - n * g.runs) * kRunsPerBlock + threadIdx.x / kLanes) * g.run;
  const int64_t rows = int64_t(g.l) + K - 1;
  const int32_t len = valid_len(lengths, n, g.l);
  const bool live = vec < g.vecs && j0 < rows;
  const int64_t c0 = int64_t(vec < g.vecs ? vec : 0) * V;
  float dw[V][K], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) dw[v][k] = 0.0f;
  }
  if (live) {
    const Elem<DT>* xn = x + n * g.xs[0] + c0;
    const Elem<DT>* gn = dy + n * g.dys[0] + c0;
    const int64_t so = n * (K - 1) * int64_t(g.c) + c0;
    const Elem<DT>* sn = state ? state + so : nullptr;
    Elem<DT>* dxn = dx + n * g.l * int64_t(g.c) + c0;
    Taps<DT, V, K> tap;
    tap.load(wp, bp, c0);
    float win[K][V], dpre[K][V];  // X rows t..t+K-1 and dpre of t-K+1..t
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) dpre[k][v] = win[k][v] = 0.0f;
    // rows before the first position whose dpre this run needs, t = j0 - (K-1)
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      const Pack<DT, V> p = load_row<DT, V, K>(xn, sn, g.xs[1], g.c, j0 - 2 * (K - 1) + k, len);
#pragma unroll
      for (int v = 0; v < V; ++v) win[k + 1][v] = to_f<DT>(p.e[v]);
    }
    const int64_t end = j0 + g.run < rows ? j0 + g.run : rows;
    const int64_t touched = end < int64_t(len) + K - 1 ? end : int64_t(len) + K - 1;  // rows past it are 0
    Pack<DT, V> px[kBatch], pg[kBatch], nx[kBatch], ng[kBatch];
    const int64_t first = j0 - (K - 1);
    load_rows<DT, V, K>(px, xn, sn, g.xs[1], g.c, first, j0 < touched ? len : 0);
    load_rows<DT, V, K>(pg, gn, nullptr, g.dys[1], g.c, first, j0 < touched ? len : 0);
    for (int64_t tb = first; tb < touched; tb += kBatch) {
      load_rows<DT, V, K>(nx, xn, sn, g.xs[1], g.c, tb + kBatch, tb + kBatch < touched ? len : 0);
      load_rows<DT, V, K>(ng, gn, nullptr, g.dys[1], g.c, tb + kBatch, tb + kBatch < touched ? len : 0);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t t = tb + i;
        const bool valid = t >= 0 && t < len, own = t >= j0 && t < touched;
        const int64_t fin = t - len;  // row of dfin that belongs to dX row t
        Pack<DT, V> pf{};
        if (own && dfin && fin >= 0 && fin < K - 1) pf = load_pack<DT, V>(dfin + so + fin * int64_t(g.c));
        Pack<DT, V> o;
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
          for (int k = 0; k < K - 1; ++k) {
            win[k][v] = win[k + 1][v];
            dpre[k][v] = dpre[k + 1][v];
          }
          win[K - 1][v] = to_f<DT>(px[i].e[v]);
          float d = to_f<DT>(pg[i].e[v]);
          if (g.act == CNHWC_ACT_SILU) {
            float a = tap.b[v];
#pragma unroll
            for (int k = 0; k < K; ++k) a = __builtin_fmaf(tap.w[v][k], win[k][v], a);
            const float s = sigmoid_for<DT>(a);
            d *= s * __builtin_fmaf(a, 1.0f - s, 1.0f);
          }
          dpre[K - 1][v] = d = valid ? d : 0.0f;
          float r = to_f<DT>(pf.e[v]);
#pragma unroll
          for (int k = 0; k < K; ++k) r = __builtin_fmaf(tap.w[v][k], dpre[K - 1 - k][v], r);
          o.e[v] = from_f<DT>(r);
          // positions before the run are the neighbour's; past the valid ones X
          // may hold anything
          if (own && valid) {
            db[v] += d;
#pragma unroll
            for (int k = 0; k < K; ++k) dw[v][k] = __builtin_fmaf(d, win[k][v], dw[v][k]);
          }
        }
        px[i] = nx[i];
        pg[i] = ng[i];
        if (!own) continue;
        if (t < K - 1) {
          if (dstate) store_pack<DT, V>(dstate + so + t * int64_t(g.c), o);
        } else {
          store_pack<DT, V>(dxn + (t - (K - 1)) * int64_t(g.c), o);
        }
      }
    }
    for (int64_t t = j0 > touched ? j0 : touched; t < end; ++t)
      store_pack<DT, V>(dxn + (t - (K - 1)) * int64_t(g.c), Pack<DT, V>{});
  }
  // the two runs of a wavefront, then the wavefronts through LDS in order
  __shared__ float sum[4][kLanes * V * (K + 1)];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float r = add_halves(dw[v][k]);
      if (lane < kLanes) sum[wave][(lane * V + v) * K + k] = r;
    }
    const float r = add_halves(db[v]);
    if (lane < kLanes) sum[wave][kLanes * V * K + lane * V + v] = r;
  }
  __syncthreads();
  float* pr = part + row_id * (int64_t(g.c) * (K + 1));
  const int64_t cb = col * kLanes * V;
  for (int i = threadIdx.x; i < kLanes * V * (K + 1); i += 256) {
    const float r = sum[0][i] + sum[1][i] + sum[2][i] + sum[3][i];
    if (i < kLanes * V * K) {
      if (cb * K + i < int64_t(g.c) * K) pr[cb * K + i] = r;
    } else if (cb + (i - kLanes * V * K) < g.c) {
      pr[int64_t(g.c) * K + cb + (i - kLanes * V * K)] = r;
    }
  }
}

// ---------------------------------------------------------------- host

ConvGeo geo_of(const cnhwc_causal_conv_desc_t& d, int ve) {
  ConvGeo g{};
  g.l = int32_t(d.l);
  g.c = int32_t(d.c);
  g.act = d.activation;
  g.vecs = int32_t(d.c / ve);
  for (int i = 0; i < 2; ++i) {
    g.xs[i] = d.x_stride[i];
    g.dys[i] = d.dy_stride[i];
  }
  return g;
}

// Aligned vectors of rows at these strides.
bool vectors(const cnhwc_causal_conv_desc_t& d, const int64_t (&s)[2], const void* p, int64_t bytes) {
  const int64_t v = bytes / int64_t(dtype_size(d.dtype));
  return aligned(p, bytes) && d.c % v == 0 && (d.n == 1 || s[0] % v == 0) && (d.l == 1 || s[1] % v == 0);
}

// Positions per thread: long runs load fewer rows twice, short ones fill the
// device; `threads` of them for each of the 256 compute units.
int32_t pick_run(int64_t work, int64_t threads, int32_t most) {
  int64_t run = work / (256 * threads);
  run = run < kBatch ? kBatch : (run > most ? most : run);
  return int32_t(ceil_div(run, kBatch) * kBatch);
}
// Measured forward: 4 x 4096 x 4096 bf16 with 512 threads 52 us, 2048 56, 4096 68.
constexpr int64_t kFwdThreads = 512;
// Backward, with two channels to a thread.  What decides is how many of the
// rows are there: batches with lengths leave runs without work, so they are
// cut twice as fine.  Microseconds with 768 / 1536 threads: several sequences of
// several lengths, 5 x 2047 x 2048 f16 38.7 / 32.9, f32 62.1 / 49.0, 6 x 8000 x
// 512 f32 66.5 / 48.5, bf16 34.0 / 29.0 (against it: 8 x 2047 x 2048 f32 86 to 89 / 94);
// without lengths 2 x 2048 x 2048 f16 24.2 / 27.5, f32 30.1 / 34.9, 3 x 1000 x
// 2048 f32 23.5 / 29.0, bf16 18.2 / 22.2, 4 x 4096 x 4096 bf16 and f32 the same
// (against it: 8 x 2047 x 2048 f32 142 / 112); one sequence with its length 1 x
// 4000 x 2048 bf16 23.0 / 25.8, f32 38.1 / 36.2.  (Four f16 channels to a
// thread, in more registers: the first case 35 at best.  Batches of eight rows: 51.
// Occupancy bounds of 3 and 4 wavefronts: 90 and 195, registers spilled.)
constexpr int kBwdChannels = 2;
int64_t bwd_threads(int64_t n, bool lengths) { return lengths && n > 1 ? 1536 : 768; }

template <int N>
using Int = std::integral_constant<int, N>;

template <typename F>
void with_taps(int32_t k, F&& f) {
  switch (k) {
    case 1: f(Int<1>{}); break;
    case 2: f(Int<2>{}); break;
    case 3: f(Int<3>{}); break;
    case 4: f(Int<4>{}); break;
    case 5: f(Int<5>{}); break;
    case 6: f(Int<6>{}); break;
    case 7: f(Int<7>{}); break;
    default: f(Int<8>{}); break;
  }
}

template <int DT, int V>
hipError_t conv_fwd_t(const cnhwc_causal_conv_desc_t& d, const void* x, const void* w, const void* b,
                      const void* state, const int32_t* lengths, void* y, void* state_out, hipStream_t st) {
  using E = Elem<DT>;
  ConvGeo g = geo_of(d, V);
  g.run = pick_run(d.n * d.l * g.vecs, kFwdThreads, 32);
  g.runs = ceil_div(d.l, g.run);
  const int64_t total = d.n * g.runs * g.vecs;
  with_taps(d.k, [&](auto k) {
    hipLaunchKernelGGL((conv_fwd_kernel<DT, V, decltype(k)::value>), grid_of(ceil_div(total, 256)), dim3(256),
                       0, st, static_cast<const E*>(x), static_cast<const E*>(w), static_cast<const E*>(b),
                       static_cast<const E*>(state), lengths, static_cast<E*>(y), static_cast<E*>(state_out), g,
                       total);
  });
  return hipGetLastError();
}

template <int DT, int V>
hipError_t conv_step_t(const cnhwc_causal_conv_desc_t& d, const void* x, const void* state, const void* w,
                       const void* b, void* y, void* state_out, hipStream_t st) {
  using E = Elem<DT>;
  const ConvGeo g = geo_of(d, V);
  const int64_t total = d.n * g.vecs;
  with_taps(d.k, [&](auto k) {
    hipLaunchKernelGGL((conv_step_kernel<DT, V, decltype(k)::value>), grid_of(ceil_div(total, 256)), dim3(256),
                       0, st, static_cast<const E*>(x), static_cast<const E*>(state), static_cast<const E*>(w),
                       static_cast<const E*>(b), static_cast<E*>(y), static_cast<E*>(state_out), g, total);
  });
  return hipGetLastError();
}

// Run length and workgroups per sequence of the backward pass.
void bwd_runs(const cnhwc_causal_conv_desc_t& d, int64_t ve, bool lengths, int32_t* run, int64_t* blocks) {
  const int64_t rows = d.l + d.k - 1;
  *run = pick_run(d.n * rows * ceil_div(d.c, ve), bwd_threads(d.n, lengths), 64);
  *blocks = ceil_div(rows, int64_t(*run) * kRunsPerBlock);
}

// Workgroups of one launch: 2^31 threads, where a launch takes fewer than 2^32.
// Every sequence has a workgroup of its own at least, so very many short ones
// take several launches.
constexpr int64_t kMostBlocks = 1ll << 23;

template <int DT, int V>
hipError_t conv_bwd_t(const cnhwc_causal_conv_desc_t& d, const void* dy, const void* dfin, const void* x,
                      const void* w, const void* b, const void* state, const int32_t* lengths, void* dx, void* dw,
                      void* db, void* dstate, float* part, hipStream_t st) {
  using E = Elem<DT>;
  ConvGeo g = geo_of(d, V);
  bwd_runs(d, V, lengths != nullptr, &g.run, &g.runs);
  const int64_t cols = ceil_div(g.vecs, kLanes), parts = d.n * g.runs;
  for (int64_t first = 0; first < cols * parts; first += kMostBlocks) {
    const int64_t blocks = cols * parts - first < kMostBlocks ? cols * parts - first : kMostBlocks;
    with_taps(d.k, [&](auto k) {
      constexpr int K = decltype(k)::value;
      if constexpr (V == 1 || K <= 4)  // more taps than four hold too many registers with vectors
        hipLaunchKernelGGL((conv_bwd_kernel<DT, V, K>), dim3(unsigned(blocks)), dim3(256), 0, st,
                           static_cast<const E*>(dy), static_cast<const E*>(dfin), static_cast<const E*>(x),
                           static_cast<const E*>(w), static_cast<const E*>(b), static_cast<const E*>(state), lengths,
                           static_cast<E*>(dx), static_cast<E*>(dstate), part, g, cols, first);
    });
    // the sums would read rows that a failed launch did not write
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  sum_parts<DT>(part, parts, SumOut{{dw, db, nullptr}, {d.c * d.k, d.c, 0}}, false, st);
  return hipGetLastError();
}

cnhwc_status_t check_desc(const cnhwc_causal_conv_desc_t* d, bool bwd) {
  if (!d || !dtype_ok(d->dtype) || d->reserved != 0) return CNHWC_ERR_INVALID_ARGUMENT;
  if (d->activation != CNHWC_ACT_NONE && d->activation != CNHWC_ACT_SILU) return CNHWC_ERR_INVALID_ARGUMENT;
  if (!extent_ok(d->n) || !extent_ok(d->l) || !extent_ok(d->c) || d->k < 1) return CNHWC_ERR_INVALID_ARGUMENT;
  if (!strides_ok(d->n, d->l, d->c, d->x_stride)) return CNHWC_ERR_INVALID_ARGUMENT;
  if (bwd && !strides_ok(d->n, d->l, d->c, d->dy_stride)) return CNHWC_ERR_INVALID_ARGUMENT;
  if (d->k > CNHWC_CAUSAL_CONV_MAX_K) return CNHWC_ERR_UNSUPPORTED;
  // positions fit 32 bits with the run's overhang, the workgroups of the backward
  // pass and the elements 64, and the grid of its reduction stays in range
  if (d->l > INT_MAX - 1024 || d->c > (1ll << 23) || !dense_ok(d->n, d->l + d->k, d->c) ||
      d->n * (d->l + d->k) * d->c > (1ll << 37))
    return CNHWC_ERR_UNSUPPORTED;
  return CNHWC_OK;
}

// The K-1 state rows of every sequence, in bytes.
uint64_t state_bytes(const cnhwc_causal_conv_desc_t& d) {
  return uint64_t(d.n) * (d.k - 1) * d.c * dtype_size(d.dtype);
}

}  // namespace
}  // namespace seq
}  // namespace cnhwc

using namespace cnhwc;
using namespace cnhwc::seq;

// With one tap there is no state: its pointers are not looked at.
extern "C" cnhwc_status_t cnhwc_causal_conv_fwd(const cnhwc_causal_conv_desc_t* desc, const void* x, const void* w,
                                                const void* bias, const void* state, const int32_t* lengths,
                                                void* y, void* state_out, void* hip_stream) {
  const cnhwc_status_t st = check_desc(desc, false);
  if (st != CNHWC_OK) return st;
  const cnhwc_causal_conv_desc_t& d = *desc;
  if (d.k == 1) state = nullptr, state_out = nullptr;
  const uint64_t es = dtype_size(d.dtype);
  Buffers bf;
  bf.in(x, span(d.n, d.l, d.c, d.x_stride) * es, es, true);
  bf.in(w, uint64_t(d.c) * d.k * es, es, true);
  bf.in(bias, d.c * es, es, false);
  bf.in(state, state_bytes(d), es, false);
  bf.in(lengths, d.n * 4, 4, false);
  bf.out(y, uint64_t(d.n) * d.l * d.c * es, es, true);
  bf.out(state_out, state_bytes(d), es, false);
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  const bool vec = vectors(d, d.x_stride, x, 16) && aligned(w, 16) && aligned(bias, 16) && aligned(state, 16) &&
                   aligned(y, 16) && aligned(state_out, 16);
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  hipError_t e;
  if (d.dtype == CNHWC_F32)
    e = vec ? conv_fwd_t<CNHWC_F32, 4>(d, x, w, bias, state, lengths, y, state_out, s)
            : conv_fwd_t<CNHWC_F32, 1>(d, x, w, bias, state, lengths, y, state_out, s);
  else if (d.dtype == CNHWC_F16)
    e = vec ? conv_fwd_t<CNHWC_F16, 8>(d, x, w, bias, state, lengths, y, state_out, s)
            : conv_fwd_t<CNHWC_F16, 1>(d, x, w, bias, state, lengths, y, state_out, s);
  else
    e = vec ? conv_fwd_t<CNHWC_BF16, 8>(d, x, w, bias, state, lengths, y, state_out, s)
            : conv_fwd_t<CNHWC_BF16, 1>(d, x, w, bias, state, lengths, y, state_out, s);
  return e == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
}

extern "C" cnhwc_status_t cnhwc_causal_conv_bwd_workspace(const cnhwc_causal_conv_desc_t* desc, uint64_t* bytes) {
  const cnhwc_status_t st = check_desc(desc, true);
  if (st != CNHWC_OK) return st;
  if (!bytes) return CNHWC_ERR_INVALID_ARGUMENT;
  // the vector and the element form alike, with and without lengths: which one
  // runs depends on the pointers
  uint64_t most = 0;
  for (int64_t ve : {int64_t(1), int64_t(kBwdChannels)})
    for (bool lengths : {false, true}) {
      int32_t run;
      int64_t blocks;
      bwd_runs(*desc, ve, lengths, &run, &blocks);
      const uint64_t b = uint64_t(desc->n) * blocks * (uint64_t(desc->c) * (desc->k + 1)) * 4;
      most = b > most ? b : most;
    }
  *bytes = most;
  return CNHWC_OK;
}

extern "C" cnhwc_status_t cnhwc_causal_conv_bwd(const cnhwc_causal_conv_desc_t* desc, const void* dy,
                                                const void* dstate_out, const void* x, const void* w,
                                                const void* bias, const void* state, const int32_t* lengths,
                                                void* dx, void* dw, void* dbias, void* dstate, void* workspace,
                                                uint64_t workspace_bytes, void* hip_stream) {
  uint64_t need = 0;
  const cnhwc_status_t st = cnhwc_causal_conv_bwd_workspace(desc, &need);
  if (st != CNHWC_OK) return st;
  const cnhwc_causal_conv_desc_t& d = *desc;
  if (d.k == 1) state = nullptr, dstate_out = nullptr, dstate = nullptr;
  if ((bias == nullptr) != (dbias == nullptr)) return CNHWC_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < need) return CNHWC_ERR_WORKSPACE_TOO_SMALL;
  const uint64_t es = dtype_size(d.dtype);
  Buffers bf;
  bf.in(dy, span(d.n, d.l, d.c, d.dy_stride) * es, es, true);
  bf.in(dstate_out, state_bytes(d), es, false);
  bf.in(x, span(d.n, d.l, d.c, d.x_stride) * es, es, true);
  bf.in(w, uint64_t(d.c) * d.k * es, es, true);
  bf.in(bias, d.c * es, es, false);
  bf.in(state, state_bytes(d), es, false);
  bf.in(lengths, d.n * 4, 4, false);
  bf.out(dx, uint64_t(d.n) * d.l * d.c * es, es, true);
  bf.out(dw, uint64_t(d.c) * d.k * es, es, true);
  bf.out(dbias, d.c * es, es, false);
  bf.out(dstate, state_bytes(d), es, false);
  bf.out(workspace, need, 16, true);
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  const int64_t bytes = kBwdChannels * int64_t(es);
  const bool vec = d.k <= 4 && vectors(d, d.x_stride, x, bytes) && vectors(d, d.dy_stride, dy, bytes) &&
                   aligned(dstate_out, bytes) && aligned(w, bytes) && aligned(bias, bytes) && aligned(state, bytes) &&
                   aligned(dx, bytes) && aligned(dstate, bytes);
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  float* part = static_cast<float*>(workspace);
  hipError_t e;
  auto run = [&](auto dt, auto v) {
    return conv_bwd_t<decltype(dt)::value, decltype(v)::value>(d, dy, dstate_out, x, w, bias, state, lengths, dx, dw,
                                                               dbias, dstate, part, s);
  };
  if (d.dtype == CNHWC_F32) e = vec ? run(Int<CNHWC_F32>{}, Int<kBwdChannels>{}) : run(Int<CNHWC_F32>{}, Int<1>{});
  else if (d.dtype == CNHWC_F16) e = vec ? run(Int<CNHWC_F16>{}, Int<kBwdChannels>{}) : run(Int<CNHWC_F16>{}, Int<1>{});
  else e = vec ? run(Int<CNHWC_BF16>{}, Int<kBwdChannels>{}) : run(Int<CNHWC_BF16>{}, Int<1>{});
  return e == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
}

extern "C" cnhwc_status_t cnhwc_causal_conv_step(const cnhwc_causal_conv_desc_t* desc, const void* x,
                                                 const void* state, const void* w, const void* bias, void* y,
                                                 void* state_out, void* hip_stream) {
  const cnhwc_status_t st = check_desc(desc, false);
  if (st != CNHWC_OK) return st;
  const cnhwc_causal_conv_desc_t& d = *desc;
  if (d.l != 1) return CNHWC_ERR_INVALID_ARGUMENT;
  if (d.k == 1) state = nullptr, state_out = nullptr;
  const uint64_t es = dtype_size(d.dtype);
  Buffers bf;
  bf.in(x, span(d.n, d.l, d.c, d.x_stride) * es, es, true);
  if (state != state_out) bf.in(state, state_bytes(d), es, true);
  bf.in(w, uint64_t(d.c) * d.k * es, es, true);
  bf.in(bias, d.c * es, es, false);
  bf.out(y, uint64_t(d.n) * d.c * es, es, true);
  bf.out(state_out, state_bytes(d), es, d.k > 1);
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  const bool vec = vectors(d, d.x_stride, x, 16) && aligned(w, 16) && aligned(bias, 16) && aligned(state, 16) &&
                   aligned(y, 16) && aligned(state_out, 16);
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  hipError_t e;
  if (d.dtype == CNHWC_F32)
    e = vec ? conv_step_t<CNHWC_F32, 4>(d, x, state, w, bias, y, state_out, s)
            : conv_step_t<CNHWC_F32, 1>(d, x, state, w, bias, y, state_out, s);
  else if (d.dtype == CNHWC_F16)
    e = vec ? conv_step_t<CNHWC_F16, 8>(d, x, state, w, bias, y, state_out, s)
            : conv_step_t<CNHWC_F16, 1>(d, x, state, w, bias, y, state_out, s);
  else
    e = vec ? conv_step_t<CNHWC_BF16, 8>(d, x, state, w, bias, y, state_out, s)
            : conv_step_t<CNHWC_BF16, 1>(d, x, state, w, bias, y, state_out, s);
  return e == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
}
