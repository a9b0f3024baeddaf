// Selective state space scan, forward, backward and single tokens, for gfx950.
//
//   D[t,d] = softplus(delta[t,d] + delta_bias[d])
//   h[t,d,s] = e[t,d,s] h[t-1,d,s] + D[t,d] u[t,d] b[t,s],  e = exp(D[t,d] a[d,s])
//   y[t,d] = (sum_s c[t,s] h[t,d,s] + skip[d] u[t,d]) silu(gate[t,d])
//
// Every channel and state has its own decay, so no product over t or s has the
// form of a matrix product: the work is vector instructions.  Per position,
// channel and state the forward pass needs four products and sums and one
// exponential, which counts as two (measured: 4.4 cycles a wavefront for a
// product and sum, 9.0 for an exponential).
//
// A wavefront holds 64 / SL groups of SL lanes; a group holds four channels and
// SL * SPL states, each lane SPL states of all four channels.  So per position a
// lane reads b and c for its own states once for four channels, the sum over
// the states is log2(SL) lane permutations for every SPL terms, and what
// belongs to a channel alone (softplus, gate, loads and stores) is done once
// by the four lanes of a quad, one channel each, and handed round by quad
// permutations.  b and c come through LDS, converted once per workgroup.
//
// Long sequences are cut into chunks.  One kernel runs each chunk from a zero
// state and leaves the chunk's end state and sum of D; a second one, along the
// chunks, turns these into the state that enters every chunk (a chunk scales
// what enters it by exp(a sum D)); the last runs each chunk from there.
//
// Measured, 1 x 16384 x 2048 channels x 16 states, bf16: 279 us (7982 us in one
// chunk), of them 111 the local chunks, 13 the join, 155 the outputs (each of
// them launched by itself, again and again).  The vector pipes are busy 81 and
// 83% of the kernels' cycles; the bytes that have to move (270 MB) would take 56 us.
// Positions past a sequence's length go through all of it: 6 sequences of 1023
// x 1000 x 16 fp32 of which 2449 of 6138 positions are valid take 72 us (24, 8, 39).
#include <hip/hip_runtime.h>

#include <cfloat>
#include <climits>

#include "internal.hpp"
#include "seq_common.hpp"
#include "seq_host.hpp"

namespace cnhwc {
namespace seq {
namespace {

constexpr int kTile = 8;    // positions whose loads are issued together
constexpr int kHalf = kTile / 2;
constexpr int kWaves = 4;   // wavefronts of a workgroup
constexpr float kLog2e = 1.44269504f;
constexpr float kLn2 = 0.693147181f;

struct ScanGeo {
  int32_t l, d, s, softplus;
  int32_t chunk;         // positions per chunk, a multiple of kTile
  int32_t chunks;        // per sequence
  int32_t col_blocks;    // workgroups along the channels
  int64_t us[2], ds[2], bs[2], cs[2], gs[2], ys[2];
};

template <int DT>
struct ScanIn {
  const Elem<DT>* u;
  const Elem<DT>* delta;
  const float* a;
  const Elem<DT>* b;
  const Elem<DT>* c;
  const float* skip;
  const Elem<DT>* gate;
  const float* delta_bias;
  const float* state;
  const int32_t* lengths;
};

// Where a thread stands: its group's four channels, its own channel of them,
// its states.
template <int SL, int SPL>
struct Place {
  static constexpr int kChannels = 64 / SL * 4;  // per wavefront
  int32_t dq, d, s0;
  uint32_t at;  // the own channel to load from: the last one where it does not exist
  bool live;    // the own channel exists
  bool first;   // this lane stores for its channel
  __device__ __forceinline__ Place(int32_t wave_d0, int32_t d_all) {
    const int lane = threadIdx.x & 63;
    dq = wave_d0 + lane / SL * 4;
    d = dq + (lane & 3);
    s0 = lane % SL * SPL;
    live = d < d_all;
    first = lane % SL < 4 && live;
    at = live ? d : d_all - 1;
  }
};

// The own channel's elements of a tile of positions (0 past the valid ones);
// row: the sequence's first position, uniform over the wavefront.
template <int DT>
__device__ __forceinline__ void load_tile(Elem<DT> (&v)[kTile], const Elem<DT>* __restrict__ row, int64_t stride,
                                          uint32_t d, int32_t t0, int32_t t_valid) {
  if (t0 + kTile <= t_valid) {
#pragma unroll
    for (int i = 0; i < kTile; ++i) v[i] = (row + (t0 + i) * stride)[d];
  } else {
#pragma unroll
    for (int i = 0; i < kTile; ++i) v[i] = t0 + i < t_valid ? (row + (t0 + i) * stride)[d] : Elem<DT>(0);
  }
}

// The [D,S] values of a thread's four channels by SPL states; zero outside.
template <int SL, int SPL>
__device__ __forceinline__ void load_states(float (&h)[4][SPL], const float* __restrict__ p, const Place<SL, SPL>& at,
                                            const ScanGeo& g) {
  const bool whole = SPL == 4 && g.s == SL * SPL && aligned16(p);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t base = int64_t(at.dq + j) * g.s + at.s0;
    if (whole) {
      float4 v = make_float4(0, 0, 0, 0);
      if (at.dq + j < g.d) v = *reinterpret_cast<const float4*>(p + base);
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < SPL; ++i) h[j][i] = f[i];
    } else {
#pragma unroll
      for (int i = 0; i < SPL; ++i) h[j][i] = at.dq + j < g.d && at.s0 + i < g.s ? p[base + i] : 0.0f;
    }
  }
}

template <int SL, int SPL>
__device__ __forceinline__ void store_states(const float (&h)[4][SPL], float* __restrict__ p, const Place<SL, SPL>& at,
                                             const ScanGeo& g) {
  const bool whole = SPL == 4 && g.s == SL * SPL && aligned16(p);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t base = int64_t(at.dq + j) * g.s + at.s0;
    if (at.dq + j >= g.d) continue;
    if (whole) {
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = h[j][i < SPL ? i : 0];
      *reinterpret_cast<float4*>(p + base) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
#pragma unroll
      for (int i = 0; i < SPL; ++i)
        if (at.s0 + i < g.s) p[base + i] = h[j][i];
    }
  }
}

// The values are computed here and not later: without this the compiler moves
// a tile's whole arithmetic behind the next tile's staging and holds the
// operands of all its positions in registers meanwhile.
template <int N>
__device__ __forceinline__ void settle(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(v[i]));
}
template <int SPL>
__device__ __forceinline__ void settle(float (&h)[4][SPL]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) settle(h[j]);
}

// a log2(e), finite for a of minus infinity too: where D is 0, as past the
// valid positions, the state stands still, and 0 times infinity is no number.
__device__ __forceinline__ float rate(float a) {
  const float r = a * kLog2e;
  return r < -FLT_MAX ? -FLT_MAX : r;
}
template <int SPL>
__device__ __forceinline__ void rates(float (&a)[4][SPL]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < SPL; ++i) a[j][i] = rate(a[j][i]);
}

template <int SPL>
__device__ __forceinline__ void copy(const float (&from)[4][SPL], float (&to)[4][SPL]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < SPL; ++i) to[j][i] = from[j][i];
}

// The value of lane j of the quad (j a constant after unrolling): as an operand
// of a product it costs no instruction of its own.
__device__ __forceinline__ float quad_lane(float v, int j) {
  switch (j) {
    case 0: return dpp<0 * kQuadBcast>(v);
    case 1: return dpp<1 * kQuadBcast>(v);
    case 2: return dpp<2 * kQuadBcast>(v);
    default: return dpp<3 * kQuadBcast>(v);
  }
}

// Four channels by SPL states per lane, in the order of the lanes:
// [workgroup][wavefront][SPL][64 lanes] of the four channels' values.
template <int SPL>
__device__ __forceinline__ int64_t lane_order(int64_t workgroup) {
  return (workgroup * kWaves + (threadIdx.x >> 6)) * (SPL * 64) + (threadIdx.x & 63);
}
template <int SPL>
__device__ __forceinline__ void put_lanes(float4* __restrict__ p, int64_t workgroup, const float (&h)[4][SPL]) {
  const int64_t at = lane_order<SPL>(workgroup);
#pragma unroll
  for (int i = 0; i < SPL; ++i) p[at + i * 64] = make_float4(h[0][i], h[1][i], h[2][i], h[3][i]);
}
template <int SPL>
__device__ __forceinline__ void get_lanes(const float4* __restrict__ p, int64_t workgroup, float (&h)[4][SPL]) {
  const int64_t at = lane_order<SPL>(workgroup);
#pragma unroll
  for (int i = 0; i < SPL; ++i) {
    const float4 f = p[at + i * 64];
    h[0][i] = f.x, h[1][i] = f.y, h[2][i] = f.z, h[3][i] = f.w;
  }
}

// Of the four channels' sums over the group's lanes, the own channel's: lanes
// trade the channels that are not theirs, so the four sums take three additions.
template <int SL>
__device__ __forceinline__ float own_sum(const float (&v)[4]) {
  const bool odd = threadIdx.x & 1, upper = threadIdx.x & 2;
  const float p = (odd ? v[1] : v[0]) + dpp<kQuadXor1>(odd ? v[0] : v[1]);
  const float q = (odd ? v[3] : v[2]) + dpp<kQuadXor1>(odd ? v[2] : v[3]);
  float r = (upper ? q : p) + dpp<kQuadXor2>(upper ? p : q);
  if constexpr (SL >= 8) r += dpp<kHalfMirror>(dpp<kQuadReverse>(r));  // lane ^ 4
  if constexpr (SL >= 16) r += dpp<kRor8>(r);
  return r;
}

// b and c of a tile of positions in LDS as floats, zero past the valid
// positions and past S.  stage() issues the loads, put() writes them.
template <int DT, int NS>
struct StagedBC {
  static constexpr int kAll = kTile * 2 * NS;
  static constexpr int kPer = (kAll + 255) / 256;
  Elem<DT> v[kPer];
  __device__ __forceinline__ void stage(const Elem<DT>* __restrict__ b, const Elem<DT>* __restrict__ c,
                                        const ScanGeo& g, int32_t t0, int32_t end) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = threadIdx.x + k * 256;
      const int s = i % NS, which = i / NS % 2, t = t0 + i / (2 * NS);
      v[k] = Elem<DT>(0);
      if (i < kAll && s < g.s && t < end) v[k] = which ? c[t * g.cs[1] + s] : b[t * g.bs[1] + s];
    }
  }
  __device__ __forceinline__ void put(float* lds) const {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = threadIdx.x + k * 256;
      if (i < kAll) lds[i] = to_f<DT>(v[k]);
    }
  }
};

template <int SPL>
__device__ __forceinline__ void lds_states(const float* p, float (&f)[SPL]) {
  if constexpr (SPL == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < SPL; ++i) f[i] = p[i];
  }
}

// Workgroup -> sequence, chunk, first channel of this wavefront.
template <int SL, int SPL>
__device__ __forceinline__ void locate(const ScanGeo& g, int32_t chunks, int64_t& n, int32_t& chunk,
                                       int32_t& wave_d0) {
  const int64_t row = blockIdx.x / g.col_blocks;
  const int32_t col = int32_t(blockIdx.x - row * g.col_blocks);
  n = row / chunks;
  chunk = int32_t(row - n * chunks);
  wave_d0 = __builtin_amdgcn_readfirstlane((col * kWaves + int32_t(threadIdx.x >> 6)) * Place<SL, SPL>::kChannels);
}

// ---------------------------------------------------------------- forward

// LOCAL: every chunk but the last of its sequence from a zero state; its end
// state and sum of D, in lane order.  Otherwise the outputs, from the entering
// states (the first chunk's is the initial one), and the final state.
template <int DT, int SL, int SPL, bool LOCAL>
__global__ __launch_bounds__(256) void scan_fwd_kernel(ScanIn<DT> in, ScanGeo g, Elem<DT>* __restrict__ y,
                                                       float4* __restrict__ states, float* __restrict__ sums,
                                                       float* __restrict__ state_out) {
  constexpr int NS = SL * SPL;
  __shared__ __attribute__((aligned(16))) float bc[2][kTile * 2 * NS];
  int64_t n;
  int32_t chunk, wave_d0;
  locate<SL, SPL>(g, LOCAL ? g.chunks - 1 : g.chunks, n, chunk, wave_d0);
  const Place<SL, SPL> at(wave_d0, g.d);
  const int32_t len = valid_len(in.lengths, n, g.l);
  const int32_t t_begin = chunk * g.chunk;
  const int32_t t_end = t_begin + g.chunk < g.l ? t_begin + g.chunk : g.l;
  const int32_t t_valid = t_end < len ? t_end : len;

  float a2[4][SPL], h[4][SPL];
  load_states<SL, SPL>(a2, in.a, at, g);
  rates(a2);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < SPL; ++i) h[j][i] = 0.0f;
  const int64_t ds = int64_t(g.d) * g.s;
  if constexpr (!LOCAL) {
    if (chunk > 0) get_lanes<SPL>(states, blockIdx.x, h);
    else if (in.state) load_states<SL, SPL>(h, in.state + n * ds, at, g);
  }
  const float bias = in.delta_bias ? in.delta_bias[at.at] : 0.0f;
  const float skip = !LOCAL && in.skip ? in.skip[at.at] : 0.0f;
  const Elem<DT>* un = in.u + n * g.us[0];
  const Elem<DT>* dn = in.delta + n * g.ds[0];
  const Elem<DT>* gn = !LOCAL && in.gate ? in.gate + n * g.gs[0] : nullptr;
  const Elem<DT>* bn = in.b + n * g.bs[0];
  const Elem<DT>* cn = in.c + n * g.cs[0];
  Elem<DT>* yn = LOCAL ? nullptr : y + n * g.l * int64_t(g.d);

  Elem<DT> u_t[kTile], d_t[kTile], g_t[kTile] = {};
  StagedBC<DT, NS> st;
  auto fetch = [&](int32_t t0) {
    st.stage(bn, cn, g, t0, t_valid);
    load_tile<DT>(u_t, un, g.us[1], at.at, t0, t_valid);
    load_tile<DT>(d_t, dn, g.ds[1], at.at, t0, t_valid);
    if (gn) load_tile<DT>(g_t, gn, g.gs[1], at.at, t0, t_valid);
  };
  float sum = 0.0f;
  fetch(t_begin);
  st.put(bc[0]);
  __syncthreads();
  int buf = 0;
  for (int32_t t0 = t_begin; t0 < t_end; t0 += kTile, buf ^= 1) {
    // what belongs to a channel alone, for the whole tile: D, u, and the gate's factor
    float uf[kTile], df[kTile], gf[kTile];
#pragma unroll
    for (int i = 0; i < kTile; ++i) {
      uf[i] = to_f<DT>(u_t[i]);
      df[i] = to_f<DT>(d_t[i]) + bias;
      gf[i] = to_f<DT>(g_t[i]);
    }
    if (t0 + kTile < t_end) fetch(t0 + kTile);
    if (g.softplus) {
#pragma unroll
      for (int i = 0; i < kTile; ++i) df[i] = softplus(df[i]);
    }
    if (!LOCAL && in.gate) {
#pragma unroll
      for (int i = 0; i < kTile; ++i) gf[i] *= sigmoid_for<DT>(gf[i]);
    }
#pragma unroll
    for (int i = 0; i < kTile; ++i) {
      const bool valid = t0 + i < t_valid;
      const float dl = valid && at.live ? df[i] : 0.0f;
      const float dx = dl * uf[i];
      if (LOCAL) sum += dl;
      float bf[SPL], cf[SPL], yq[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      lds_states<SPL>(&bc[buf][i * 2 * NS + at.s0], bf);
      if (!LOCAL) lds_states<SPL>(&bc[buf][i * 2 * NS + NS + at.s0], cf);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < SPL; ++k) {
          const float e = __builtin_amdgcn_exp2f(quad_lane(dl, j) * a2[j][k]);
          h[j][k] = __builtin_fmaf(e, h[j][k], quad_lane(dx, j) * bf[k]);
          if (!LOCAL) yq[j] = __builtin_fmaf(h[j][k], cf[k], yq[j]);
        }
      settle(h);
      if constexpr (!LOCAL) {
        float v = __builtin_fmaf(skip, uf[i], own_sum<SL>(yq));
        if (in.gate) v *= gf[i];
        if (at.first && t0 + i < t_end) (yn + (t0 + i) * int64_t(g.d))[at.at] = from_f<DT>(valid ? v : 0.0f);
      }
    }
    if (t0 + kTile < t_end) st.put(bc[buf ^ 1]);
    __syncthreads();
  }
  if constexpr (LOCAL) {
    // at the next chunk's place, which this chunk's end enters
    const int64_t next = blockIdx.x + (n + 1) * g.col_blocks;
    put_lanes<SPL>(states, next, h);
    sums[next * 256 + threadIdx.x] = sum;
  } else {
    if (state_out && chunk == g.chunks - 1) store_states<SL, SPL>(h, state_out + n * ds, at, g);
  }
}

// One value of the lane order: its sequence, place within a workgroup's chunks,
// channel, state and decay.
template <int SL, int SPL>
struct Column {
  int64_t n, at, step;      // first chunk's float in the lane order, floats to the next chunk
  int64_t sum_at, sum_step;
  int64_t user;             // in [N,D,S]
  float a2;
  bool live;
  __device__ __forceinline__ Column(int64_t id, const float* __restrict__ a, const ScanGeo& g) {
    constexpr int kWave = SPL * 64 * 4, kGroup = kWaves * kWave;  // floats
    const int64_t per = int64_t(g.col_blocks) * kGroup;
    n = id / per;
    const int64_t r = id - n * per;
    const int32_t wave = int32_t(r / kWave), q = int32_t(r % kWave);  // wavefront along the channels
    const int32_t i = q / 256, lane = q / 4 % 64, j = q % 4;
    const int64_t d = int64_t(wave) * Place<SL, SPL>::kChannels + lane / SL * 4 + j;
    const int32_t s = lane % SL * SPL + i;
    at = n * g.chunks * per + r;
    step = per;
    sum_at = (n * g.chunks * int64_t(g.col_blocks) * kWaves + wave) * 64 + (lane & ~3) + j;
    sum_step = int64_t(g.col_blocks) * kWaves * 64;
    live = d < g.d && s < g.s;
    user = (n * g.d + d) * g.s + s;
    a2 = live ? rate(a[d * g.s + s]) : 0.0f;
  }
};

// The entering states of one value, in place, from its chunks' end states and
// sums of D, of which chunk k's stand at k + ahead; returns the final state
// where ahead is 0.  The chunks' values are loaded kJoin at a time: only the sum
// along them is serial.
constexpr int kJoin = 16;
template <int SL, int SPL>
__device__ __forceinline__ float join_forward(float* states, const float* sums, float h, const Column<SL, SPL>& c,
                                              const ScanGeo& g, int ahead) {
  for (int32_t k0 = ahead; k0 < g.chunks; k0 += kJoin) {
    float p[kJoin], e[kJoin];
#pragma unroll
    for (int i = 0; i < kJoin; ++i) {
      const bool ok = k0 + i < g.chunks;
      p[i] = ok ? states[c.at + (k0 + i) * c.step] : 0.0f;
      e[i] = ok ? sums[c.sum_at + (k0 + i) * c.sum_step] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kJoin; ++i) {
      if (k0 + i >= g.chunks) break;
      const float next = __builtin_fmaf(__builtin_amdgcn_exp2f(c.a2 * e[i]), h, p[i]);
      states[c.at + (k0 + i) * c.step] = ahead ? next : h;
      h = next;
    }
  }
  return h;
}

// Along the chunks: the states that enter all but the first.
template <int SL, int SPL>
__global__ __launch_bounds__(256) void scan_join_kernel(float* __restrict__ states, const float* __restrict__ sums,
                                                        const float* __restrict__ a, const float* __restrict__ state,
                                                        ScanGeo g, int64_t total) {
  for (int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x; id < total; id += int64_t(gridDim.x) * 256) {
    const Column<SL, SPL> c(id, a, g);
    join_forward(states, sums, state && c.live ? state[c.user] : 0.0f, c, g, 1);
  }
}

// One token: groups of SL lanes by SPL states of one channel each, for NB
// sequences at once, so that a is read once for them and all their loads are in
// flight together.  The state is the traffic: read once, written once.  The
// same operations in the same order as a prompt in one chunk: a prompt fed token
// by token leaves the same bits.
template <int DT, int SL, int SPL, int NB, bool WHOLE>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanIn<DT> in, ScanGeo g, Elem<DT>* __restrict__ y,
                                                        float* state_out, int64_t seqs) {
  constexpr int kGroups = 256 / SL;
  const int s0 = int(threadIdx.x) % SL * SPL;
  const int32_t d = int32_t(blockIdx.x) * kGroups + int32_t(threadIdx.x) / SL;
  if (d >= g.d) return;  // whole groups of SL lanes
  float a2[SPL];
  if constexpr (WHOLE) lds_states<SPL>(in.a + int64_t(d) * g.s + s0, a2);
  else {
#pragma unroll
    for (int k = 0; k < SPL; ++k) a2[k] = s0 + k < g.s ? in.a[int64_t(d) * g.s + s0 + k] : 0.0f;
  }
  const float bias = in.delta_bias ? in.delta_bias[d] : 0.0f;
  const float skip = in.skip ? in.skip[d] : 0.0f;
  for (int64_t n0 = int64_t(blockIdx.y) * NB; n0 < seqs; n0 += int64_t(gridDim.y) * NB) {
    float h[NB][SPL], bf[NB][SPL], cf[NB][SPL], u[NB], dl[NB], z[NB];
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int64_t n = n0 + q < seqs ? n0 + q : seqs - 1;
      const float* hp = in.state + (n * g.d + d) * g.s + s0;
      const Elem<DT>* bp = in.b + n * g.bs[0] + s0;
      const Elem<DT>* cp = in.c + n * g.cs[0] + s0;
      if constexpr (WHOLE) {
        lds_states<SPL>(hp, h[q]);
        const Pack<DT, SPL> pb = load_pack<DT, SPL>(bp), pc = load_pack<DT, SPL>(cp);
#pragma unroll
        for (int k = 0; k < SPL; ++k) bf[q][k] = to_f<DT>(pb.e[k]), cf[q][k] = to_f<DT>(pc.e[k]);
      } else {
#pragma unroll
        for (int k = 0; k < SPL; ++k) {
          const bool ok = s0 + k < g.s;
          h[q][k] = ok ? hp[k] : 0.0f;
          bf[q][k] = ok ? to_f<DT>(bp[k]) : 0.0f;
          cf[q][k] = ok ? to_f<DT>(cp[k]) : 0.0f;
        }
      }
      u[q] = to_f<DT>(in.u[n * g.us[0] + d]);
      dl[q] = to_f<DT>(in.delta[n * g.ds[0] + d]) + bias;
      z[q] = in.gate ? to_f<DT>(in.gate[n * g.gs[0] + d]) : 0.0f;
    }
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int64_t n = n0 + q;
      if (n >= seqs) break;
      if (g.softplus) dl[q] = softplus(dl[q]);
      const float dx = dl[q] * u[q];
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < SPL; ++k) {
        const float e = __builtin_amdgcn_exp2f(dl[q] * rate(a2[k]));
        h[q][k] = __builtin_fmaf(e, h[q][k], dx * bf[q][k]);
        v = __builtin_fmaf(h[q][k], cf[q][k], v);
      }
      float* hp = state_out + (n * g.d + d) * g.s + s0;
      if constexpr (WHOLE) {
        *reinterpret_cast<float4*>(hp) = make_float4(h[q][0], h[q][1], h[q][2], h[q][3]);
      } else {
#pragma unroll
        for (int k = 0; k < SPL; ++k)
          if (s0 + k < g.s) hp[k] = h[q][k];
      }
      v = __builtin_fmaf(skip, u[q], group_sum<SL>(v));
      if (in.gate) v *= z[q] * sigmoid_for<DT>(z[q]);
      if (s0 == 0) y[n * g.d + d] = from_f<DT>(v);
    }
  }
}

// ---------------------------------------------------------------- backward
//
// With gy = dy silu(gate) and g[t] the gradient of h[t], along t from the end:
//   g[t] = c[t] gy[t] + e[t+1] g[t+1]
//   db[t,s] = sum_d g D u,  dc[t,s] = sum_d gy h,  da[d,s] = sum_t g e h[t-1] D,
//   du = D sum_s g b + skip gy,  dD = sum_s g e h[t-1] a + u sum_s g b,
//   dgate = dy y silu'(gate),  dskip = sum_t gy u.
// Nothing is saved by the forward pass.  The chunk kernel runs along t from a
// zero state and, beside the end state, sums what the chunk's outputs pass to
// the state that entered it, sum_t (e[begin] ... e[t]) c[t] gy[t]: the same
// exponentials serve both.  The join kernel then knows the state that enters
// every chunk and the gradient that comes back into its end.

// The state at every tile of a chunk costs less to keep than to run again: the
// chunk kernel leaves it (from its zero start) with the sum of D up to there,
// in the order of its lanes, and the gradient kernel adds what the entering
// state has become by then, one exponential per state and tile.  (Tiles of four
// positions instead of eight move twice the states: 789 us against 710.)
//
// Measured, 8 x 2048 x 2048 channels x 16 states, bf16: 700 us, of them 179 the
// chunk kernel, 14 the join, 489 the gradient (each launched by itself, again
// and again), the rest the two sums.  The gradient
// kernel issues 384 vector instructions per position and wavefront (16 elements
// a lane) and keeps the vector pipes busy 74% of its cycles, with two wavefronts
// to a SIMD (registers); the bytes that have to move (472 MB) would take 98 us.

template <int DT>
struct ScanOut {
  Elem<DT>* u;
  Elem<DT>* delta;
  Elem<DT>* gate;
  float* bc_part;     // [col_blocks][N*L][2][S] sums of db and dc
  float* param_part;  // [N*chunks][D*S | D | D] sums of da, dskip, ddelta_bias
};

// The kept states in lane order, [workgroup][tile], and their sums of D.
struct Kept {
  float4* h;
  float* sum;
};

template <int DT, int SL, int SPL>
__global__ __launch_bounds__(256, 2) void scan_bwd_local_kernel(ScanIn<DT> in, ScanGeo g,
                                                             const Elem<DT>* __restrict__ dy,
                                                             float4* __restrict__ states, float4* __restrict__ backs,
                                                             float* __restrict__ sums, Kept kept) {
  constexpr int NS = SL * SPL;
  __shared__ __attribute__((aligned(16))) float bc[2][kTile * 2 * NS];
  int64_t n;
  int32_t chunk, wave_d0;
  locate<SL, SPL>(g, g.chunks, n, chunk, wave_d0);
  const Place<SL, SPL> at(wave_d0, g.d);
  const int32_t len = valid_len(in.lengths, n, g.l);
  const int32_t t_begin = chunk * g.chunk;
  const int32_t t_end = t_begin + g.chunk < g.l ? t_begin + g.chunk : g.l;
  const int32_t t_valid = t_end < len ? t_end : len;

  float a2[4][SPL], h[4][SPL], p[4][SPL], r[4][SPL];
  load_states<SL, SPL>(a2, in.a, at, g);
  rates(a2);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < SPL; ++i) h[j][i] = 0.0f, p[j][i] = 1.0f, r[j][i] = 0.0f;
  const float bias = in.delta_bias ? in.delta_bias[at.at] : 0.0f;
  const Elem<DT>* un = in.u + n * g.us[0];
  const Elem<DT>* dn = in.delta + n * g.ds[0];
  const Elem<DT>* gn = in.gate ? in.gate + n * g.gs[0] : nullptr;
  const Elem<DT>* yn = dy + n * g.ys[0];
  const Elem<DT>* bn = in.b + n * g.bs[0];
  const Elem<DT>* cn = in.c + n * g.cs[0];

  Elem<DT> u_t[kTile], d_t[kTile], g_t[kTile] = {}, y_t[kTile];
  StagedBC<DT, NS> st;
  auto fetch = [&](int32_t t0) {
    st.stage(bn, cn, g, t0, t_valid);
    load_tile<DT>(u_t, un, g.us[1], at.at, t0, t_valid);
    load_tile<DT>(d_t, dn, g.ds[1], at.at, t0, t_valid);
    load_tile<DT>(y_t, yn, g.ys[1], at.at, t0, t_valid);
    if (gn) load_tile<DT>(g_t, gn, g.gs[1], at.at, t0, t_valid);
  };
  float sum = 0.0f;
  fetch(t_begin);
  st.put(bc[0]);
  __syncthreads();
  int buf = 0;
  for (int32_t t0 = t_begin; t0 < t_valid; t0 += kTile, buf ^= 1) {
    if (t0 > t_begin) {
      const int64_t k = int64_t(blockIdx.x) * (g.chunk / kTile) + (t0 - t_begin) / kTile;
      put_lanes<SPL>(kept.h, k, h);
      kept.sum[k * 256 + threadIdx.x] = sum;
    }
    float uf[kTile], df[kTile], gf[kTile], yf[kTile];
#pragma unroll
    for (int i = 0; i < kTile; ++i) {
      uf[i] = to_f<DT>(u_t[i]);
      df[i] = to_f<DT>(d_t[i]) + bias;
      gf[i] = to_f<DT>(g_t[i]);
      yf[i] = to_f<DT>(y_t[i]);
    }
    if (t0 + kTile < t_valid) fetch(t0 + kTile);
    if (g.softplus) {
#pragma unroll
      for (int i = 0; i < kTile; ++i) df[i] = softplus(df[i]);
    }
    if (in.gate) {
#pragma unroll
      for (int i = 0; i < kTile; ++i) yf[i] *= gf[i] * sigmoid_for<DT>(gf[i]);
    }
#pragma unroll
    for (int i = 0; i < kTile; ++i) {
      const float dl = t0 + i < t_valid && at.live ? df[i] : 0.0f;
      const float dx = dl * uf[i];
      sum += dl;
      float bf[SPL], cf[SPL];
      lds_states<SPL>(&bc[buf][i * 2 * NS + at.s0], bf);
      lds_states<SPL>(&bc[buf][i * 2 * NS + NS + at.s0], cf);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < SPL; ++k) {
          const float e = __builtin_amdgcn_exp2f(quad_lane(dl, j) * a2[j][k]);
          h[j][k] = __builtin_fmaf(e, h[j][k], quad_lane(dx, j) * bf[k]);
          p[j][k] *= e;
          r[j][k] = __builtin_fmaf(p[j][k], quad_lane(yf[i], j) * cf[k], r[j][k]);
        }
      settle(h);
      settle(r);
    }
    if (t0 + kTile < t_valid) st.put(bc[buf ^ 1]);
    __syncthreads();
  }
  put_lanes<SPL>(states, blockIdx.x, h);
  put_lanes<SPL>(backs, blockIdx.x, r);
  sums[int64_t(blockIdx.x) * 256 + threadIdx.x] = sum;
}

// In place: ends -> entering states; what each chunk passes back -> the
// gradient that enters at its end.  dstate: the initial state's gradient.
template <int SL, int SPL>
__global__ __launch_bounds__(256) void scan_bwd_join_kernel(float* __restrict__ states, float* __restrict__ backs,
                                                            const float* __restrict__ sums,
                                                            const float* __restrict__ a,
                                                            const float* __restrict__ state,
                                                            const float* __restrict__ dstate_out,
                                                            float* __restrict__ dstate, ScanGeo g, int64_t total) {
  for (int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x; id < total; id += int64_t(gridDim.x) * 256) {
    const Column<SL, SPL> c(id, a, g);
    join_forward(states, sums, state && c.live ? state[c.user] : 0.0f, c, g, 0);
    float r = dstate_out && c.live ? dstate_out[c.user] : 0.0f;
    for (int32_t k0 = g.chunks - 1; k0 >= 0; k0 -= kJoin) {
      float p[kJoin], e[kJoin];
#pragma unroll
      for (int i = 0; i < kJoin; ++i) {
        const bool ok = k0 - i >= 0;
        p[i] = ok ? backs[c.at + (k0 - i) * c.step] : 0.0f;
        e[i] = ok ? sums[c.sum_at + (k0 - i) * c.sum_step] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kJoin; ++i) {
        if (k0 - i < 0) break;
        backs[c.at + (k0 - i) * c.step] = r;
        r = __builtin_fmaf(__builtin_amdgcn_exp2f(c.a2 * e[i]), r, p[i]);
      }
    }
    if (dstate && c.live) dstate[c.user] = r;
  }
}

// Two elements as they were loaded, in one register where they are 16 bits.
template <int DT>
struct Two {
  uint32_t v;
  __device__ __forceinline__ void set(uint16_t a, uint16_t b) { v = uint32_t(b) << 16 | a; }
  __device__ __forceinline__ float first() const { return to_f<DT>(uint16_t(v)); }
  __device__ __forceinline__ float second() const { return to_f<DT>(uint16_t(v >> 16)); }
};
template <>
struct Two<CNHWC_F32> {
  float a, b;
  __device__ __forceinline__ void set(float x, float y) { a = x, b = y; }
  __device__ __forceinline__ float first() const { return a; }
  __device__ __forceinline__ float second() const { return b; }
};

// x's sum over both halves (or over both rows of a pair) in the lower half
// (even rows), y's in the upper half (odd rows).
__device__ __forceinline__ float halves_add(float x, float y) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y),
                                                  false, false);
  return __builtin_bit_cast(float, uint32_t(r[0])) + __builtin_bit_cast(float, uint32_t(r[1]));
}
__device__ __forceinline__ float rows_add(float x, float y) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y),
                                                  false, false);
  return __builtin_bit_cast(float, uint32_t(r[0])) + __builtin_bit_cast(float, uint32_t(r[1]));
}

// db and dc of one position summed over the wavefront's groups (the lanes of
// equal state index) into out[2][NS]: db and dc part at the halves, then two
// states at the rows, so every step adds half as many registers; the rest of
// the sum is within rows of 16 lanes.
template <int SL, int SPL>
__device__ __forceinline__ void sum_groups(const float (&db)[SPL], const float (&dc)[SPL], float* out, int s0) {
  constexpr int NS = SL * SPL;
  const int lane = threadIdx.x & 63, half = lane >> 5, row = lane >> 4 & 1;
  float v[SPL];
#pragma unroll
  for (int s = 0; s < SPL; ++s) v[s] = halves_add(db[s], dc[s]);
#pragma unroll
  for (int s = 0; s < SPL; s += 2) {
    float w = SPL > 1 ? rows_add(v[s], v[s + 1 < SPL ? s + 1 : s]) : add_row_pairs(v[s]);
    if constexpr (SL <= 8) w += dpp<kRor8>(w);
    if constexpr (SL <= 4) w += dpp<kRor4>(w);
    if ((lane & 15) < SL && s + row < SPL) out[half * NS + s0 + s + row] = w;
  }
}

// Tile after tile from the end of the chunk: the tile's states are run again
// into registers from the kept one, then the gradient comes back through them.
template <int DT, int SL, int SPL>
__global__ __launch_bounds__(256, 2) void scan_bwd_kernel(ScanIn<DT> in, ScanGeo g, const Elem<DT>* __restrict__ dy,
                                                       const float4* __restrict__ states,
                                                       const float4* __restrict__ backs, Kept kept, ScanOut<DT> out) {
  constexpr int NS = SL * SPL;
  // LDS for two workgroups per compute unit: up to 16 states it holds the lower
  // half tile's states and two sets of partial sums, up to 32 one set
  constexpr bool kSaveLow = NS <= 32;
  constexpr int kParts = NS <= 16 ? 2 : 1;
  __shared__ __attribute__((aligned(16))) float bc2[2][kTile * 2 * NS];
  __shared__ float part[kParts][kWaves][kTile][2 * NS];
  __shared__ float4 enter[kWaves][SPL][64];                // the state that enters the chunk
  __shared__ float4 low[kSaveLow ? kHalf - 1 : 1][kWaves][SPL][64];  // states 1, 2, 3 of a tile
  int64_t n;
  int32_t chunk, wave_d0;
  locate<SL, SPL>(g, g.chunks, n, chunk, wave_d0);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const Place<SL, SPL> at(wave_d0, g.d);
  const int32_t len = valid_len(in.lengths, n, g.l);
  const int32_t t_begin = chunk * g.chunk;
  const int32_t t_end = t_begin + g.chunk < g.l ? t_begin + g.chunk : g.l;
  const int32_t t_valid = t_end < len ? t_end : len;
  const int64_t c_id = n * g.chunks + chunk, ds = int64_t(g.d) * g.s;

  float a2[4][SPL], carry[4][SPL], da[4][SPL];
#pragma unroll
  for (int i = 0; i < SPL; ++i) enter[wave][i][lane] = states[lane_order<SPL>(blockIdx.x) + i * 64];
  load_states<SL, SPL>(a2, in.a, at, g);
  rates(a2);
  get_lanes<SPL>(backs, blockIdx.x, carry);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < SPL; ++i) da[j][i] = 0.0f;
  const float bias = in.delta_bias ? in.delta_bias[at.at] : 0.0f;
  const float skip = in.skip ? in.skip[at.at] : 0.0f;
  const Elem<DT>* un = in.u + n * g.us[0];
  const Elem<DT>* dn = in.delta + n * g.ds[0];
  const Elem<DT>* gn = in.gate ? in.gate + n * g.gs[0] : nullptr;
  const Elem<DT>* yn = dy + n * g.ys[0];
  const Elem<DT>* bn = in.b + n * g.bs[0];
  const Elem<DT>* cn = in.c + n * g.cs[0];
  const int64_t out_n = n * g.l * int64_t(g.d);

  StagedBC<DT, NS> st;
  float dskip = 0.0f, dbias = 0.0f;
  const int64_t rows = (int64_t(gridDim.x) / (int64_t(g.col_blocks) * g.chunks)) * g.l;  // N * L
  const int64_t col = blockIdx.x % g.col_blocks;
  const int32_t tiles = (t_end - t_begin + kTile - 1) / kTile;
  st.stage(bn, cn, g, t_begin + (tiles - 1) * kTile, t_valid);
  st.put(bc2[(tiles - 1) & 1]);
  __syncthreads();
  // One barrier to a tile: it stands behind the tile's partial sums and the next
  // tile's b and c.
  for (int32_t k = tiles - 1; k >= 0; --k) {
    const int32_t t0 = t_begin + k * kTile;
    const float* bc = bc2[k & 1];
    if (k > 0) st.stage(bn, cn, g, t0 - kTile, t_valid);
    float df[kTile], sg[kTile];
    Elem<DT> u_t[kTile];
    Two<DT> yz[kTile];  // dy and gate
    load_tile<DT>(u_t, un, g.us[1], at.at, t0, t_valid);
    {
      Elem<DT> d_t[kTile], g_t[kTile] = {}, y_t[kTile];
      load_tile<DT>(d_t, dn, g.ds[1], at.at, t0, t_valid);
      load_tile<DT>(y_t, yn, g.ys[1], at.at, t0, t_valid);
      if (gn) load_tile<DT>(g_t, gn, g.gs[1], at.at, t0, t_valid);
#pragma unroll
      for (int i = 0; i < kTile; ++i) {
        df[i] = to_f<DT>(d_t[i]) + bias;
        yz[i].set(y_t[i], g_t[i]);
        sg[i] = 1.0f;
      }
    }
    // the state that enters the tile
    float h0[4][SPL];
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
      const float4 f = enter[wave][i][lane];
      h0[0][i] = f.x, h0[1][i] = f.y, h0[2][i] = f.z, h0[3][i] = f.w;
    }
    if (k > 0 && t0 < t_valid) {
      const int64_t o = int64_t(blockIdx.x) * (g.chunk / kTile) + k;
      const float sum = kept.sum[o * 256 + threadIdx.x];
      float hk[4][SPL];
      get_lanes<SPL>(kept.h, o, hk);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < SPL; ++i)
          h0[j][i] = __builtin_fmaf(__builtin_amdgcn_exp2f(quad_lane(sum, j) * a2[j][i]), h0[j][i], hk[j][i]);
    }
    if (g.softplus) {
#pragma unroll
      for (int i = 0; i < kTile; ++i) df[i] = softplus(df[i], sg[i]);
    }
    // one position further; what a position needs of its quad and of b is made
    // again at each use (again() hides that it is the same), for the registers
    auto again = [](float v) __attribute__((always_inline)) {
      asm volatile("" : "+v"(v));
      return v;
    };
    auto advance = [&](int i, const float (&from)[4][SPL], float (&to)[4][SPL]) __attribute__((always_inline)) {
      float bf[SPL];
      const float dl = again(df[i]);
      const float dx = dl * to_f<DT>(u_t[i]);
      int s0 = at.s0;
      asm volatile("" : "+v"(s0));
      lds_states<SPL>(&bc[i * 2 * NS + s0], bf);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int s = 0; s < SPL; ++s)
          to[j][s] = __builtin_fmaf(__builtin_amdgcn_exp2f(quad_lane(dl, j) * a2[j][s]), from[j][s],
                                    quad_lane(dx, j) * bf[s]);
      settle(to);
    };
#pragma unroll
    for (int i = 0; i < kTile; ++i) df[i] = t0 + i < t_valid && at.live ? df[i] : 0.0f;
    // half a tile's states are held at a time (all eight would take 64 registers
    // more); those of the lower half wait in LDS, or are made again
    float hs[kHalf + 1][4][SPL];
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      if (i == 0) advance(0, h0, hs[0]);
      else advance(i, hs[0], hs[0]);
      if (kSaveLow && i < kHalf - 1) {
#pragma unroll
        for (int s = 0; s < SPL; ++s)
          low[i][wave][s][lane] = make_float4(hs[0][0][s], hs[0][1][s], hs[0][2][s], hs[0][3][s]);
      }
    }
#pragma unroll
    for (int i = 0; i < kHalf; ++i) advance(kHalf + i, hs[i], hs[i + 1]);
    // the gradient comes back through position i, from state `before` to `after`
    auto back = [&](int i, const float (&before)[4][SPL], const float (&after)[4][SPL]) __attribute__((always_inline)) {
      const float u = to_f<DT>(u_t[i]), yg = yz[i].first(), z = yz[i].second();
      const float sz = in.gate ? sigmoid_for<DT>(z) : 0.0f;
      const float gy = in.gate ? yg * (z * sz) : yg;  // yg * z alone can overflow where sz is 0
      float bf[SPL], cf[SPL], db[SPL], dc[SPL];
      const float dl = again(df[i]);
      const float dx = dl * u;
      int s0 = at.s0;
      asm volatile("" : "+v"(s0));
      lds_states<SPL>(&bc[i * 2 * NS + s0], bf);
      lds_states<SPL>(&bc[i * 2 * NS + NS + s0], cf);
#pragma unroll
      for (int s = 0; s < SPL; ++s) db[s] = dc[s] = 0.0f;
      float yq[4], bq[4], eq[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        yq[j] = bq[j] = eq[j] = 0.0f;
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
          const float e = __builtin_amdgcn_exp2f(quad_lane(dl, j) * a2[j][s]);
          const float gr = __builtin_fmaf(quad_lane(gy, j), cf[s], carry[j][s]);
          carry[j][s] = e * gr;  // h[t-1]'s gradient
          const float w = carry[j][s] * before[j][s];
          yq[j] = __builtin_fmaf(after[j][s], cf[s], yq[j]);
          bq[j] = __builtin_fmaf(gr, bf[s], bq[j]);
          eq[j] = __builtin_fmaf(w, a2[j][s], eq[j]);
          da[j][s] = __builtin_fmaf(quad_lane(dl, j), w, da[j][s]);
          db[s] = __builtin_fmaf(quad_lane(dx, j), gr, db[s]);
          dc[s] = __builtin_fmaf(quad_lane(gy, j), after[j][s], dc[s]);
        }
      }
      settle(carry);
      settle(da);
      settle(db);
      settle(dc);
      const float yo = own_sum<SL>(yq), bo = own_sum<SL>(bq), eo = own_sum<SL>(eq);
      const bool valid = t0 + i < t_valid && at.live;
      const float dd = valid ? (eo * kLn2 + u * bo) * sg[i] : 0.0f;
      dbias += dd;
      dskip = __builtin_fmaf(gy, u, dskip);
      if (at.first && t0 + i < t_end) {
        const int64_t o = out_n + (t0 + i) * int64_t(g.d);
        (out.u + o)[at.at] = from_f<DT>(valid ? __builtin_fmaf(df[i], bo, skip * gy) : 0.0f);
        (out.delta + o)[at.at] = from_f<DT>(dd);
        if (in.gate) {
          const float dz = yg * __builtin_fmaf(skip, u, yo) * sz * __builtin_fmaf(z, 1.0f - sz, 1.0f);
          (out.gate + o)[at.at] = from_f<DT>(valid ? dz : 0.0f);
        }
      }
      sum_groups<SL, SPL>(db, dc, part[k % kParts][wave][i], at.s0);
    };
#pragma unroll
    for (int i = kHalf - 1; i >= 0; --i) back(kHalf + i, hs[i], hs[i + 1]);
    copy(hs[0], hs[kHalf]);
    copy(h0, hs[0]);
#pragma unroll
    for (int i = 0; i < kHalf - 1; ++i) {
      if constexpr (kSaveLow) {
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
          const float4 f = low[i][wave][s][lane];
          hs[i + 1][0][s] = f.x, hs[i + 1][1][s] = f.y, hs[i + 1][2][s] = f.z, hs[i + 1][3][s] = f.w;
        }
      } else {
        advance(i, hs[i], hs[i + 1]);
      }
    }
#pragma unroll
    for (int i = kHalf - 1; i >= 0; --i) back(i, hs[i], hs[i + 1]);
    if (k > 0) st.put(bc2[(k - 1) & 1]);
    __syncthreads();
    // the workgroup's channels; with two buffers, the next tile's barrier stands
    // between these reads and the writes of the tile after it
    for (int i = threadIdx.x; i < kTile * 2 * NS; i += 256) {
      const int t = i / (2 * NS), q = i % (2 * NS), which = q / NS, s = q % NS;
      if (t0 + t >= t_valid || s >= g.s) continue;
      float v = part[k % kParts][0][t][q];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += part[k % kParts][w][t][q];
      out.bc_part[((col * rows + n * g.l + t0 + t) * 2 + which) * g.s + s] = v;
    }
    if constexpr (kParts == 1) __syncthreads();
  }
  float* pp = out.param_part + c_id * (ds + 2 * int64_t(g.d));
  store_states<SL, SPL>(da, pp, at, g);
  if (at.first) {
    pp[ds + at.d] = dskip;
    pp[ds + g.d + at.d] = dbias;
  }
}

// db, dc = the sums over the workgroups along the channels; 0 past the valid positions.
template <int DT>
__global__ __launch_bounds__(256) void scan_bwd_bc_kernel(const float* __restrict__ part,
                                                          const int32_t* __restrict__ lengths, ScanGeo g,
                                                          Elem<DT>* __restrict__ db, Elem<DT>* __restrict__ dc,
                                                          int64_t total) {
  for (int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x; id < total; id += int64_t(gridDim.x) * 256) {
    const int64_t row = id / (2 * g.s);
    const int32_t q = int32_t(id - row * 2 * g.s);
    const int64_t n = row / g.l;
    float v = 0.0f;
    if (row - n * g.l < valid_len(lengths, n, g.l)) {
#pragma unroll 4
      for (int32_t k = 0; k < g.col_blocks; ++k) v += part[k * total + id];
    }
    if (q < g.s) db[row * g.s + q] = from_f<DT>(v);
    else dc[row * g.s + q - g.s] = from_f<DT>(v);
  }
}

// ---------------------------------------------------------------- host

ScanGeo geo_of(const cnhwc_scan_desc_t& d) {
  ScanGeo g{};
  g.l = int32_t(d.l);
  g.d = int32_t(d.d);
  g.s = d.s;
  g.softplus = d.softplus;
  for (int i = 0; i < 2; ++i) {
    g.us[i] = d.u_stride[i];
    g.ds[i] = d.delta_stride[i];
    g.bs[i] = d.b_stride[i];
    g.cs[i] = d.c_stride[i];
    g.gs[i] = d.gate_stride[i];
    g.ys[i] = d.dy_stride[i];
  }
  return g;
}

template <int DT>
ScanIn<DT> inputs_of(const cnhwc_scan_inputs_t& in) {
  using E = Elem<DT>;
  return {static_cast<const E*>(in.u), static_cast<const E*>(in.delta), in.a, static_cast<const E*>(in.b),
          static_cast<const E*>(in.c), in.skip, static_cast<const E*>(in.gate), in.delta_bias, in.state, in.lengths};
}

template <int SL, int SPL>
struct Shape {
  static constexpr int sl = SL, spl = SPL;
};
// Lanes per group and states per lane for S states.
template <typename F>
auto with_shape(int32_t s, F&& f) {
  if (s <= 4) return f(Shape<4, 1>{});
  if (s <= 8) return f(Shape<4, 2>{});
  if (s <= 16) return f(Shape<4, 4>{});
  if (s <= 32) return f(Shape<8, 4>{});
  return f(Shape<16, 4>{});
}

template <int N>
using Int = std::integral_constant<int, N>;
template <typename F>
auto with_dtype(int32_t dt, F&& f) {
  if (dt == CNHWC_F32) return f(Int<CNHWC_F32>{});
  if (dt == CNHWC_F16) return f(Int<CNHWC_F16>{});
  return f(Int<CNHWC_BF16>{});
}

// Workgroups along the channels, of kWaves wavefronts each.
int32_t columns(const cnhwc_scan_desc_t& d) {
  const int64_t channels = d.s <= 16 ? 64 : (d.s <= 32 ? 32 : 16);  // per wavefront, as Place has them
  return int32_t(ceil_div(d.d, channels * kWaves));
}

// Positions per chunk of the forward pass.  Chunks cost a second run over the
// data, so there is one where 1024 wavefronts (one for each SIMD) come without
// them: 32 sequences of 512 x 2048 channels take 233 us so, 273 us in two
// chunks.  Otherwise enough of them for 4096 wavefronts (16384 x 2048 channels:
// 292 us; 2048 wavefronts 316, 8192 322 us).  With little to do the time is a
// chunk's steps, one after the other, and the join's along the chunks, so
// chunks have 16 positions at least and 32 in long sequences (2 x 984 x 311
// channels: chunks of 16 take 29 us, of 32 36; 4 x 2048 x 64: 44 and 40), and up
// to 64 positions are one chunk (2 x 40 x 128: 21 us, 31 in two).
int32_t fwd_chunk(const cnhwc_scan_desc_t& d) {
  const int64_t one = d.n * columns(d) * kWaves;
  int64_t chunk = d.l;
  if (one < 1024 && d.l > 64) {
    const int64_t least = d.l < 1536 ? 16 : 32;
    chunk = ceil_div(d.l * one, 4096);
    chunk = chunk < least ? least : chunk;
  }
  return int32_t(ceil_div(chunk, kTile) * kTile);
}

// Positions per chunk of the backward pass: enough chunks for 2048 wavefronts,
// the two that each SIMD holds, but at most 128 positions, at least 16.
// (4 x 1024 x 1024 channels, 32 states: chunks of 128 take 208 us, of 64 212, of
// 32 228 us; 8 x 2048 x 2048 channels, 16 states: 256 744 us, 128 740, 64 747.)
int32_t bwd_chunk(const cnhwc_scan_desc_t& d) {
  int64_t chunk = ceil_div(d.l * d.n * columns(d) * kWaves, 2048);
  chunk = chunk < 16 ? 16 : (chunk > 128 ? 128 : chunk);
  return int32_t(ceil_div(chunk, kTile) * kTile);
}

// States per lane.
uint64_t lane_states(int32_t s) { return s <= 4 ? 1 : (s <= 8 ? 2 : 4); }

struct FwdLayout {
  uint64_t states, sums, total;
};
FwdLayout fwd_layout(const cnhwc_scan_desc_t& d) {
  const int64_t chunks = ceil_div(d.l, fwd_chunk(d));
  const uint64_t lanes = uint64_t(d.n) * chunks * columns(d) * kWaves * 64;
  if (chunks == 1) return {0, 0, 0};
  return {0, lanes * lane_states(d.s) * 16, lanes * (lane_states(d.s) * 16 + 4)};
}

struct BwdLayout {
  uint64_t states, backs, sums, bc, params, kept_h, kept_sum, total;
};
BwdLayout bwd_layout(const cnhwc_scan_desc_t& d) {
  const uint64_t cols = columns(d), chunk = bwd_chunk(d), ds = uint64_t(d.d) * d.s;
  const uint64_t nc = uint64_t(d.n) * ceil_div(d.l, chunk), lanes = nc * cols * kWaves * 64;
  BwdLayout L;
  uint64_t at = 0;
  auto take = [&](uint64_t floats) {
    const uint64_t o = at;
    at = align_up(at + floats * 4, 256);
    return o;
  };
  L.states = take(lanes * lane_states(d.s) * 4);
  L.backs = take(lanes * lane_states(d.s) * 4);
  L.sums = take(lanes);
  L.bc = take(cols * d.n * d.l * 2 * d.s);
  L.params = take(nc * (ds + 2 * uint64_t(d.d)));
  L.kept_h = take(lanes * (chunk / kTile) * lane_states(d.s) * 4);
  L.kept_sum = take(lanes * (chunk / kTile));
  L.total = at;
  return L;
}

cnhwc_status_t check_desc(const cnhwc_scan_desc_t* d, bool bwd) {
  if (!d || !dtype_ok(d->dtype) || d->reserved != 0 || (d->softplus != 0 && d->softplus != 1))
    return CNHWC_ERR_INVALID_ARGUMENT;
  if (!extent_ok(d->n) || !extent_ok(d->l) || !extent_ok(d->d) || d->s < 1) return CNHWC_ERR_INVALID_ARGUMENT;
  if (!strides_ok(d->n, d->l, d->d, d->u_stride) || !strides_ok(d->n, d->l, d->d, d->delta_stride) ||
      !strides_ok(d->n, d->l, d->s, d->b_stride) || !strides_ok(d->n, d->l, d->s, d->c_stride) ||
      !strides_ok(d->n, d->l, d->d, d->gate_stride) || (bwd && !strides_ok(d->n, d->l, d->d, d->dy_stride)))
    return CNHWC_ERR_INVALID_ARGUMENT;
  if (d->s > CNHWC_SCAN_MAX_STATE) return CNHWC_ERR_UNSUPPORTED;
  // positions fit 32 bits with a chunk's overhang; 64-bit offsets; the grids of
  // the backward pass (chunks of 128 positions at these sizes) and of its sums
  if (d->l > INT_MAX - 1024 || d->d > (1ll << 23) || d->d * (d->s + 2) > (1ll << 27) ||
      !dense_ok(d->n, d->l, d->d * d->s) ||
      d->n * ceil_div(d->l, 128) * ceil_div(d->d, 64) > (1ll << 23))
    return CNHWC_ERR_UNSUPPORTED;
  return CNHWC_OK;
}

void add_inputs(Buffers& bf, const cnhwc_scan_desc_t& d, const cnhwc_scan_inputs_t& in, bool state) {
  const uint64_t es = dtype_size(d.dtype);
  bf.in(in.u, span(d.n, d.l, d.d, d.u_stride) * es, es, true);
  bf.in(in.delta, span(d.n, d.l, d.d, d.delta_stride) * es, es, true);
  bf.in(in.a, uint64_t(d.d) * d.s * 4, 4, true);
  bf.in(in.b, span(d.n, d.l, d.s, d.b_stride) * es, es, true);
  bf.in(in.c, span(d.n, d.l, d.s, d.c_stride) * es, es, true);
  bf.in(in.skip, d.d * 4, 4, false);
  bf.in(in.gate, span(d.n, d.l, d.d, d.gate_stride) * es, es, false);
  bf.in(in.delta_bias, d.d * 4, 4, false);
  if (state) bf.in(in.state, uint64_t(d.n) * d.d * d.s * 4, 4, false);
  bf.in(in.lengths, d.n * 4, 4, false);
}

}  // namespace
}  // namespace seq
}  // namespace cnhwc

using namespace cnhwc;
using namespace cnhwc::seq;

extern "C" cnhwc_status_t cnhwc_scan_fwd_workspace(const cnhwc_scan_desc_t* desc, uint64_t* bytes) {
  const cnhwc_status_t st = check_desc(desc, false);
  if (st != CNHWC_OK) return st;
  if (!bytes) return CNHWC_ERR_INVALID_ARGUMENT;
  *bytes = fwd_layout(*desc).total;
  return CNHWC_OK;
}

extern "C" cnhwc_status_t cnhwc_scan_fwd(const cnhwc_scan_desc_t* desc, const cnhwc_scan_inputs_t* in, void* y,
                                         float* state_out, void* workspace, uint64_t workspace_bytes,
                                         void* hip_stream) {
  const cnhwc_status_t st = check_desc(desc, false);
  if (st != CNHWC_OK) return st;
  if (!in) return CNHWC_ERR_INVALID_ARGUMENT;
  const cnhwc_scan_desc_t& d = *desc;
  const FwdLayout L = fwd_layout(d);
  const uint64_t need = L.total;
  if (workspace_bytes < need) return CNHWC_ERR_WORKSPACE_TOO_SMALL;
  const uint64_t es = dtype_size(d.dtype);
  Buffers bf;
  add_inputs(bf, d, *in, true);
  bf.out(y, uint64_t(d.n) * d.l * d.d * es, es, true);
  bf.out(state_out, uint64_t(d.n) * d.d * d.s * 4, 4, false);
  if (need) bf.out(workspace, need, 16, true);
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  ScanGeo g = geo_of(d);
  g.col_blocks = columns(d);
  g.chunk = fwd_chunk(d);
  g.chunks = int32_t(ceil_div(d.l, g.chunk));
  const dim3 grid(unsigned(d.n * g.chunks * g.col_blocks)), block(256);
  float* states = static_cast<float*>(workspace);
  float4* states4 = static_cast<float4*>(workspace);
  float* sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.sums);
  return with_dtype(d.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    const ScanIn<DT> si = inputs_of<DT>(*in);
    Elem<DT>* yo = static_cast<Elem<DT>*>(y);
    return with_shape(d.s, [&](auto sh) {
      constexpr int SL = decltype(sh)::sl, SPL = decltype(sh)::spl;
      if (g.chunks > 1) {
        const dim3 all_but_last(unsigned(d.n * (g.chunks - 1) * g.col_blocks));
        hipLaunchKernelGGL((scan_fwd_kernel<DT, SL, SPL, true>), all_but_last, block, 0, s, si, g, yo, states4, sums,
                           nullptr);
        const int64_t total = d.n * g.col_blocks * (kWaves * 64 * 4 * SPL);
        hipLaunchKernelGGL((scan_join_kernel<SL, SPL>), grid_of(ceil_div(total, 256)), dim3(256), 0, s, states, sums,
                           in->a, in->state, g, total);
      }
      hipLaunchKernelGGL((scan_fwd_kernel<DT, SL, SPL, false>), grid, block, 0, s, si, g, yo, states4, sums, state_out);
      return hipGetLastError() == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
    });
  });
}

extern "C" cnhwc_status_t cnhwc_scan_bwd_workspace(const cnhwc_scan_desc_t* desc, uint64_t* bytes) {
  const cnhwc_status_t st = check_desc(desc, true);
  if (st != CNHWC_OK) return st;
  if (!bytes) return CNHWC_ERR_INVALID_ARGUMENT;
  *bytes = bwd_layout(*desc).total;
  return CNHWC_OK;
}

extern "C" cnhwc_status_t cnhwc_scan_bwd(const cnhwc_scan_desc_t* desc, const cnhwc_scan_inputs_t* in,
                                         const void* dy, const float* dstate_out, const cnhwc_scan_grads_t* grads,
                                         void* workspace, uint64_t workspace_bytes, void* hip_stream) {
  const cnhwc_status_t st = check_desc(desc, true);
  if (st != CNHWC_OK) return st;
  if (!in || !grads) return CNHWC_ERR_INVALID_ARGUMENT;
  const cnhwc_scan_desc_t& d = *desc;
  if ((in->skip == nullptr) != (grads->skip == nullptr) || (in->gate == nullptr) != (grads->gate == nullptr) ||
      (in->delta_bias == nullptr) != (grads->delta_bias == nullptr))
    return CNHWC_ERR_INVALID_ARGUMENT;
  const BwdLayout L = bwd_layout(d);
  if (workspace_bytes < L.total) return CNHWC_ERR_WORKSPACE_TOO_SMALL;
  const uint64_t es = dtype_size(d.dtype), act = uint64_t(d.n) * d.l * d.d * es, nls = uint64_t(d.n) * d.l * d.s * es;
  const uint64_t state_bytes = uint64_t(d.n) * d.d * d.s * 4;
  Buffers bf;
  add_inputs(bf, d, *in, true);
  bf.in(dy, span(d.n, d.l, d.d, d.dy_stride) * es, es, true);
  bf.in(dstate_out, state_bytes, 4, false);
  bf.out(grads->u, act, es, true);
  bf.out(grads->delta, act, es, true);
  bf.out(grads->a, uint64_t(d.d) * d.s * 4, 4, true);
  bf.out(grads->b, nls, es, true);
  bf.out(grads->c, nls, es, true);
  bf.out(grads->skip, d.d * 4, 4, false);
  bf.out(grads->gate, act, es, false);
  bf.out(grads->delta_bias, d.d * 4, 4, false);
  bf.out(grads->state, state_bytes, 4, false);
  bf.out(workspace, L.total, 16, true);
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  ScanGeo g = geo_of(d);
  g.col_blocks = columns(d);
  g.chunk = bwd_chunk(d);
  g.chunks = int32_t(ceil_div(d.l, g.chunk));
  const dim3 grid(unsigned(d.n * g.chunks * g.col_blocks)), block(256);
  char* ws = static_cast<char*>(workspace);
  float* states = reinterpret_cast<float*>(ws + L.states);
  float* backs = reinterpret_cast<float*>(ws + L.backs);
  float* sums = reinterpret_cast<float*>(ws + L.sums);
  float* bc = reinterpret_cast<float*>(ws + L.bc);
  float* params = reinterpret_cast<float*>(ws + L.params);
  const Kept kept{reinterpret_cast<float4*>(ws + L.kept_h), reinterpret_cast<float*>(ws + L.kept_sum)};
  return with_dtype(d.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    using E = Elem<DT>;
    const ScanIn<DT> si = inputs_of<DT>(*in);
    const E* gy = static_cast<const E*>(dy);
    const ScanOut<DT> so{static_cast<E*>(grads->u), static_cast<E*>(grads->delta), static_cast<E*>(grads->gate), bc,
                         params};
    with_shape(d.s, [&](auto sh) {
      constexpr int SL = decltype(sh)::sl, SPL = decltype(sh)::spl;
      float4 *states4 = reinterpret_cast<float4*>(states), *backs4 = reinterpret_cast<float4*>(backs);
      hipLaunchKernelGGL((scan_bwd_local_kernel<DT, SL, SPL>), grid, block, 0, s, si, g, gy, states4, backs4, sums,
                         kept);
      const int64_t total = d.n * g.col_blocks * (kWaves * 64 * 4 * SPL);
      hipLaunchKernelGGL((scan_bwd_join_kernel<SL, SPL>), grid_of(ceil_div(total, 256)), dim3(256), 0, s, states,
                         backs, sums, in->a, in->state, dstate_out, grads->state, g, total);
      hipLaunchKernelGGL((scan_bwd_kernel<DT, SL, SPL>), grid, block, 0, s, si, g, gy, states4, backs4, kept, so);
    });
    const int64_t bc_total = d.n * d.l * 2 * d.s;
    hipLaunchKernelGGL((scan_bwd_bc_kernel<DT>), grid_of(ceil_div(bc_total, 256)), dim3(256), 0, s, bc, in->lengths,
                       g, static_cast<E*>(grads->b), static_cast<E*>(grads->c), bc_total);
    sum_parts<CNHWC_F32>(params, d.n * g.chunks,
                         SumOut{{grads->a, grads->skip, grads->delta_bias}, {d.d * d.s, d.d, d.d}}, true, s);
    return hipGetLastError() == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
  });
}

extern "C" cnhwc_status_t cnhwc_scan_step(const cnhwc_scan_desc_t* desc, const cnhwc_scan_inputs_t* in, void* y,
                                          float* state_out, void* hip_stream) {
  const cnhwc_status_t st = check_desc(desc, false);
  if (st != CNHWC_OK) return st;
  if (!in || desc->l != 1 || !in->state || in->lengths) return CNHWC_ERR_INVALID_ARGUMENT;
  const cnhwc_scan_desc_t& d = *desc;
  const uint64_t es = dtype_size(d.dtype);
  Buffers bf;
  add_inputs(bf, d, *in, in->state != state_out);
  bf.out(y, uint64_t(d.n) * d.d * es, es, true);
  bf.out(state_out, uint64_t(d.n) * d.d * d.s * 4, 4, true);
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  const ScanGeo g = geo_of(d);
  // whole vectors of four states, and of four elements of b and c
  const uint64_t quad = 4 * es;
  const bool whole = (d.s == 16 || d.s == 32 || d.s == 64) && aligned(in->state, 16) && aligned(state_out, 16) &&
                     aligned(in->a, 16) && aligned(in->b, quad) && aligned(in->c, quad) &&
                     (d.n == 1 || (d.b_stride[0] % 4 == 0 && d.c_stride[0] % 4 == 0));
  return with_dtype(d.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    const ScanIn<DT> si = inputs_of<DT>(*in);
    return with_shape(d.s, [&](auto sh) {
      constexpr int SL = decltype(sh)::sl, SPL = decltype(sh)::spl;
      const int64_t cols = ceil_div(d.d, 256 / SL);
      auto go = [&](auto nb, auto wh) {
        constexpr int NB = decltype(nb)::value;
        const int64_t rows = ceil_div(d.n, NB);
        hipLaunchKernelGGL((scan_step_kernel<DT, SL, SPL, NB, decltype(wh)::value>),
                           dim3(unsigned(cols), unsigned(rows < 65535 ? rows : 65535)), dim3(256), 0, s, si, g,
                           static_cast<Elem<DT>*>(y), state_out, d.n);
      };
      // two sequences to a thread once there are more workgroups than the device
      // holds at a time (256 x 4096 channels, 16 states: one 31.3 us, two 28.7,
      // four 31.5)
      const bool many = cols * d.n > 2048;
      if constexpr (SPL == 4) {
        if (whole) {
          if (many) go(Int<2>{}, std::true_type{});
          else go(Int<1>{}, std::true_type{});
          return hipGetLastError() == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
        }
      }
      if (many) go(Int<2>{}, std::false_type{});
      else go(Int<1>{}, std::false_type{});
      return hipGetLastError() == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
    });
  });
}
