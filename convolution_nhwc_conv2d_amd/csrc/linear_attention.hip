// Linear attention with a decay for each head, forward, backward and single
// tokens, for gfx950.
//
//   S[t] = exp(g) S[t-1] + k[t]^T v[t],   y[t] = scale q[t] S[t]
//
// The gradients have the same form, with the tensors in other places and, for k
// and v, the positions from the end (G the state's gradient):
//   dq = attention(dy, v, k),  dk = attention_back(v, dy, q),  dv = attention_back(k, q, dy)
// where the backward ones meet G before a position's decay: G[t] = exp(g) G[t+1] ...
#include <hip/hip_runtime.h>

#include <cfloat>
#include <type_traits>

#include "internal.hpp"
#include "seq_common.hpp"
#include "seq_host.hpp"

namespace cnhwc {
namespace seq {
namespace {

// One pass: y = scale q S with S from k and v.  The backward pass puts other
// tensors into these places.
template <int DT>
struct Pass {
  const Elem<DT>* q;
  const Elem<DT>* k;
  const Elem<DT>* v;
  Elem<DT>* y;             // dense [N,L,H,DV]
  const float* state;      // element (i, j) of [DK,DV] at i * state_k + j * state_v
  float* state_out;
  int64_t qs[3], ks[3], vs[3];  // element strides: sequence, position, head
  int64_t state_k, state_v;
  int32_t dk, dv;
  bool back;               // positions from the end, the state decays after its use
  float scale_k, scale_y;  // of what enters the state, of what leaves it
};

struct LaGeo {
  int32_t l, h;
  const float* log_decay;
  const int32_t* lengths;
};

// log_decay, finite for minus infinity too (0 times it is 0).
__device__ __forceinline__ float rate(float g) { return g < -FLT_MAX ? -FLT_MAX : g; }

// x -> exp(g) x without losing what a slow decay is about: exp(g) - 1 keeps its
// digits where exp(g), rounded, would be off by 2^-25 at every position, 10^-4
// after 4096 of them.
struct Decay {
  float m;     // exp(g) - 1, or exp(g)
  float keep;  // 1, or 0
  __device__ __forceinline__ explicit Decay(float g) {
    const bool slow = __builtin_fabsf(g) < 0.5f;
    m = slow ? expm1f(g) : exp_full(g);
    keep = slow ? 1.0f : 0.0f;
  }
  __device__ __forceinline__ float operator()(float x) const { return __builtin_fmaf(m, x, keep * x); }
};

// ---------------------------------------------------------------- position by position

// A workgroup holds 64 columns of one head's state: 16 lanes by four columns, 16
// row groups, rows r, r + 16, ... of NI.
template <int DT, int NI>
__global__ __launch_bounds__(256) void la_step_kernel(Pass<DT> p, LaGeo g) {
  __shared__ float part[2][4][64];
  const int64_t nh = blockIdx.x;
  const int64_t n = nh / g.h, hd = nh - n * g.h;
  const int j0 = int(blockIdx.y) * 64 + int(threadIdx.x & 15) * 4, r0 = threadIdx.x >> 4;
  const int64_t base = nh * p.dk * p.dv;
  float s[NI][4];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = r0 + 16 * i, j = j0 + e;
      s[i][e] = p.state && r < p.dk && j < p.dv ? p.state[base + r * p.state_k + j * p.state_v] : 0.0f;
    }
  const Decay decay(rate(g.log_decay[hd]));
  const int32_t len = valid_len(g.lengths, n, g.l);
  const Elem<DT>* qn = p.q + n * p.qs[0] + hd * p.qs[2];
  const Elem<DT>* kn = p.k + n * p.ks[0] + hd * p.ks[2];
  const Elem<DT>* vn = p.v + n * p.vs[0] + hd * p.vs[2];
  for (int32_t i = 0; i < g.l; ++i) {
    const int32_t t = p.back ? g.l - 1 - i : i;
    Elem<DT>* y = p.y + ((n * g.l + t) * g.h + hd) * p.dv;
    if (t >= len) {  // uniform over the workgroup
      if (threadIdx.x < 64 && blockIdx.y * 64 + threadIdx.x < p.dv) y[blockIdx.y * 64 + threadIdx.x] = Elem<DT>(0);
      continue;
    }
    float v[4], acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = j0 + e < p.dv ? to_f<DT>(vn[t * p.vs[1] + j0 + e]) : 0.0f;
#pragma unroll
    for (int a = 0; a < NI; ++a) {
      const int r = r0 + 16 * a;
      const float k = r < p.dk ? to_f<DT>(kn[t * p.ks[1] + r]) * p.scale_k : 0.0f;
      const float q = r < p.dk ? to_f<DT>(qn[t * p.qs[1] + r]) : 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[a][e] = __builtin_fmaf(k, v[e], p.back ? s[a][e] : decay(s[a][e]));
        acc[e] = __builtin_fmaf(q, s[a][e], acc[e]);
        if (p.back) s[a][e] = decay(s[a][e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc[e] = add_halves(add_row_pairs(acc[e]));
      if ((threadIdx.x & 48) == 0) part[i & 1][threadIdx.x >> 6][(threadIdx.x & 15) * 4 + e] = acc[e];
    }
    __syncthreads();
    if (threadIdx.x < 64) {
      const int j = int(blockIdx.y) * 64 + threadIdx.x;
      const float (&w)[4][64] = part[i & 1];
      const float sum = (w[0][threadIdx.x] + w[1][threadIdx.x]) + (w[2][threadIdx.x] + w[3][threadIdx.x]);
      if (j < p.dv) y[j] = from_f<DT>(sum * p.scale_y);
    }
  }
  if (!p.state_out) return;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = r0 + 16 * i, j = j0 + e;
      if (r < p.dk && j < p.dv) p.state_out[base + r * p.state_k + j * p.state_v] = s[i][e];
    }
}

// The gradient of log_decay: with T[t] = exp(g) (T[t-1] + S[t-1]), the state's
// derivative, sum_t scale dy[t] q[t] T[t] + dstate T[L].  part: one sum for each workgroup.
template <int DT, int NI>
__global__ __launch_bounds__(256) void la_decay_grad_kernel(Pass<DT> p, const Elem<DT>* dy, int64_t ds0, int64_t ds1,
                                                            int64_t ds2, const float* dstate_out, LaGeo g,
                                                            float* part) {
  __shared__ float sum[4];
  const int64_t nh = blockIdx.x;
  const int64_t n = nh / g.h, hd = nh - n * g.h;
  const int j0 = int(blockIdx.y) * 64 + int(threadIdx.x & 15) * 4, r0 = threadIdx.x >> 4;
  const int64_t base = nh * p.dk * p.dv;
  float s[NI][4], grow[NI][4];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = r0 + 16 * i, j = j0 + e;
      s[i][e] = p.state && r < p.dk && j < p.dv ? p.state[base + r * p.state_k + j * p.state_v] : 0.0f;
      grow[i][e] = 0.0f;
    }
  const Decay decay(rate(g.log_decay[hd]));
  const int32_t len = valid_len(g.lengths, n, g.l);
  double total = 0.0;
  for (int32_t t = 0; t < len; ++t) {
    float acc = 0.0f;
#pragma unroll
    for (int a = 0; a < NI; ++a) {
      const int r = r0 + 16 * a;
      const float k = r < p.dk ? to_f<DT>(p.k[n * p.ks[0] + t * p.ks[1] + hd * p.ks[2] + r]) : 0.0f;
      const float q = r < p.dk ? to_f<DT>(p.q[n * p.qs[0] + t * p.qs[1] + hd * p.qs[2] + r]) : 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = j0 + e;
        const float v = j < p.dv ? to_f<DT>(p.v[n * p.vs[0] + t * p.vs[1] + hd * p.vs[2] + j]) : 0.0f;
        const float d = j < p.dv ? to_f<DT>(dy[n * ds0 + t * ds1 + hd * ds2 + j]) : 0.0f;
        grow[a][e] = decay(grow[a][e] + s[a][e]);
        s[a][e] = __builtin_fmaf(k, v, decay(s[a][e]));
        acc = __builtin_fmaf(q * d, grow[a][e], acc);
      }
    }
    total += double(acc);
  }
  total *= p.scale_y;
  if (dstate_out) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 16 * i, j = j0 + e;
        if (r < p.dk && j < p.dv) total += double(dstate_out[base + int64_t(r) * p.dv + j] * grow[i][e]);
      }
  }
  const float one = group_sum<64>(float(total));
  if ((threadIdx.x & 63) == 0) sum[threadIdx.x >> 6] = one;
  __syncthreads();
  if (threadIdx.x == 0) part[nh * gridDim.y + blockIdx.y] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

__global__ __launch_bounds__(256) void la_decay_sum_kernel(const float* __restrict__ part, float* __restrict__ out,
                                                           int64_t seqs, int32_t heads, int32_t blocks) {
  const int64_t h = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (h >= heads) return;
  double v = 0.0;
  for (int64_t n = 0; n < seqs; ++n)
    for (int32_t b = 0; b < blocks; ++b) v += double(part[(n * heads + h) * blocks + b]);
  out[h] = float(v);
}

// ---------------------------------------------------------------- host

using Desc = cnhwc_linear_attention_desc_t;

template <typename F>
void with_rows(int32_t dk, F&& f) {  // rows of 16 that a thread holds one of
  if (dk <= 32) f(std::integral_constant<int, 2>{});
  else if (dk <= 64) f(std::integral_constant<int, 4>{});
  else if (dk <= 128) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

template <int DT>
void launch_steps(const Pass<DT>& p, const LaGeo& g, int64_t nh, hipStream_t st) {
  with_rows(p.dk, [&](auto ni) {
    hipLaunchKernelGGL((la_step_kernel<DT, decltype(ni)::value>), dim3(unsigned(nh), unsigned((p.dv + 63) / 64)),
                       dim3(256), 0, st, p, g);
  });
}

template <int DT>
Pass<DT> pass_of(const void* q, const int64_t (&qs)[3], const void* k, const int64_t (&ks)[3], const void* v,
                 const int64_t (&vs)[3], void* y, int32_t dk, int32_t dv, float scale, bool back) {
  using E = Elem<DT>;
  Pass<DT> p{};
  p.q = static_cast<const E*>(q), p.k = static_cast<const E*>(k), p.v = static_cast<const E*>(v);
  p.y = static_cast<E*>(y);
  for (int i = 0; i < 3; ++i) p.qs[i] = qs[i], p.ks[i] = ks[i], p.vs[i] = vs[i];
  p.dk = dk, p.dv = dv, p.back = back;
  p.scale_k = back ? scale : 1.0f, p.scale_y = back ? 1.0f : scale;
  p.state_k = dv, p.state_v = 1;
  return p;
}

bool strides3_ok(const Desc& d, int64_t c, const int64_t (&s)[3]) {
  constexpr int64_t kMax = 1ll << 60;
  const int64_t ext[3] = {d.n, d.l, d.h};
  int64_t end = c;
  for (int i = 0; i < 3; ++i) {
    if (ext[i] == 1) continue;
    if (s[i] < 0 || s[i] > kMax / ext[i]) return false;
    end += (ext[i] - 1) * s[i];
  }
  return end <= kMax;
}

uint64_t span3(const Desc& d, int64_t c, const int64_t (&s)[3]) {
  return uint64_t((d.n > 1 ? (d.n - 1) * s[0] : 0) + (d.l > 1 ? (d.l - 1) * s[1] : 0) +
                  (d.h > 1 ? (d.h - 1) * s[2] : 0) + c);
}

cnhwc_status_t check_desc(const Desc* d, bool bwd) {
  if (!d || !dtype_ok(d->dtype) || d->reserved != 0 || d->reserved2 != 0) return CNHWC_ERR_INVALID_ARGUMENT;
  if (!extent_ok(d->n) || !extent_ok(d->l) || !extent_ok(d->h) || d->dk < 1 || d->dv < 1)
    return CNHWC_ERR_INVALID_ARGUMENT;
  if (!strides3_ok(*d, d->dk, d->q_stride) || !strides3_ok(*d, d->dk, d->k_stride) ||
      !strides3_ok(*d, d->dv, d->v_stride) || (bwd && !strides3_ok(*d, d->dv, d->dy_stride)))
    return CNHWC_ERR_INVALID_ARGUMENT;
  if (d->dk > CNHWC_LINEAR_ATTENTION_MAX_DIM || d->dv > CNHWC_LINEAR_ATTENTION_MAX_DIM) return CNHWC_ERR_UNSUPPORTED;
  // the grid's first dimension, and 64-bit offsets
  if (d->n * d->h > (1ll << 23) || d->l > (1ll << 30) || !dense_ok(d->n * d->h, d->l, d->dk > d->dv ? d->dk : d->dv))
    return CNHWC_ERR_UNSUPPORTED;
  return CNHWC_OK;
}

bool inputs_ok(const Desc& d, const cnhwc_linear_attention_inputs_t* in, Buffers& bf, bool state_is_out) {
  if (!in) return false;
  const uint64_t es = dtype_size(d.dtype);
  bf.in(in->q, span3(d, d.dk, d.q_stride) * es, es, true);
  bf.in(in->k, span3(d, d.dk, d.k_stride) * es, es, true);
  bf.in(in->v, span3(d, d.dv, d.v_stride) * es, es, true);
  bf.in(in->log_decay, uint64_t(d.h) * 4, 4, true);
  if (!state_is_out) bf.in(in->state, uint64_t(d.n) * d.h * d.dk * d.dv * 4, 16, false);
  bf.in(in->lengths, uint64_t(d.n) * 4, 4, false);
  return true;
}

LaGeo geo_of(const Desc& d, const cnhwc_linear_attention_inputs_t& in) {
  return {int32_t(d.l), int32_t(d.h), in.log_decay, in.lengths};
}

template <int DT>
hipError_t forward_t(const Desc& d, const cnhwc_linear_attention_inputs_t& in, void* y, float* state_out,
                     hipStream_t st) {
  Pass<DT> p = pass_of<DT>(in.q, d.q_stride, in.k, d.k_stride, in.v, d.v_stride, y, d.dk, d.dv, d.scale, false);
  p.state = in.state, p.state_out = state_out;
  launch_steps(p, geo_of(d, in), d.n * d.h, st);
  return hipGetLastError();
}

template <int DT>
hipError_t backward_t(const Desc& d, const cnhwc_linear_attention_inputs_t& in, const void* dy,
                      const float* dstate_out, const cnhwc_linear_attention_grads_t& gr, float* part,
                      hipStream_t st) {
  const LaGeo g = geo_of(d, in);
  const int64_t nh = d.n * d.h;
  Pass<DT> q = pass_of<DT>(dy, d.dy_stride, in.v, d.v_stride, in.k, d.k_stride, gr.q, d.dv, d.dk, d.scale, false);
  q.state = in.state, q.state_k = 1, q.state_v = d.dv;  // S^T
  launch_steps(q, g, nh, st);
  Pass<DT> v = pass_of<DT>(in.k, d.k_stride, in.q, d.q_stride, dy, d.dy_stride, gr.v, d.dk, d.dv, d.scale, true);
  v.state = dstate_out, v.state_out = gr.state;
  launch_steps(v, g, nh, st);
  Pass<DT> k = pass_of<DT>(in.v, d.v_stride, dy, d.dy_stride, in.q, d.q_stride, gr.k, d.dv, d.dk, d.scale, true);
  k.state = dstate_out, k.state_k = 1, k.state_v = d.dv;
  launch_steps(k, g, nh, st);
  if (gr.log_decay) {
    Pass<DT> s = pass_of<DT>(in.q, d.q_stride, in.k, d.k_stride, in.v, d.v_stride, nullptr, d.dk, d.dv, d.scale, false);
    s.state = in.state;
    const unsigned blocks = unsigned((d.dv + 63) / 64);
    with_rows(d.dk, [&](auto ni) {
      hipLaunchKernelGGL((la_decay_grad_kernel<DT, decltype(ni)::value>), dim3(unsigned(nh), blocks), dim3(256), 0, st,
                         s, static_cast<const Elem<DT>*>(dy), d.dy_stride[0], d.dy_stride[1], d.dy_stride[2],
                         dstate_out, g, part);
    });
    hipLaunchKernelGGL(la_decay_sum_kernel, dim3(unsigned((d.h + 255) / 256)), dim3(256), 0, st, part, gr.log_decay,
                       d.n, int32_t(d.h), int32_t(blocks));
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace seq
}  // namespace cnhwc

using namespace cnhwc;
using namespace cnhwc::seq;

extern "C" cnhwc_status_t cnhwc_linear_attention_fwd_workspace(const Desc* desc, uint64_t* bytes) {
  const cnhwc_status_t st = check_desc(desc, false);
  if (st != CNHWC_OK) return st;
  if (!bytes) return CNHWC_ERR_INVALID_ARGUMENT;
  *bytes = 0;
  return CNHWC_OK;
}

extern "C" cnhwc_status_t cnhwc_linear_attention_fwd(const Desc* desc, const cnhwc_linear_attention_inputs_t* in,
                                                     void* y, float* state_out, void* workspace,
                                                     uint64_t workspace_bytes, void* hip_stream) {
  uint64_t need = 0;
  const cnhwc_status_t st = cnhwc_linear_attention_fwd_workspace(desc, &need);
  if (st != CNHWC_OK) return st;
  const Desc& d = *desc;
  const uint64_t es = dtype_size(d.dtype);
  Buffers bf;
  if (!inputs_ok(d, in, bf, false)) return CNHWC_ERR_INVALID_ARGUMENT;
  bf.out(y, uint64_t(d.n) * d.l * d.h * d.dv * es, es, true);
  bf.out(state_out, uint64_t(d.n) * d.h * d.dk * d.dv * 4, 16, false);
  if (need) {
    if (workspace_bytes < need) return CNHWC_ERR_WORKSPACE_TOO_SMALL;
    bf.out(workspace, need, 16, true);
  }
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  const hipError_t e = d.dtype == CNHWC_F32   ? forward_t<CNHWC_F32>(d, *in, y, state_out, s)
                       : d.dtype == CNHWC_F16 ? forward_t<CNHWC_F16>(d, *in, y, state_out, s)
                                              : forward_t<CNHWC_BF16>(d, *in, y, state_out, s);
  return e == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
}

extern "C" cnhwc_status_t cnhwc_linear_attention_bwd_workspace(const Desc* desc, int32_t decay_grad,
                                                               uint64_t* bytes) {
  const cnhwc_status_t st = check_desc(desc, true);
  if (st != CNHWC_OK) return st;
  if (!bytes) return CNHWC_ERR_INVALID_ARGUMENT;
  *bytes = decay_grad ? uint64_t(desc->n) * desc->h * ((desc->dv + 63) / 64) * 4 : 0;
  return CNHWC_OK;
}

extern "C" cnhwc_status_t cnhwc_linear_attention_bwd(const Desc* desc, const cnhwc_linear_attention_inputs_t* in,
                                                     const void* dy, const float* dstate_out,
                                                     const cnhwc_linear_attention_grads_t* grads, void* workspace,
                                                     uint64_t workspace_bytes, void* hip_stream) {
  if (!grads) return CNHWC_ERR_INVALID_ARGUMENT;
  uint64_t need = 0;
  const cnhwc_status_t st = cnhwc_linear_attention_bwd_workspace(desc, grads->log_decay != nullptr, &need);
  if (st != CNHWC_OK) return st;
  const Desc& d = *desc;
  const uint64_t es = dtype_size(d.dtype), rows = uint64_t(d.n) * d.l * d.h;
  const uint64_t state = uint64_t(d.n) * d.h * d.dk * d.dv * 4;
  Buffers bf;
  if (!inputs_ok(d, in, bf, false)) return CNHWC_ERR_INVALID_ARGUMENT;
  bf.in(dy, span3(d, d.dv, d.dy_stride) * es, es, true);
  bf.in(dstate_out, state, 16, false);
  bf.out(grads->q, rows * d.dk * es, es, true);
  bf.out(grads->k, rows * d.dk * es, es, true);
  bf.out(grads->v, rows * d.dv * es, es, true);
  bf.out(grads->log_decay, uint64_t(d.h) * 4, 4, false);
  bf.out(grads->state, state, 16, false);
  if (need) {
    if (workspace_bytes < need) return CNHWC_ERR_WORKSPACE_TOO_SMALL;
    bf.out(workspace, need, 16, true);
  }
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  float* part = static_cast<float*>(workspace);
  const hipError_t e = d.dtype == CNHWC_F32   ? backward_t<CNHWC_F32>(d, *in, dy, dstate_out, *grads, part, s)
                       : d.dtype == CNHWC_F16 ? backward_t<CNHWC_F16>(d, *in, dy, dstate_out, *grads, part, s)
                                              : backward_t<CNHWC_BF16>(d, *in, dy, dstate_out, *grads, part, s);
  return e == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
}

extern "C" cnhwc_status_t cnhwc_linear_attention_step(const Desc* desc, const cnhwc_linear_attention_inputs_t* in,
                                                      void* y, float* state_out, void* hip_stream) {
  const cnhwc_status_t st = check_desc(desc, false);
  if (st != CNHWC_OK) return st;
  const Desc& d = *desc;
  if (d.l != 1 || !in || !in->state || in->lengths) return CNHWC_ERR_INVALID_ARGUMENT;
  const uint64_t es = dtype_size(d.dtype);
  Buffers bf;
  if (!inputs_ok(d, in, bf, state_out == in->state)) return CNHWC_ERR_INVALID_ARGUMENT;
  bf.out(y, uint64_t(d.n) * d.h * d.dv * es, es, true);
  bf.out(state_out, uint64_t(d.n) * d.h * d.dk * d.dv * 4, 16, true);
  if (!bf.ok()) return CNHWC_ERR_INVALID_ARGUMENT;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  const hipError_t e = d.dtype == CNHWC_F32   ? forward_t<CNHWC_F32>(d, *in, y, state_out, s)
                       : d.dtype == CNHWC_F16 ? forward_t<CNHWC_F16>(d, *in, y, state_out, s)
                                              : forward_t<CNHWC_BF16>(d, *in, y, state_out, s);
  return e == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
}
