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

#include "internal.hpp"
#include "linear_attention_host.hpp"
#include "seq_common.hpp"
#include "seq_host.hpp"

namespace cnhwc {
namespace seq {
namespace {

// ---------------------------------------------------------------- position by position

// A token of every sequence: a workgroup holds 64 columns of one head's state, 16 lanes by
// four columns, 16 row groups of NI consecutive rows.  The state is the traffic, read
// once and written once: VEC with whole vectors of it, and of q and k, whose elements
// one by one are as many loads as the state's vectors (64 x 16 x 128 x 128 bf16: single elements of
// all 51 us, whole vectors of the state 33, of q and k too 29, 4.6 TB/s: memory).  That is for DK
// of 32, 64, 128 and 256; any other goes by single elements: 80 x 80 25 us for 10.5 at 5 TB/s, 96 x 96 29
// for 15, 192 x 192 133 for 60.
template <int DT, int NI, bool VEC>
__global__ __launch_bounds__(256) void la_step_kernel(Pass<DT> p, LaGeo g) {
  __shared__ float part[4][64];
  const int64_t nh = blockIdx.x;
  const int64_t n = nh / g.h, hd = nh - n * g.h;
  const int j0 = int(blockIdx.y) * 64 + int(threadIdx.x & 15) * 4, r0 = int(threadIdx.x >> 4) * NI;
  const int64_t base = nh * p.dk * p.dv;
  const Elem<DT>* qn = p.q + n * p.qs[0] + hd * p.qs[2] + r0;
  const Elem<DT>* kn = p.k + n * p.ks[0] + hd * p.ks[2] + r0;
  const Elem<DT>* vn = p.v + n * p.vs[0] + hd * p.vs[2] + j0;
  float s[NI][4], v[4], k[NI], q[NI], acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (VEC) {
    constexpr int V = NI * sizeof(Elem<DT>) > 16 ? 16 / sizeof(Elem<DT>) : NI;
    Pack<DT, V> kp[NI / V], qp[NI / V];
    Pack<DT, 4> vp{};
#pragma unroll
    for (int i = 0; i < NI / V; ++i) kp[i] = load_pack<DT, V>(kn + i * V), qp[i] = load_pack<DT, V>(qn + i * V);
    if (j0 < p.dv) vp = load_pack<DT, 4>(vn);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (j0 < p.dv) f = *reinterpret_cast<const float4*>(p.state + base + (r0 + i) * p.dv + j0);
      s[i][0] = f.x, s[i][1] = f.y, s[i][2] = f.z, s[i][3] = f.w;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) k[i] = to_f<DT>(kp[i / V].e[i % V]), q[i] = to_f<DT>(qp[i / V].e[i % V]);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = to_f<DT>(vp.e[e]);
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const bool in = r0 + i < p.dk;
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = in && j0 + e < p.dv ? p.state[base + (r0 + i) * p.dv + j0 + e] : 0.0f;
      k[i] = in ? to_f<DT>(kn[i]) : 0.0f;
      q[i] = in ? to_f<DT>(qn[i]) : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = j0 + e < p.dv ? to_f<DT>(vn[e]) : 0.0f;
  }
  const Decay decay(rate(g.log_decay[hd]));
#pragma unroll
  for (int i = 0; i < NI; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[i][e] = __builtin_fmaf(k[i], v[e], decay(s[i][e]));
      acc[e] = __builtin_fmaf(q[i], s[i][e], acc[e]);
    }
    float* to = p.state_out + base + (r0 + i) * p.dv + j0;
    if constexpr (VEC) {
      if (j0 < p.dv) *reinterpret_cast<float4*>(to) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r0 + i < p.dk && j0 + e < p.dv) to[e] = s[i][e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    acc[e] = add_halves(add_row_pairs(acc[e]));
    if ((threadIdx.x & 48) == 0) part[threadIdx.x >> 6][(threadIdx.x & 15) * 4 + e] = acc[e];
  }
  __syncthreads();
  const int j = int(blockIdx.y) * 64 + threadIdx.x;
  if (threadIdx.x < 64 && j < p.dv) {
    const float sum = (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
    p.y[nh * p.dv + j] = from_f<DT>(sum * p.scale_y);
  }
}

// ---------------------------------------------------------------- host

using Desc = cnhwc_linear_attention_desc_t;

// f(the type's constant)
template <typename F>
auto with_type(const Desc& d, F&& f) {
  if (d.dtype == CNHWC_F32) return f(std::integral_constant<int, CNHWC_F32>{});
  if (d.dtype == CNHWC_F16) return f(std::integral_constant<int, CNHWC_F16>{});
  return f(std::integral_constant<int, CNHWC_BF16>{});
}

template <typename F>
void with_rows(int32_t dk, F&& f) {  // rows of a thread
  if (dk <= 32) f(std::integral_constant<int, 2>{});
  else if (dk <= 64) f(std::integral_constant<int, 4>{});
  else if (dk <= 128) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

template <int DT>
void launch_step(const Pass<DT>& p, const LaGeo& g, int64_t nh, hipStream_t st) {
  const dim3 grid(unsigned(nh), unsigned((p.dv + 63) / 64));
  with_rows(p.dk, [&](auto ni) {
    constexpr int NI = decltype(ni)::value;
    constexpr uint64_t es = sizeof(Elem<DT>);
    constexpr int64_t V = NI * es > 16 ? 16 / es : NI;
    auto rows = [&](const void* q, const int64_t (&s)[3], int64_t v) {
      return aligned(q, v * es) && s[0] % v == 0 && s[2] % v == 0;
    };
    const bool vec = p.dk == 16 * NI && p.dv % 4 == 0 && rows(p.q, p.qs, V) && rows(p.k, p.ks, V) && rows(p.v, p.vs, 4);
    if (vec) hipLaunchKernelGGL((la_step_kernel<DT, NI, true>), grid, dim3(256), 0, st, p, g);
    else hipLaunchKernelGGL((la_step_kernel<DT, NI, false>), grid, dim3(256), 0, st, p, g);
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
  // the threads of a launch, and 64-bit offsets
  if (d->n * d->h > (1ll << 20) || d->l > (1ll << 30) || !dense_ok(d->n * d->h, d->l, d->dk > d->dv ? d->dk : d->dv))
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
  return {int32_t(d.l), int32_t(d.h), in.log_decay, in.lengths, 0, 0, 0};
}

template <int DT>
hipError_t forward_t(const Desc& d, const cnhwc_linear_attention_inputs_t& in, void* y, float* state_out,
                     char* workspace, hipStream_t st) {
  Passes<DT> ps{};
  ps.p[0] = pass_of<DT>(in.q, d.q_stride, in.k, d.k_stride, in.v, d.v_stride, y, d.dk, d.dv, d.scale, false);
  ps.p[0].state = in.state, ps.p[0].state_out = state_out;
  return launch_passes(ps, 1, geo_of(d, in), cut_of<DT>(d, d.dk, d.dv, 1), d.n * d.h, workspace, st);
}

template <int DT>
hipError_t step_t(const Desc& d, const cnhwc_linear_attention_inputs_t& in, void* y, float* state_out,
                  hipStream_t st) {
  Pass<DT> p = pass_of<DT>(in.q, d.q_stride, in.k, d.k_stride, in.v, d.v_stride, y, d.dk, d.dv, d.scale, false);
  p.state = in.state, p.state_out = state_out;
  launch_step(p, geo_of(d, in), d.n * d.h, st);
  return hipGetLastError();
}

// The cuts of the backward passes: of v's, whose state is [DK,DV], and of q's and k's,
// whose state is [DV,DK].  Where the two have one form all three go in one launch.
template <int DT>
bool one_form(const Desc& d) {
  int a = 0, b = 0;
  with_shape(d.dk, d.dv, false, [&](auto dkt, auto w) { a = dkt.value * 16 + w.value; });
  with_shape(d.dv, d.dk, false, [&](auto dkt, auto w) { b = dkt.value * 16 + w.value; });
  return a == b && (d.dk + 127) / 128 == (d.dv + 127) / 128;
}
template <int DT>
void backward_cuts(const Desc& d, Cut& v, Cut& qk) {
  if (one_form<DT>(d)) {
    v = qk = cut_of<DT>(d, d.dk, d.dv, 3);
  } else {
    v = cut_of<DT>(d, d.dk, d.dv, 1);
    qk = cut_of<DT>(d, d.dv, d.dk, 2);
  }
}
uint64_t backward_bytes(const Desc& d, bool decay_grad) {
  Cut v, qk;
  with_type(d, [&](auto dt) { backward_cuts<dt.value>(d, v, qk); });
  return v.bytes + 2 * qk.bytes + (decay_grad ? with_type(d, [&](auto dt) { return decay_cut_of<dt.value>(d).bytes; }) : 0);
}

template <int DT>
hipError_t backward_t(const Desc& d, const cnhwc_linear_attention_inputs_t& in, const void* dy,
                      const float* dstate_out, const cnhwc_linear_attention_grads_t& gr, char* workspace,
                      hipStream_t st) {
  const LaGeo g = geo_of(d, in);
  const int64_t nh = d.n * d.h;
  Pass<DT> q = pass_of<DT>(dy, d.dy_stride, in.v, d.v_stride, in.k, d.k_stride, gr.q, d.dv, d.dk, d.scale, false);
  q.state = in.state, q.state_k = 1, q.state_v = d.dv;  // S^T
  Pass<DT> v = pass_of<DT>(in.k, d.k_stride, in.q, d.q_stride, dy, d.dy_stride, gr.v, d.dk, d.dv, d.scale, true);
  v.state = dstate_out, v.state_out = gr.state;
  Pass<DT> k = pass_of<DT>(in.v, d.v_stride, dy, d.dy_stride, in.q, d.q_stride, gr.k, d.dv, d.dk, d.scale, true);
  k.state = dstate_out, k.state_k = 1, k.state_v = d.dv;
  Cut cv, cqk;
  backward_cuts<DT>(d, cv, cqk);
  hipError_t e;
  if (one_form<DT>(d)) {
    Passes<DT> ps{{q, k, v}};
    e = launch_passes(ps, 3, g, cv, nh, workspace, st);
  } else {
    Passes<DT> ps{{q, k}}, pv{{v}};
    e = launch_passes(ps, 2, g, cqk, nh, workspace, st);
    if (e == hipSuccess) e = launch_passes(pv, 1, g, cv, nh, workspace + 2 * cqk.bytes, st);
  }
  if (e != hipSuccess) return e;
  if (!gr.log_decay) return hipSuccess;
  DecayPass<DT> t{};
  t.a = pass_of<DT>(in.q, d.q_stride, in.k, d.k_stride, in.v, d.v_stride, nullptr, d.dk, d.dv, d.scale, false);
  t.a.state = in.state;
  t.dy = static_cast<const Elem<DT>*>(dy);
  for (int i = 0; i < 3; ++i) t.dys[i] = d.dy_stride[i];
  t.dstate = dstate_out;
  return launch_decay(t, g, decay_cut_of<DT>(d), nh, workspace + cv.bytes + 2 * cqk.bytes,
                      gr.log_decay, st);
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
  const Desc& d = *desc;
  *bytes = with_type(d, [&](auto dt) { return cut_of<dt.value>(d, d.dk, d.dv, 1).bytes; });
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
  char* ws = static_cast<char*>(workspace);
  const hipError_t e = with_type(d, [&](auto dt) { return forward_t<dt.value>(d, *in, y, state_out, ws, s); });
  return e == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
}

extern "C" cnhwc_status_t cnhwc_linear_attention_bwd_workspace(const Desc* desc, int32_t decay_grad,
                                                               uint64_t* bytes) {
  const cnhwc_status_t st = check_desc(desc, true);
  if (st != CNHWC_OK) return st;
  if (!bytes) return CNHWC_ERR_INVALID_ARGUMENT;
  *bytes = backward_bytes(*desc, decay_grad != 0);
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
  char* ws = static_cast<char*>(workspace);
  const hipError_t e = with_type(d, [&](auto dt) { return backward_t<dt.value>(d, *in, dy, dstate_out, *grads, ws, s); });
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
  const hipError_t e = with_type(d, [&](auto dt) { return step_t<dt.value>(d, *in, y, state_out, s); });
  return e == hipSuccess ? CNHWC_OK : CNHWC_ERR_HIP;
}
