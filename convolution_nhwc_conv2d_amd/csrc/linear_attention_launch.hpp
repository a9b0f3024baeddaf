// The launches of linear attention's passes, for the source of each type.
#pragma once
#include "linear_attention_host.hpp"

namespace cnhwc {
namespace seq {

template <int DT>
hipError_t launch_passes(Passes<DT>& ps, int count, LaGeo g, const Cut& c, int64_t heads, char* workspace,
                         hipStream_t st) {
  const uint64_t es = sizeof(Elem<DT>);
  constexpr int kPiece = Mma<DT>::kPiece;
  g.chunks = c.chunks, g.run = c.run, g.runs = c.runs;
  bool vec = true, halves = true;
  for (int i = 0; i < count; ++i) {
    Pass<DT>& p = ps.p[i];
    vec = vec && whole(p.q, p.qs, p.dk, kPiece, es) && whole(p.k, p.ks, p.dk, kPiece, es) &&
          whole(p.v, p.vs, p.dv, kPiece, es) && aligned(p.y, 4 * es) && int64_t(g.h) * p.dv < (1 << 23);
    halves = halves && whole(p.q, p.qs, p.dk, 4, es) && whole(p.k, p.ks, p.dk, 4, es) && whole(p.v, p.vs, p.dv, 4, es);
    p.kept = reinterpret_cast<float4*>(workspace + i * c.bytes);
  }
  for (int i = 0; i < count; ++i) ps.p[i].halves = halves;
  with_shape(ps.p[0].dk, ps.p[0].dv, c.narrow, [&](auto dkt, auto w) {
    constexpr int DKT = decltype(dkt)::value, W = decltype(w)::value;
    const int64_t blocks = heads * c.parts;
    auto run = [&](auto v) {
      constexpr bool VEC = decltype(v)::value;
      if (c.runs > 1) {
        hipLaunchKernelGGL((la_chunk_kernel<DT, DKT, W, true, VEC>), dim3(unsigned(blocks * (c.runs - 1)), count),
                           dim3(64 * W), 0, st, ps, g);
        const int64_t total = heads * c.per;
        hipLaunchKernelGGL((la_join_kernel<DT>), dim3(grid_of(ceil_div(total, int64_t(256))).x, count), dim3(256), 0,
                           st, ps, g, heads, c.per, c.chunk);
      }
      hipLaunchKernelGGL((la_chunk_kernel<DT, DKT, W, false, VEC>), dim3(unsigned(blocks * c.runs), count), dim3(64 * W),
                         0, st, ps, g);
    };
    if (vec) run(std::true_type{});
    else run(std::false_type{});
  });
  return hipGetLastError();
}

// The sums of a head, in a fixed order.
static __global__ __launch_bounds__(256) void la_decay_sum_kernel(const float* __restrict__ part,
                                                                  float* __restrict__ out, int64_t seqs, int64_t heads,
                                                                  int64_t blocks) {
  __shared__ double sum[256];
  const int64_t h = blockIdx.x, all = seqs * blocks;
  double v = 0.0;
  for (int64_t i = threadIdx.x; i < all; i += 256) v += double(part[(i / blocks * heads + h) * blocks + i % blocks]);
  sum[threadIdx.x] = v;
  __syncthreads();
  for (int k = 128; k > 0; k >>= 1) {
    if (int(threadIdx.x) < k) sum[threadIdx.x] += sum[threadIdx.x + k];
    __syncthreads();
  }
  if (threadIdx.x == 0) out[h] = float(sum[0]);
}

template <int DT>
hipError_t launch_decay(DecayPass<DT>& pass, LaGeo g, const Cut& c, int64_t heads, char* workspace, float* out,
                        hipStream_t st) {
  const uint64_t es = sizeof(Elem<DT>);
  constexpr int kPiece = Mma<DT == CNHWC_F16 ? CNHWC_F32 : DT>::kPiece;
  g.chunks = c.chunks, g.run = c.run, g.runs = c.runs;
  Pass<DT>& p = pass.a;
  const bool vec = whole(p.q, p.qs, p.dk, kPiece, es) && whole(p.k, p.ks, p.dk, kPiece, es) &&
                   whole(p.v, p.vs, p.dv, kPiece, es) && whole(pass.dy, pass.dys, p.dv, kPiece, es);
  p.halves = whole(p.q, p.qs, p.dk, 4, es) && whole(p.k, p.ks, p.dk, 4, es) && whole(p.v, p.vs, p.dv, 4, es) &&
             whole(pass.dy, pass.dys, p.dv, 4, es);
  const uint64_t states = uint64_t(heads) * (c.runs - 1) * c.per * 16;
  p.kept = reinterpret_cast<float4*>(workspace);
  pass.sums = reinterpret_cast<float*>(workspace + states);
  with_shape(p.dk, 64, false, [&](auto dkt, auto) {
    constexpr int DKT = decltype(dkt)::value;
    const int64_t blocks = heads * c.parts;
    auto run = [&](auto v) {
      constexpr bool VEC = decltype(v)::value;
      if (c.runs > 1) {
        hipLaunchKernelGGL((la_decay_kernel<DT, DKT, true, VEC>), dim3(unsigned(blocks * (c.runs - 1))),
                           dim3(DecayShape<DT, DKT>::kThreads), 0, st, pass, g);
        hipLaunchKernelGGL((la_decay_join_kernel<DT>), grid_of(ceil_div(heads * c.per / 2, int64_t(256))), dim3(256), 0,
                           st, pass, g, heads, c.per, c.chunk);
      }
      hipLaunchKernelGGL((la_decay_kernel<DT, DKT, false, VEC>), dim3(unsigned(blocks * c.runs)),
                         dim3(DecayShape<DT, DKT>::kThreads), 0, st, pass, g);
    };
    if (vec) run(std::true_type{});
    else run(std::false_type{});
  });
  hipLaunchKernelGGL(la_decay_sum_kernel, dim3(unsigned(g.h)), dim3(256), 0, st, pass.sums, out, heads / g.h,
                     int64_t(g.h), int64_t(c.parts) * c.runs);
  return hipGetLastError();
}

}  // namespace seq
}  // namespace cnhwc
