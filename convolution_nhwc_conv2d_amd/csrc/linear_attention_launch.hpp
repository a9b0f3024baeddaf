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
  bool vec = true;
  for (int i = 0; i < count; ++i) {
    Pass<DT>& p = ps.p[i];
    vec = vec && whole(p.q, p.qs, p.dk, kPiece, es) && whole(p.k, p.ks, p.dk, kPiece, es) &&
          whole(p.v, p.vs, p.dv, kPiece, es) && aligned(p.y, 4 * es);
    p.kept = reinterpret_cast<float4*>(workspace + i * c.bytes);
  }
  with_shape(ps.p[0].dk, ps.p[0].dv, [&](auto dkt, auto nt) {
    constexpr int DKT = decltype(dkt)::value, NT = decltype(nt)::value;
    const int64_t blocks = heads * c.parts;
    auto run = [&](auto v) {
      constexpr bool VEC = decltype(v)::value;
      if (c.runs > 1) {
        hipLaunchKernelGGL((la_chunk_kernel<DT, DKT, NT, true, VEC>), dim3(unsigned(blocks * (c.runs - 1)), count),
                           dim3(256), 0, st, ps, g);
        const int64_t total = heads * c.per;
        hipLaunchKernelGGL((la_join_kernel<DT>), dim3(grid_of(ceil_div(total, int64_t(256))).x, count), dim3(256), 0,
                           st, ps, g, heads, c.per, c.chunk);
      }
      hipLaunchKernelGGL((la_chunk_kernel<DT, DKT, NT, false, VEC>), dim3(unsigned(blocks * c.runs), count), dim3(256),
                         0, st, ps, g);
    };
    if (vec) run(std::true_type{});
    else run(std::false_type{});
  });
  return hipGetLastError();
}

}  // namespace seq
}  // namespace cnhwc
