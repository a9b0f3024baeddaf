// Linear attention's passes on the host: how they are cut, and their launches.
#pragma once
#include "internal.hpp"
#include "linear_attention.hpp"
#include "seq_host.hpp"

namespace cnhwc {
namespace seq {

// The form of a pass: 16-row tiles of a state, wavefronts of a workgroup, 16 columns each.
// Eight where there are columns for them, since each workgroup takes up all of k and q and
// their products (16 heads of 128 x 128, bf16: 1 x 16384 122 us, with four 129; 8 x 2048 109, 121; backward
// 202, 213; f16 138, 158; 128, 158; but backward 271, 259).  fp32, where the matrix instructions weigh
// more than what they are fed from, has four (narrow) where half as many columns even out the
// workgroups, from 128 of eight wavefronts on: 8 x 2048 293 us, with four 257, backward 757, 638; but
// with 16 of them (1 x 16384) 298, 310, with 64 (4 x 4096 x 16 x 100 x 80) 298, 312, and with 256 rows 2 x 4096 x 8
// 282, 355, 8 x 2048 x 16 695, 959.
template <typename F>
void with_shape(int32_t dk, int32_t dv, bool narrow, F&& f) {
  auto wide = [&](auto dkt) {
    if (dv <= 64 || narrow) f(dkt, std::integral_constant<int, 4>{});
    else f(dkt, std::integral_constant<int, 8>{});
  };
  if (dk <= 32) wide(std::integral_constant<int, 2>{});
  else if (dk <= 64) wide(std::integral_constant<int, 4>{});
  else if (dk <= 128) wide(std::integral_constant<int, 8>{});
  else wide(std::integral_constant<int, 16>{});
}

// How a pass is cut: its chunk, the workgroups along a state's columns, the runs of
// chunks, and the bytes of the states between them.  A function of the sizes alone.
struct Cut {
  int32_t chunk, parts, chunks, run, runs;
  int32_t per;     // float4 of a head's state in lane order
  bool narrow;
  uint64_t bytes;
};
// More than one run costs a kernel over k and v, about 0.6 of the other one, and the
// states between them: worth it up to five workgroups for eight compute units.
// Measured (128 x 128 bf16, 2048 positions): 256 workgroups in one run 155 us, in two 181; 192
// 151 and 155; 128 in four 109, in two 125, in one 150, fp32 in two 293, in one 382; 64 x 64, 4096
// positions, 64 workgroups in eight 58, in four 81.  At least three chunks to a run, fewer only
// while every run has a compute unit to itself (1 x 300 x 4 heads of 64 x 64 one chunk 16 us, three
// 18; 3 x 591 x 96 x 100 fp32 26, 39, backward with the decay's gradient 65, 109; 2 x 1000 x 8 heads of
// 64 x 128 two 26, three 25, one 33, fp32 30, 32, 36; but 1 x 4096 x 8 x 128 x 128 two 49, three 44, four
// 39), and one run up to `few` chunks, whose time the two other kernels would not save.
inline void cut_runs(Cut& c, int64_t l, int64_t all, int64_t room, int64_t few) {
  c.chunks = int32_t((l + c.chunk - 1) / c.chunk);
  int64_t runs = all > 160 ? 1 : room / all;
  int64_t most = c.chunks / 3 > 256 / all ? c.chunks / 3 : 256 / all;
  if (most > c.chunks) most = c.chunks;
  if (runs > most) runs = most;
  if (runs < 1 || c.chunks <= few) runs = 1;
  c.run = int32_t((c.chunks + runs - 1) / runs);
  c.runs = (c.chunks + c.run - 1) / c.run;
}
template <int DT>
Cut cut_of(const cnhwc_linear_attention_desc_t& d, int32_t dk, int32_t dv, int64_t passes) {
  Cut c{};
  c.narrow = DT == CNHWC_F32 && dk <= 128 && dv <= 128 && d.n * d.h * passes >= 128;
  with_shape(dk, dv, c.narrow, [&](auto dkt, auto w) {
    constexpr int DKT = decltype(dkt)::value, W = decltype(w)::value;
    using Sh = ChunkShape<DT, DKT, W>;
    c.chunk = Sh::kChunk;
    c.parts = (dv + Sh::kCols - 1) / Sh::kCols;
    c.per = c.parts * W * DKT * 64;
    // a chunk in fp32 takes longer: 1 x 128 x 4 heads of 128 x 128 in four runs 21 us, in one 29, 64 x 64 15
    // and 14, 32 x 32 14 and 11; 2 x 130 x 8 of 64 x 96 in five 19, in one 23
    const int few = DT == CNHWC_F32 && DKT * W > 16 ? 3 : 5;
    cut_runs(c, d.l, d.n * d.h * c.parts * passes, 256 * Sh::kGroups, few);
  });
  c.bytes = uint64_t(d.n) * d.h * (c.runs - 1) * c.per * 16;
  return c;
}

// Whole pieces to load, and 64 rows within 32 bits of a byte offset.
inline bool whole(const void* p, const int64_t (&s)[3], int32_t c, int64_t piece, uint64_t es) {
  return aligned(p, piece * es) && c % piece == 0 && s[1] < (1 << 23) && s[0] % piece == 0 && s[1] % piece == 0 && s[2] % piece == 0;
}

// The same of the decay's gradient: both states, 64 columns a workgroup, and the
// workgroups' sums behind them.
template <int DT>
Cut decay_cut_of(const cnhwc_linear_attention_desc_t& d) {
  Cut c{};
  with_shape(d.dk, 64, false, [&](auto dkt, auto) {
    constexpr int DKT = decltype(dkt)::value;
    using Sh = DecayShape<DT, DKT>;
    c.chunk = Sh::kChunk;
    c.parts = (d.dv + 63) / 64;
    c.per = c.parts * 4 * DKT * 64 * 2;
    cut_runs(c, d.l, d.n * d.h * c.parts, 256 * Sh::kGroups, 3);
  });
  c.bytes = uint64_t(d.n) * d.h * (c.runs - 1) * c.per * 16 + (uint64_t(d.n) * d.h * c.parts * c.runs * 4 + 15) / 16 * 16;
  return c;
}

// One or several passes of the same form; each type's kernels are in a source of their own.
template <int DT>
hipError_t launch_passes(Passes<DT>& ps, int count, LaGeo g, const Cut& c, int64_t heads, char* workspace,
                         hipStream_t st);
template <int DT>
hipError_t launch_decay(DecayPass<DT>& pass, LaGeo g, const Cut& c, int64_t heads, char* workspace, float* out,
                        hipStream_t st);

}  // namespace seq
}  // namespace cnhwc
