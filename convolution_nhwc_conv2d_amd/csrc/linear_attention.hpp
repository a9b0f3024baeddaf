// Linear attention's passes in chunks of positions, as matrix products.
//
// A pass is y = scale q S with S from k and v (the gradients are passes with other
// tensors in these places).  In a chunk of C positions that starts from the state S,
//   y[u] = e^(g (u+1)) q[u] S + sum_{s <= u} e^(g (u-s)) (q[u] . k[s]) v[s]
//   S'   = e^(g C) S + sum_t k[t]^T (e^(g (C-1-t)) v[t])
// which is four matrix products: q k^T under its decays, that times v, q S, and k^T
// times the decayed v.  A pass from the end has u and s the other way round.
//
// A workgroup owns one head's state, or 64 or 128 columns of it, for a run of chunks.  A
// wavefront has 16 columns, in fp32 accumulators: a lane holds
// four consecutive rows of one column, which is just what the next product takes
// as its left operand (S^T), so the state never leaves the registers.  y is computed
// transposed for the same reason, and a lane then stores consecutive channels.
// Only the products of q and k go through LDS, since every wavefront needs all of them.
//
// Where one run of chunks a head would leave compute units without work, the sequence is
// cut into runs: one kernel takes the state that each leaves from a zero state, one joins
// these, and one takes the outputs.
//
// 16-bit types round two operands to themselves once, on the way to y (dq, dk, dv): the
// products of q and k under their decays, and the state that enters.  With the rounding of y
// itself that is 0.00235 of y's norm in bf16 and 0.00029 in f16, where y's alone is 0.00166 and
// 0.00021.  Both in two terms would leave that alone, and take bf16 1 x 16384 from 121 us to
// 136, 8 x 2048 114 to 124, its backward 202 to 243, f16 147 to 157, 131 to 139, 270 to 295 (16 heads of
// 128 x 128): not worth it for what is stored in 16 bits.  The state and its sums keep fp32's.
//
// Measured, bf16, 16 heads of 128 x 128.  1 x 16384: 118 us; on a trace, whose clocks are lower,
// the states of 32 runs 42, the join 15, the outputs 68; k and v are read twice and the states
// between runs written and read twice, 535 MB, at 4.5 TB/s.  8 x 2048 backward, three passes in
// one launch of 384 workgroups: 203 us; the vector pipes are busy for 35% of it, the matrix pipes
// 22%, the LDS 29%, and the rest is waiting: what a chunk does follows what the one before left
// (barriers, the state), two workgroups on half of the compute units and one on the others.
// f16 138 and 271, fp32 (matrix instructions of 154 TFLOP/s) 298 and 637.
#pragma once
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "device_common.hpp"
#include "seq_common.hpp"

namespace cnhwc {
namespace seq {

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
  bool halves;             // where not whole 16-byte pieces can be loaded: 8-byte ones can
  float4* kept;            // the states that enter all runs of chunks but the first, in lane order
};

struct LaGeo {
  int32_t l, h;
  const float* log_decay;
  const int32_t* lengths;
  int32_t chunks, run, runs;  // chunks of a sequence, of a run, runs of a sequence
};

// log_decay, finite for minus infinity too (0 times it is 0).
__device__ __forceinline__ float rate(float g) { return g < -FLT_MAX ? -FLT_MAX : g; }

// x -> exp(g) x without losing what a slow decay is about: exp(g) - 1 keeps its
// digits where exp(g), rounded, would be off by 2^-25 at every position, 10^-4
// after 4096 of them.
struct Decay {
  float m;    // exp(g) - 1, or exp(g)
  bool slow;  // the first
  __device__ __forceinline__ explicit Decay(float g) {
    slow = __builtin_fabsf(g) < 0.5f;
    m = slow ? expm1f(g) : exp_full(g);
  }
  // a choice, not a sum with 0 x: that would make NaN of an infinite state
  __device__ __forceinline__ float operator()(float x) const { return slow ? __builtin_fmaf(m, x, x) : m * x; }
  // of many: one instruction each
  template <int A>
  __device__ __forceinline__ void apply(v4f (&s)[A]) const {
    if (slow) {
#pragma unroll
      for (int a = 0; a < A; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[a][r] = __builtin_fmaf(m, s[a][r], s[a][r]);
    } else {
#pragma unroll
      for (int a = 0; a < A; ++a) s[a] *= m;
    }
  }
};

// The same over a run of chunks.  Growth there may be past fp32 where the states are 0 or so
// small that they stay within it: past e^88 it is taken in three factors, enough for any
// two fp32 values (e^-104 to e^88.7), so that 0 stays 0 and nothing is NaN.
struct RunDecay {
  Decay d;     // or its cube root
  float more;  // then that again, else 1
  __device__ __forceinline__ explicit RunDecay(float g)
      : d(g > 88.0f ? (g < 264.0f ? g : 264.0f) * (1.0f / 3.0f) : g), more(g > 88.0f ? d.m : 1.0f) {}
  __device__ __forceinline__ float operator()(float x) const { return d(x) * more * more; }
};

// Positions that a chunk's products take at a time: all of them, fewer where the state grows
// so fast that a way across the chunk would pass e^44, half of fp32's range: a value of
// k or v that the other one's zeros keep out of the state would be past fp32 with it, and
// infinity times 0 NaN.  f16, where a product's small operands lose digits beside large
// ones (Range), goes to e^8.  Decays, which is what this is for, take whole chunks.
template <int DT>
__device__ __forceinline__ int32_t step_shift(float g, int32_t chunk) {
  int32_t shift = 0;
  for (const float most = DT == CNHWC_F16 ? 8.0f : 44.0f; chunk >> shift > 1 && g * float(chunk >> shift) > most;) ++shift;
  return __builtin_amdgcn_readfirstlane(shift);
}

// What the matrix products are made of.  bf16 and f16: operands as they are, 32 deep; an
// fp32 operand is one or several 16-bit terms that add up to it (8 or 11 digits each).
// fp32: 16 deep in four instructions.  The depth runs over the lanes' four groups g in
// the order that the accumulators have (16 i + 4 g + r): a lane's elements are rows
// 4 g ... 4 g + 3 of one 16-row tile (fp32), or of two (16 bits).
template <int CT>
struct Mma {
  using T = uint16_t;
  using Frag = uint4;
  static constexpr bool kBf16 = CT == CNHWC_BF16;
  static constexpr int kDeep = 32, kPiece = 8, kTerms = kBf16 ? 3 : 2;
  static constexpr bool kScaled = !kBf16;  // fp32 operands are brought into f16's range first
  static __device__ __forceinline__ void mul(const Frag& a, const Frag& b, v4f& c) {
    if constexpr (kBf16)
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
    else
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
  // Two floats in one conversion, the first in the lower half; and back.
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    if constexpr (kBf16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{a, b}, v2bf));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{a, b}, v2h));
  }
  static __device__ __forceinline__ float low(uint32_t v) {
    if constexpr (kBf16) return __builtin_bit_cast(float, v << 16);
    else return to_f<CNHWC_F16>(uint16_t(v));
  }
  static __device__ __forceinline__ float high(uint32_t v) {
    if constexpr (kBf16) return __builtin_bit_cast(float, v & 0xffff0000u);
    else return to_f<CNHWC_F16>(uint16_t(v >> 16));
  }
};
template <>
struct Mma<CNHWC_F32> {
  using T = float;
  using Frag = float4;
  static constexpr int kDeep = 16, kPiece = 4, kTerms = 1;
  static constexpr bool kScaled = false;
  static __device__ __forceinline__ void mul(const Frag& a, const Frag& b, v4f& c) {
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.x, b.x, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.y, b.y, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.z, b.z, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.w, b.w, c, 0, 0, 0);
  }
};

// Whether an operand holds an infinity or NaN.
template <int CT>
__device__ __forceinline__ bool odd(const typename Mma<CT>::Frag& f) {
  if constexpr (CT == CNHWC_F32) {
    const float m = __builtin_fabsf(f.x) + __builtin_fabsf(f.y) + __builtin_fabsf(f.z) + __builtin_fabsf(f.w);
    return !(m <= FLT_MAX);  // or a sum past fp32, which the careful way takes as well
  } else {
    constexpr uint32_t kAll = CT == CNHWC_BF16 ? 0x7f807f80u : 0x7c007c00u;  // both exponents
    const uint32_t u[4] = {f.x, f.y, f.z, f.w};
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = ~u[i] & kAll;  // a half that is 0
      any |= (x - 0x00010001u) & ~x & 0x80008000u;
    }
    return any != 0;
  }
}
// An operand with 0 in the place of infinities and NaN; at(e) is called for each of those.
template <int CT, typename F>
__device__ __forceinline__ typename Mma<CT>::Frag without_odd(const typename Mma<CT>::Frag& f, F&& at) {
  if constexpr (CT == CNHWC_F32) {
    float x[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (!(__builtin_fabsf(x[e]) <= FLT_MAX)) x[e] = 0.0f, at(e);
    return make_float4(x[0], x[1], x[2], x[3]);
  } else {
    constexpr uint32_t kAll = CT == CNHWC_BF16 ? 0x7f80u : 0x7c00u;
    uint32_t u[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int up = e % 2 * 16;
      if ((u[e / 2] >> up & kAll) == kAll) u[e / 2] &= e % 2 ? 0x0000ffffu : 0xffff0000u, at(e);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// An operand of P floats as TERMS operands that add up to it, each `next` times as large as that.
template <int CT, int TERMS, int P>
__device__ __forceinline__ void split(const float (&x)[P], typename Mma<CT>::Frag (&f)[TERMS], float next = 1.0f) {
  if constexpr (P == 4) {
    f[0] = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    using M = Mma<CT>;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i];
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = M::pack(v[2 * i], v[2 * i + 1]);
        if (t + 1 < TERMS)
          v[2 * i] = (v[2 * i] - M::low(p[i])) * next, v[2 * i + 1] = (v[2 * i + 1] - M::high(p[i])) * next;
      }
      f[t] = make_uint4(p[0], p[1], p[2], p[3]);
    }
  }
}

// An operand's elements as floats.
template <int CT, int P>
__device__ __forceinline__ void unpack(const typename Mma<CT>::Frag& f, float (&x)[P]) {
  if constexpr (P == 4) {
    x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
  } else {
    const uint32_t u[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[2 * e] = Mma<CT>::low(u[e]), x[2 * e + 1] = Mma<CT>::high(u[e]);
  }
}

// Powers of two that bring fp32 values into f16's range and back: the largest of them to
// [2^14, 2^15), so that what is 2^28 times smaller still has all its 11 digits, and nothing
// is off by more than 2^-39 of the largest.  Of a position's products of q and k; of a
// wavefront's 16 columns of the state that enters y; of a column's decayed v in a chunk.
// Infinities and NaN are passed over: the values beside them keep theirs.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = __builtin_fabsf(x);
  return a <= FLT_MAX ? a : 0.0f;
}
struct Range {
  float in, out;
  __device__ __forceinline__ explicit Range(float largest) {
    int e = 15 - __builtin_amdgcn_frexp_expf(largest);
    e = e < -110 ? -110 : e > 110 ? 110 : e;
    in = __builtin_bit_cast(float, (127 + e) << 23);
    out = __builtin_bit_cast(float, (127 - e) << 23);
  }
};

// A tile of CH positions by COLS channels on its way from memory into LDS, rows of
// positions.  DEPTH: its channels are the depth of a product, and in bf16 each 32 of them
// stand in the order of the lanes (element 16 i + 4 g + r at 8 g + 4 i + r), so that an
// operand is one read of 16 bytes.  (In their own order it would be two of 8, which the
// compiler joins into a ds_read2_b64: 16 cycles a wavefront, where a ds_read_b128 takes 4
// and a transposing read 2.)  Behind a row 32 bytes in bf16 and 16 in fp32: the
// rows that are read together then lie in different banks (but for the transposing
// reads of a DEPTH tile, two to a bank, 4 cycles).
template <int DT, int CT, int COLS, int CH, int THREADS, bool DEPTH>
struct Rows2D {
  using M = Mma<CT>;
  using T = typename M::T;
  static constexpr int kPiece = M::kPiece, kPer = COLS / kPiece, kStep = THREADS / kPer;
  static constexpr int kCount = (CH + kStep - 1) / kStep;  // pieces of a thread; of some of the threads where
  static constexpr bool kSome = CH % kStep != 0;           // the tile is smaller than the workgroup
  static constexpr bool kHalf = sizeof(T) == 2;
  static constexpr int kStride = COLS * int(sizeof(T)) + (kHalf ? 32 : 16), kBytes = CH * kStride;
  static_assert(kCount == 1 || !kSome, "whole pieces for every thread");
  using Raw = PackBits<DT, kPiece>;  // held whole: as elements they would be taken apart on arrival
  Raw v[kCount];

  // Rows past `valid` and channels past `cols` are not read: VEC (whole pieces, 64 rows
  // within 32 bits of an offset) reads others instead, without a branch for every piece;
  // store() leaves them out.  halves: of 16-bit elements four at a time can be read.
  template <bool VEC>
  __device__ __forceinline__ void load(const Elem<DT>* __restrict__ base, int64_t stride, int32_t cols,
                                       int32_t valid, bool halves) {
    const int row0 = int(threadIdx.x) / kPer, col = int(threadIdx.x) % kPer * kPiece;
    const uint32_t at = uint32_t(col < cols ? col : 0), last = uint32_t(valid - 1);
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const uint32_t row = uint32_t(row0 + kStep * i);
      if constexpr (VEC) {
        v[i] = *reinterpret_cast<const Raw*>(base + (__umul24(row < last ? row : last, uint32_t(stride)) + at));
      } else {
        Pack<DT, kPiece> x{};
        if (row <= last) {
          const Elem<DT>* p = base + row * stride + col;
          if (kPiece == 8 && halves) {
#pragma unroll
            for (int e = 0; e < kPiece; e += 4)
              if (col + e < cols) {
                const Pack<DT, 4> y = load_pack<DT, 4>(p + e);
#pragma unroll
                for (int k = 0; k < 4; ++k) x.e[e + k] = y.e[k];
              }
          } else {
#pragma unroll
            for (int e = 0; e < kPiece; ++e)
              if (col + e < cols) x.e[e] = p[e];
          }
        }
        v[i] = __builtin_bit_cast(Raw, x);
      }
    }
  }

  // all: no row and no channel is left out
  __device__ __forceinline__ void store(char* lds, bool all, int32_t cols, int32_t valid) {
    const int row0 = int(threadIdx.x) / kPer, col = int(threadIdx.x) % kPer * kPiece;
    if (!all) {
#pragma unroll
      for (int i = 0; i < kCount; ++i)
        if (row0 + kStep * i >= valid || col >= cols) v[i] = Raw{};
    }
    if (kSome && row0 >= CH) return;
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const int row = row0 + kStep * i;
      char* p = lds + row * kStride;
      if constexpr (!kHalf) {
        const Pack<DT, 4> x = __builtin_bit_cast(Pack<DT, 4>, v[i]);
        *reinterpret_cast<float4*>(p + col * 4) =
            make_float4(to_f<DT>(x.e[0]), to_f<DT>(x.e[1]), to_f<DT>(x.e[2]), to_f<DT>(x.e[3]));
      } else {
        if constexpr (DEPTH) {
          char* o = p + (col & ~31) * 2 + (col & 8) * 4 + (col & 16) / 2;
          *reinterpret_cast<uint2*>(o) = make_uint2(v[i].x, v[i].y);
          *reinterpret_cast<uint2*>(o + 16) = make_uint2(v[i].z, v[i].w);
        } else {
          *reinterpret_cast<uint4*>(p + col * 2) = v[i];
        }
      }
    }
  }

  // The operand whose rows (or columns) are this tile's rows 16 i + (lane & 15), depth block kb.
  static __device__ __forceinline__ typename M::Frag along(const char* lds, int i, int kb) {
    static_assert(DEPTH, "the order of the lanes");
    const int lane = threadIdx.x & 63;
    return *reinterpret_cast<const typename M::Frag*>(lds + (16 * i + (lane & 15)) * kStride + kb * 64 + (lane >> 4) * 16);
  }
  // Stores what along() reads, for the 16 rows that the lanes are.
  static __device__ __forceinline__ void put(char* lds, int i, int kb, const typename M::Frag& f) {
    const int lane = threadIdx.x & 63;
    *reinterpret_cast<typename M::Frag*>(lds + (16 * i + (lane & 15)) * kStride + kb * 64 + (lane >> 4) * 16) = f;
  }
  // Channels 16 j + 4 g ... of position 16 i + c.
  static __device__ __forceinline__ void four(const char* lds, int i, int j, float (&x)[4]) {
    static_assert(DEPTH, "the order of the lanes");
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const char* p = lds + (16 * i + c) * kStride;
    if constexpr (!kHalf) {
      const float4 f = *reinterpret_cast<const float4*>(p + j * 64 + g * 16);
      x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
    } else {
      const uint2 f = *reinterpret_cast<const uint2*>(p + (j >> 1) * 64 + g * 16 + (j & 1) * 8);
      x[0] = M::low(f.x), x[1] = M::high(f.x), x[2] = M::low(f.y), x[3] = M::high(f.y);
    }
  }

  // The operand whose rows (or columns) are this tile's channels 16 j + (lane & 15) and
  // whose depth is its positions, block kb.  bf16: the LDS read that transposes.
  static __device__ __forceinline__ typename M::Frag across(const char* lds, int j, int kb) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    if constexpr (!kHalf) {
      const float* p = reinterpret_cast<const float*>(lds + (16 * kb + 4 * g) * kStride) + 16 * j + c;
      constexpr int s = kStride / 4;
      return make_float4(p[0], p[s], p[2 * s], p[3 * s]);
    } else {
      typedef short v4s __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) v4s lds_v4s;
      const int at = DEPTH ? (j >> 1) * 64 + (c & 3) * 16 + (j & 1) * 8 : j * 32 + (c & 3) * 8;
      const char* p = lds + (32 * kb + 4 * g + (c >> 2)) * kStride + at;
      const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p));
      const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 16 * kStride));
      const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
      return make_uint4(x.x, x.y, y.x, y.y);
    }
  }
};

// exp(g d) of the positions of a chunk, in LDS: from the entering state to a position, from a
// position to the chunk's end (0 past it), and from position to position.  Held in
// registers (36 of them) they would cost the second workgroup of a compute unit its place.
template <int CH>
struct Powers {
  float rise[CH];       // exp(g (i + 1))
  float fall[2 * CH];   // exp(g (CH - 1 - i)); 0 from CH on
  float far[2 * CH];    // exp(g |i - CH|)
  float row[CH];        // f16: what brings a row of products of q and k back from its range
  int first[8][4][16];  // where values are not finite: the first such position that a channel meets

  // by: a factor of the ways to the end and of those between positions.  Ways that are longer
  // than the sequence are 0: where the state grows (g > 0) they may be past fp32, and infinity
  // times the zeros behind the sequence would be NaN.
  __device__ __forceinline__ void fill(float gd, float by, bool back, int32_t len) {
    const int i = threadIdx.x;
    if (i < CH) {
      const float r = i < len ? exp_full(gd * float(i + 1)) : 0.0f;
      const float f = CH - 1 - i < len ? exp_full(gd * float(CH - 1 - i)) : 0.0f;
      rise[i] = back ? r * by : r;
      fall[i] = back ? f : f * by;
    } else if (i < 2 * CH) {
      fall[i] = 0.0f;
    }
    if (i < 2 * CH) {
      const int d = i < CH ? CH - i : i - CH;
      far[i] = d < len ? exp_full(gd * float(d)) * by : 0.0f;
    }
  }
  // of position t, from the start (back: to it) or to the end
  __device__ __forceinline__ const float* from_start(bool back, int valid) const {
    return back ? fall + (CH - valid) : rise;
  }
  __device__ __forceinline__ const float* to_end(bool back, int valid) const {
    return back ? rise : fall + (CH - valid);
  }
};

// The chunk of a pass's kernels and what they take: W wavefronts of 16 columns each.
// Chunks of 64 hold more registers, which the second workgroup of a compute unit needs
// (1 x 16384 x 16 x 128 x 128 bf16: 137 us with four wavefronts of 32 columns, 171 with eight of 16,
// which spill; chunks of 32 120).
template <int DT, int DKT, int W>
struct ChunkShape {
  using M = Mma<DT>;
  static constexpr int kShift = 5, kChunk = 1 << kShift;
  static constexpr int kThreads = 64 * W, kCols = 16 * W;
  static constexpr int kTiles = kChunk / 16;                  // of 16 positions
  static constexpr int kDepth = DKT * 16 / M::kDeep;          // blocks of a state's rows
  static constexpr int kBlocks = kChunk / M::kDeep;           // blocks of positions
  static constexpr int kPerBlock = M::kDeep / 16;             // 16-row tiles of a block
  using KTile = Rows2D<DT, DT, DKT * 16, kChunk, kThreads, true>;       // q and k
  using VTile = Rows2D<DT, DT, kCols, kChunk, kThreads, false>;
  using PTile = Rows2D<DT, DT, kChunk, kChunk, kThreads, true>;
  static constexpr int kLds = 2 * KTile::kBytes + VTile::kBytes + PTile::kBytes;
  // workgroups of a compute unit, eight wavefronts each: 128 registers hold 128 rows of a state
  // (64 beside fp32) and what goes with them, 256 rows take more
  static constexpr int kGroups = kLds <= 78 * 1024 && DKT * W <= (sizeof(typename M::T) == 2 ? 64 : 32) ? 2 : 1;
  static constexpr int kWaves = kGroups * W / 4;              // wavefronts of a SIMD
};

template <int DT>
struct Passes {
  Pass<DT> p[3];
};

// What a workgroup has: a part of the columns of a head's state, for a run.
struct Work {
  int32_t parts, part, run;  // run: in the order that the pass goes through them
  uint32_t nh, n, hd;
  __device__ __forceinline__ Work(int32_t columns, int32_t cols, int32_t runs, int32_t h) {
    parts = (columns + cols - 1) / cols;
    const uint32_t row = blockIdx.x / unsigned(parts);
    part = int32_t(blockIdx.x - row * unsigned(parts));
    nh = row / unsigned(runs);
    run = int32_t(row - nh * unsigned(runs));
    n = nh / unsigned(h), hd = nh - n * unsigned(h);
  }
};

constexpr float kHigher = 0x1p11f;  // of STEEP's second term

// What a workgroup does.  LOCAL: the state that a run of chunks leaves from a zero state
// (the first run: from the initial one), for all runs but the last.  Otherwise y and
// the final state.
//
// STEEP, f16 only: in the product that goes to the state v's second term loses its digits to
// f16's narrow range from 2^-17 of the column's largest on, and what is below 2^-39 of it
// is 0.  Where a chunk's decay is faster than 2^-8 that term stands 2^11 higher, in an
// accumulator of its own: digits down to 2^-27, 0 below 2^-50.  (For every head 8 x 2048 x 16 x
// 128 x 128 takes 139 us for 132, its backward 277 for 269.)
template <int DT, int DKT, int W, bool LOCAL, bool VEC, bool BACK, bool STEEP>
__device__ __forceinline__ void la_chunks(const Pass<DT>& p, const LaGeo& g, const Work& w, char* lds,
                                          Powers<ChunkShape<DT, DKT, W>::kChunk>& power) {
  using Sh = ChunkShape<DT, DKT, W>;
  using M = typename Sh::M;
  using Frag = typename M::Frag;
  using KTile = typename Sh::KTile;
  using VTile = typename Sh::VTile;
  using PTile = typename Sh::PTile;
  constexpr int CH = Sh::kChunk, MT = Sh::kTiles, PE = M::kPiece, PB = Sh::kPerBlock;
  char* const lds_k = lds;
  char* const lds_v = lds + KTile::kBytes;
  char* const lds_q = lds_v + VTile::kBytes;
  char* const lds_p = lds_q + KTile::kBytes;

  const int lane = threadIdx.x & 63, c = lane & 15, g4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t parts = w.parts, part = w.part, run = w.run;
  const int64_t nh = w.nh, n = w.n, hd = w.hd;
  const int32_t len = valid_len(g.lengths, n, g.l);
  const float gd = rate(g.log_decay[hd]);

  const int32_t at = BACK ? g.runs - 1 - run : run;
  // the run's positions; past the valid ones the state stands still
  const int32_t lo = at * g.run * CH, hi = lo + g.run * CH < g.l ? lo + g.run * CH : g.l;
  const int32_t end = len < lo ? lo : len < hi ? len : hi;
  const int32_t shift = step_shift<DT>(gd, CH), stride = CH >> shift;
  const int32_t count = (end - lo + stride - 1) >> (Sh::kShift - shift);
  const int32_t col0 = part * Sh::kCols, j = col0 + wave * 16 + c;

  // ---- the state: rows 16 a + 4 g + r of column j
  v4f s[DKT];
  float4* const kept = p.kept + ((nh * (g.runs - 1) * parts + part) * W + wave) * (DKT * 64) + lane;
  const int64_t kept_step = int64_t(parts) * W * (DKT * 64);  // to the next run's
  if (!LOCAL && run > 0) {
#pragma unroll
    for (int a = 0; a < DKT; ++a) s[a] = __builtin_bit_cast(v4f, kept[(run - 1) * kept_step + a * 64]);
  } else {
    const float* st = p.state && run == 0 ? p.state + nh * p.dk * p.dv : nullptr;
#pragma unroll
    for (int a = 0; a < DKT; ++a)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int32_t i = 16 * a + 4 * g4 + r;
        s[a][r] = st && i < p.dk && j < p.dv ? st[i * p.state_k + j * p.state_v] : 0.0f;
      }
  }

  power.fill(gd, p.scale_k, BACK, len < stride ? len : stride);
  const Decay full(gd * float(stride));

  const Elem<DT>* const qn = LOCAL ? nullptr : p.q + n * p.qs[0] + hd * p.qs[2];
  const Elem<DT>* const kn = p.k + n * p.ks[0] + hd * p.ks[2];
  const Elem<DT>* const vn = p.v + n * p.vs[0] + hd * p.vs[2] + col0;
  auto start_of = [&](int32_t i) { return lo + ((BACK ? count - 1 - i : i) << (Sh::kShift - shift)); };
  auto valid_at = [&](int32_t i) {
    const int32_t v = end - start_of(i);
    return v > stride ? stride : v;
  };
  const bool filled = p.dk == DKT * 16 && p.dv - col0 >= Sh::kCols;
  KTile tk, tq;
  VTile tv;
  auto fetch = [&](int64_t t0) {  // whole chunks: a smaller step's rows are left out on the way to LDS
    const int32_t valid = end - t0 > CH ? CH : int32_t(end - t0);
    tk.template load<VEC>(kn + t0 * p.ks[1], p.ks[1], p.dk, valid, p.halves);
    tv.template load<VEC>(vn + t0 * p.vs[1], p.vs[1], p.dv - col0, valid, p.halves);
    if constexpr (!LOCAL) tq.template load<VEC>(qn + t0 * p.qs[1], p.qs[1], p.dk, valid, p.halves);
  };
  if (end > lo) {  // loads that do not wait for the decay's; from the end a smaller step starts again
    fetch(BACK ? lo + ((end - lo - 1) & ~(CH - 1)) : lo);
    if (BACK && shift > 0) fetch(start_of(0));
  }
  if constexpr (!LOCAL) {
    const int64_t first = start_of(BACK ? -1 : count);  // behind what the steps store
    const int32_t wide = p.dv - col0 < Sh::kCols ? p.dv - col0 : Sh::kCols;
    for (int64_t e = threadIdx.x; e < (hi - first) * wide; e += Sh::kThreads)
      p.y[((n * g.l + first + e / wide) * g.h + hd) * p.dv + col0 + e % wide] = Elem<DT>(0);
  }

  // a lane has four channels of the positions 16 m + c
  using Raw4 = PackBits<DT, 4>;
  Raw4 out[LOCAL ? 1 : MT];
  int32_t out_t0 = 0;
  const int32_t j4 = col0 + wave * 16 + 4 * g4;
  auto put_y = [&]() __attribute__((always_inline)) {
    const int32_t rows = g.l - out_t0 < stride ? g.l - out_t0 : stride, live = len - out_t0;
    Elem<DT>* const base = p.y + ((n * g.l + out_t0) * g.h + hd) * p.dv;
    const int64_t step = int64_t(g.h) * p.dv;
    if constexpr (VEC) {
      const uint32_t to = __umul24(c, uint32_t(step)) + j4;  // 64 rows within 32 bits
      if (j4 < p.dv) {
        if (rows == CH && live >= CH) {
#pragma unroll
          for (int m = 0; m < MT; ++m) *reinterpret_cast<Raw4*>(base + m * 16 * step + to) = out[m];
        } else {
#pragma unroll
          for (int m = 0; m < MT; ++m)
            if (16 * m + c < rows) *reinterpret_cast<Raw4*>(base + m * 16 * step + to) = 16 * m + c < live ? out[m] : Raw4{};
        }
      }
    } else {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (16 * m + c >= rows) continue;
        const Pack<DT, 4> x = __builtin_bit_cast(Pack<DT, 4>, 16 * m + c < live ? out[m] : Raw4{});
        Elem<DT>* y = base + (16 * m + c) * step + j4;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (j4 + r < p.dv) y[r] = x.e[r];
      }
    }
  };

  for (int32_t step = 0; step < count; ++step) {
    const int32_t valid = valid_at(step);
    const int32_t t0 = start_of(step);
    __syncthreads();  // the chunk before has been read
    const bool all = filled && valid == CH;
    tk.store(lds_k, all, p.dk, valid);
    tv.store(lds_v, all, p.dv - col0, valid);
    if constexpr (!LOCAL) tq.store(lds_q, all, p.dk, valid);
    __syncthreads();
    if constexpr (!LOCAL) {
      if (step > 0) put_y();
    }
    if (step + 1 < count) fetch(start_of(step + 1));

    v4f o[LOCAL ? 1 : MT];
    if constexpr (!LOCAL) {
      // ---- (q k^T)^T under its decays, to LDS as rows of q: 16 rows by a block of k's
      // positions to a wavefront
      const int u = wave % MT;
      for (int b = wave / MT; b < Sh::kBlocks; b += W / MT) {
        if (BACK ? b < u / PB : b > u / PB) continue;
        float x[PE];
#pragma unroll
        for (int i = 0; i < PB; ++i) {
          const int tile = b * PB + i;
          v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
          if (BACK ? tile >= u : tile <= u) {
#pragma unroll
            for (int kb = 0; kb < Sh::kDepth; ++kb)
              M::mul(KTile::along(lds_k, tile, kb), KTile::along(lds_q, u, kb), acc);
          }
          const int far = 16 * (u - tile) + c - 4 * g4;  // from k's position (its first) to q's
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float by = power.far[CH + far - r];
            asm volatile("" : "+v"(by));  // read in any case: no branch around it
            x[4 * i + r] = (BACK ? far > r : far < r) ? 0.0f : acc[r] * by;
          }
        }
        if constexpr (M::kScaled) {
          static_assert(Sh::kBlocks == 1, "a row of products lies in one wavefront");
          float largest = 0.0f;
#pragma unroll
          for (int e = 0; e < PE; ++e) largest = __builtin_fmaxf(largest, finite_abs(x[e]));
          const Range to(max_halves(max_row_pairs(largest)));
#pragma unroll
          for (int e = 0; e < PE; ++e) x[e] *= to.in;
          if (g4 == 0) power.row[16 * u + c] = to.out;
        }
        Frag f[1];
        split<DT>(x, f);
        PTile::put(lds_p, u, b, f[0]);
      }
      // ---- S^T q^T, decayed from the chunk's start
#pragma unroll
      for (int m = 0; m < MT; ++m) o[m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      Range of_s(1.0f);
      if constexpr (M::kScaled) {
        float largest = 0.0f;
#pragma unroll
        for (int a = 0; a < DKT; ++a)
#pragma unroll
          for (int r = 0; r < 4; ++r) largest = __builtin_fmaxf(largest, finite_abs(s[a][r]));
        of_s = Range(group_max<64>(largest));
      }
#pragma unroll
      for (int kb = 0; kb < Sh::kDepth; ++kb) {
        float x[PE];
#pragma unroll
        for (int e = 0; e < PE; ++e) x[e] = s[kb * PB + e / 4][e % 4] * (M::kScaled ? of_s.in : 1.0f);
        Frag st[1];
        split<DT>(x, st);
#pragma unroll
        for (int m = 0; m < MT; ++m) M::mul(st[0], KTile::along(lds_q, m, kb), o[m]);
      }
      const float* const from_start = power.from_start(BACK, valid) + c;
#pragma unroll
      for (int m = 0; m < MT; ++m) o[m] *= from_start[16 * m] * (M::kScaled ? of_s.out : 1.0f);
      __syncthreads();  // the products of q and k are there
    }

    Frag vf[Sh::kBlocks];
#pragma unroll
    for (int kb = 0; kb < Sh::kBlocks; ++kb) vf[kb] = VTile::across(lds_v, wave, kb);

    if constexpr (!LOCAL) {
      bool careful = false;
#pragma unroll
      for (int kb = 0; kb < Sh::kBlocks; ++kb) careful |= odd<DT>(vf[kb]);
      if (__builtin_amdgcn_ballot_w64(careful) == 0) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          v4f acc = M::kScaled ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : o[m];
#pragma unroll
          for (int kb = 0; kb < Sh::kBlocks; ++kb) {
            if (BACK ? kb < m / PB : kb > m / PB) continue;
            M::mul(vf[kb], PTile::along(lds_p, m, kb), acc);
          }
          if constexpr (M::kScaled) {
            const float by = power.row[16 * m + c];
#pragma unroll
            for (int r = 0; r < 4; ++r) o[m][r] = __builtin_fmaf(acc[r], by, o[m][r]);
          } else {
            o[m] = acc;
          }
        }
      } else {
        // An infinity or NaN times the 0 of a pair that comes the wrong way round would reach
        // the positions before it (behind it).  So 0 in its place, and NaN for the positions
        // that see it, in its channel.
        int first = BACK ? -1 : CH;  // of the lane's channel, j0 + c
        Frag clean[Sh::kBlocks];
#pragma unroll
        for (int kb = 0; kb < Sh::kBlocks; ++kb)
          clean[kb] = without_odd<DT>(vf[kb], [&](int e) {
            const int t = kb * M::kDeep + e / 4 * 16 + 4 * g4 + e % 4;
            first = BACK ? (t > first ? t : first) : (t < first ? t : first);
          });
        power.first[wave][g4][c] = first;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          int f = power.first[wave][0][4 * g4 + r];
#pragma unroll
          for (int g = 1; g < 4; ++g) {
            const int h = power.first[wave][g][4 * g4 + r];
            f = BACK ? (h > f ? h : f) : (h < f ? h : f);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
            if (BACK ? 16 * m + c <= f : 16 * m + c >= f) o[m][r] = __builtin_nanf("");
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int kb = 0; kb < Sh::kBlocks; ++kb) {
            if (BACK ? kb < m / PB : kb > m / PB) continue;
            M::mul(clean[kb], PTile::along(lds_p, m, kb), acc);
          }
          const float by = M::kScaled ? power.row[16 * m + c] : 1.0f;
#pragma unroll
          for (int r = 0; r < 4; ++r) o[m][r] = __builtin_fmaf(acc[r], by, o[m][r]);
        }
      }
      // ---- y, to be stored when the next chunk has arrived: the wait for that chunk
      // would be for these stores too
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const v4f f = o[m] * p.scale_y;
        if constexpr (DT != CNHWC_F32) {
          out[m] = make_uint2(M::pack(f[0], f[1]), M::pack(f[2], f[3]));
        } else {
          Pack<DT, 4> x;
#pragma unroll
          for (int r = 0; r < 4; ++r) x.e[r] = from_f<DT>(f[r]);
          out[m] = __builtin_bit_cast(Raw4, x);
        }
      }
      out_t0 = t0;
    }

    // ---- S <- decay S + k^T (decayed v)
    (valid == stride ? full : Decay(gd * float(valid))).apply(s);
    const float* const to_end = power.to_end(BACK, valid) + 4 * g4;
#pragma unroll
    for (int kb = 0; kb < Sh::kBlocks; ++kb) {
      float x[PE];
      unpack<DT>(vf[kb], x);
#pragma unroll
      for (int e = 0; e < PE; ++e) x[e] *= to_end[kb * M::kDeep + (e / 4) * 16 + e % 4];
      Range of_v(1.0f);  // of the lane's column, which is the state's
      if constexpr (M::kScaled) {
        float largest = 0.0f;
#pragma unroll
        for (int e = 0; e < PE; ++e) largest = __builtin_fmaxf(largest, finite_abs(x[e]));
        of_v = Range(max_halves(max_row_pairs(largest)));
#pragma unroll
        for (int e = 0; e < PE; ++e) x[e] *= of_v.in;
      }
      Frag vt[M::kTerms];
      split<DT>(x, vt, STEEP ? kHigher : 1.0f);
#pragma unroll
      for (int a = 0; a < DKT; ++a) {
        const Frag f = KTile::across(lds_k, a, kb);
        v4f acc = M::kScaled ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : s[a];
#pragma unroll
        for (int t = 0; t < (STEEP ? 1 : M::kTerms); ++t) M::mul(f, vt[t], acc);
        if constexpr (STEEP) {
          v4f next = {0.0f, 0.0f, 0.0f, 0.0f};
          M::mul(f, vt[M::kTerms - 1], next);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(next[r], 1.0f / kHigher, acc[r]);
        }
        if constexpr (M::kScaled) {
#pragma unroll
          for (int r = 0; r < 4; ++r) s[a][r] = __builtin_fmaf(acc[r], of_v.out, s[a][r]);
        } else {
          s[a] = acc;
        }
      }
    }
  }

  if constexpr (!LOCAL) {
    if (count > 0) put_y();
  }
  if constexpr (LOCAL) {
#pragma unroll
    for (int a = 0; a < DKT; ++a) kept[run * kept_step + a * 64] = __builtin_bit_cast(float4, s[a]);
  } else if (p.state_out && run == g.runs - 1) {
    float* st = p.state_out + nh * p.dk * p.dv;
#pragma unroll
    for (int a = 0; a < DKT; ++a)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int32_t i = 16 * a + 4 * g4 + r;
        if (i < p.dk && j < p.dv) st[i * p.state_k + j * p.state_v] = s[a][r];
      }
  }
}

template <int DT, int DKT, int W, bool LOCAL, bool VEC>
__global__ __launch_bounds__(64 * W, (ChunkShape<DT, DKT, W>::kWaves)) void la_chunk_kernel(Passes<DT> passes,
                                                                                           LaGeo g) {
  using Sh = ChunkShape<DT, DKT, W>;
  __shared__ __attribute__((aligned(16))) char lds[LOCAL ? Sh::KTile::kBytes + Sh::VTile::kBytes : Sh::kLds];
  __shared__ Powers<Sh::kChunk> power;
  const Pass<DT>& p = passes.p[blockIdx.y];
  const Work w(p.dv, Sh::kCols, LOCAL ? g.runs - 1 : g.runs, g.h);
  auto run = [&](auto steep) __attribute__((always_inline)) {
    if (p.back) la_chunks<DT, DKT, W, LOCAL, VEC, true, decltype(steep)::value>(p, g, w, lds, power);
    else la_chunks<DT, DKT, W, LOCAL, VEC, false, decltype(steep)::value>(p, g, w, lds, power);
  };
  if constexpr (Sh::M::kScaled) {
    const bool steep = __builtin_fabsf(rate(g.log_decay[w.hd])) * float(Sh::kChunk) > 5.5f;
    if (__builtin_amdgcn_readfirstlane(steep)) return run(std::true_type{});
  }
  run(std::false_type{});
}

// Along the runs, in place: what each leaves from a zero state -> the state that
// enters the next one.  `per` float4 of every head and run.
template <int DT>
__global__ __launch_bounds__(256) void la_join_kernel(Passes<DT> passes, LaGeo g, int64_t heads, int32_t per,
                                                      int32_t chunk) {
  const Pass<DT>& p = passes.p[blockIdx.y];
  const int32_t slots = g.runs - 1;
  const int64_t total = heads * per;
  for (int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x; id < total; id += int64_t(gridDim.x) * 256) {
    const int64_t nh = id / per;
    const int64_t n = nh / g.h, hd = nh - n * g.h;
    const int32_t len = valid_len(g.lengths, n, g.l);
    const float gd = rate(g.log_decay[hd]);
    float4* at = p.kept + nh * slots * per + (id - nh * per);
    constexpr int kAhead = 8;
    float4 h = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int32_t k0 = 0; k0 < slots; k0 += kAhead) {
      float4 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (k0 + i < slots) v[i] = at[int64_t(k0 + i) * per];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (k0 + i >= slots) break;
        const int32_t run = p.back ? g.runs - 1 - (k0 + i) : k0 + i;
        const int32_t lo = run * g.run * chunk, hi = (run + 1 == g.runs ? g.chunks : (run + 1) * g.run) * chunk;
        const int32_t valid = (hi < len ? hi : len) - lo;
        const RunDecay d(gd * float(valid < 0 ? 0 : valid));
        h.x = d(h.x) + v[i].x, h.y = d(h.y) + v[i].y, h.z = d(h.z) + v[i].z, h.w = d(h.w) + v[i].w;
        at[int64_t(k0 + i) * per] = h;
      }
    }
  }
}

// ---------------------------------------------------------------- the decay's gradient
//
// With T[t] = e^g (T[t-1] + S[t-1]), the state's derivative by g, the gradient is
// sum_t scale dy[t] q[t] T[t] + dstate T[L].  In a chunk that starts from S and T
//   dy[u] . q[u] T[u] = e^(g (u+1)) dy[u] . q[u] (T + (u+1) S)
//                       + sum_{s < u} (u-s) e^(g (u-s)) (q[u] . k[s]) (dy[u] . v[s])
//   T' = e^(g C) (T + C S) + sum_t k[t]^T ((C-1-t) e^(g (C-1-t)) v[t])
// Every sum here is over what it is about: the shorter form sum_t t (q dq - k dk)
// would lose the gradient in the difference of sums that grow with the length.  A
// workgroup holds 64 columns of both states; S, T and the decayed v are taken in all
// their terms, so nothing is rounded below fp32.
//
// 8 x 2048 x 16 heads x 128 x 128 bf16: 178 us on a trace, 156 more for the call; vector pipes 56%
// (the terms), matrix pipes 29%, LDS 26%; one workgroup of eight wavefronts a compute unit, whose
// registers are the two states.  Chunks of 32 with three of four: 10% more for the whole backward
// pass.  f16 goes in fp32, 412 us more: in two f16 terms S, T and both decayed v would each need
// a range.  (An f16 value is two bf16 terms; with three of the states' that would be
// five products of 16 cycles for the 256 of the fp32 instructions.  Not tried.)
template <int DT>
struct DecayPass {
  Pass<DT> a;               // q, k, v, the initial state; y, state_out unused
  const Elem<DT>* dy;
  int64_t dys[3];
  const float* dstate;      // [DK,DV], or NULL
  float* sums;              // one for each workgroup
};

template <int DT, int DKT>
struct DecayShape {
  static constexpr int CT = DT == CNHWC_F16 ? CNHWC_F32 : DT;  // f16 is taken in fp32
  static constexpr int kChunk = sizeof(typename Mma<CT>::T) == 4 && DKT == 16 ? 32 : 64;
  // Four wavefronts of 16 columns, twice where the state has rows enough: one has the
  // upper half of them, one the lower (every sum here is a sum over the rows too).  One
  // workgroup of 64 columns a compute unit then has two wavefronts on a SIMD.
  static constexpr int kSplit = DKT >= 4 ? 2 : 1, kTiles = DKT / kSplit, kThreads = 256 * kSplit;
  using KTile = Rows2D<DT, CT, DKT * 16, kChunk, kThreads, true>;
  using VTile = Rows2D<DT, CT, 64, kChunk, kThreads, true>;
  static constexpr int kLds = 2 * KTile::kBytes + 2 * VTile::kBytes;
  static constexpr int kGroups = (DKT == 2 || (DKT == 4 && sizeof(typename Mma<CT>::T) == 2)) && kLds <= 76 * 1024 ? 2 : 1;
};

template <int DT, int DKT, bool LOCAL, bool VEC>
__global__ __launch_bounds__((DecayShape<DT, DKT>::kThreads),
                             (DecayShape<DT, DKT>::kGroups * DecayShape<DT, DKT>::kSplit)) void la_decay_kernel(
    DecayPass<DT> pass, LaGeo g) {
  using Sh = DecayShape<DT, DKT>;
  constexpr int CT = Sh::CT;
  using M = Mma<CT>;
  using Frag = typename M::Frag;
  using KTile = typename Sh::KTile;
  using VTile = typename Sh::VTile;
  constexpr int CH = Sh::kChunk, MT = CH / 16, PE = M::kPiece, PB = M::kDeep / 16, TERMS = M::kTerms;
  constexpr int kBlocks = CH / M::kDeep, TA = Sh::kTiles, KD = TA * 16 / M::kDeep;
  __shared__ __attribute__((aligned(16))) char lds[LOCAL ? KTile::kBytes + VTile::kBytes : Sh::kLds];
  __shared__ Powers<CH> power;
  __shared__ float red[4 * Sh::kSplit];
  char* const lds_k = lds;
  char* const lds_v = lds + KTile::kBytes;
  char* const lds_q = lds_v + VTile::kBytes;
  char* const lds_d = lds_q + KTile::kBytes;

  const Pass<DT>& p = pass.a;
  const int lane = threadIdx.x & 63, c = lane & 15, g4 = lane >> 4;
  const int every = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = every & 3, half = every >> 2;  // columns; rows of the states
  const int32_t parts = (p.dv + 63) / 64, part = int32_t(blockIdx.x % unsigned(parts));
  const int64_t row = blockIdx.x / unsigned(parts);
  const int32_t runs = LOCAL ? g.runs - 1 : g.runs;
  const int64_t nh = row / runs;
  const int32_t run = int32_t(row - nh * runs);
  const int64_t n = nh / g.h, hd = nh - n * g.h;
  const int32_t len = valid_len(g.lengths, n, g.l);
  const float gd = rate(g.log_decay[hd]);
  const int32_t lo = run * g.run * CH, hi = lo + g.run * CH < len ? lo + g.run * CH : len;  // the run's valid positions
  const int32_t stride = CH >> step_shift<CT>(gd, CH);
  const int32_t col0 = part * 64, j = col0 + wave * 16 + c;

  v4f s[TA], grow[TA];  // rows row0 + 16 a + 4 g + r, column j
  const int32_t row0 = half * TA * 16 + 4 * g4;
  float4* const kept = p.kept + ((nh * (g.runs - 1) * parts + part) * (4 * Sh::kSplit) + every) * (2 * TA * 64) + lane;
  const int64_t kept_step = int64_t(parts) * 4 * (2 * DKT * 64);
  const float* st = p.state && run == 0 ? p.state + nh * p.dk * p.dv : nullptr;
#pragma unroll
  for (int a = 0; a < TA; ++a) {
    if (!LOCAL && run > 0) {
      s[a] = __builtin_bit_cast(v4f, kept[(run - 1) * kept_step + 2 * a * 64]);
      grow[a] = __builtin_bit_cast(v4f, kept[(run - 1) * kept_step + (2 * a + 1) * 64]);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int32_t i = row0 + 16 * a + r;
        s[a][r] = st && i < p.dk && j < p.dv ? st[int64_t(i) * p.dv + j] : 0.0f;
        grow[a][r] = 0.0f;
      }
    }
  }
  power.fill(gd, 1.0f, false, len < stride ? len : stride);

  const Elem<DT>* const qn = p.q + n * p.qs[0] + hd * p.qs[2];
  const Elem<DT>* const kn = p.k + n * p.ks[0] + hd * p.ks[2];
  const Elem<DT>* const vn = p.v + n * p.vs[0] + hd * p.vs[2] + col0;
  const Elem<DT>* const dn = LOCAL ? nullptr : pass.dy + n * pass.dys[0] + hd * pass.dys[2] + col0;
  const bool filled = p.dk == DKT * 16 && p.dv - col0 >= 64;
  KTile tk, tq;
  VTile tv, td;
  auto fetch = [&](int64_t t0) {  // whole chunks: a smaller step's rows are left out on the way to LDS
    const int32_t valid = hi - t0 > CH ? CH : int32_t(hi - t0);
    tk.template load<VEC>(kn + t0 * p.ks[1], p.ks[1], p.dk, valid, p.halves);
    tv.template load<VEC>(vn + t0 * p.vs[1], p.vs[1], p.dv - col0, valid, p.halves);
    if constexpr (!LOCAL) {
      tq.template load<VEC>(qn + t0 * p.qs[1], p.qs[1], p.dk, valid, p.halves);
      td.template load<VEC>(dn + t0 * pass.dys[1], pass.dys[1], p.dv - col0, valid, p.halves);
    }
  };
  if (lo < hi) fetch(lo);
  double total = 0.0;
  for (int32_t at = lo; at < hi; at += stride) {
    const int32_t valid = hi - at > stride ? stride : hi - at;
    __syncthreads();  // the chunk before has been read
    const bool all = filled && valid == CH;
    tk.store(lds_k, all, p.dk, valid);
    tv.store(lds_v, all, p.dv - col0, valid);
    if constexpr (!LOCAL) {
      tq.store(lds_q, all, p.dk, valid);
      td.store(lds_d, all, p.dv - col0, valid);
    }
    __syncthreads();
    if (at + stride < hi) fetch(at + stride);

    if constexpr (!LOCAL) {
      float sum = 0.0f;
      // ---- pairs of positions: the wavefront's 16 u = 16 wave + c, s = 16 i + 4 g + r
      if (wave < MT) {
        for (int i = half; i <= wave; i += Sh::kSplit) {
          v4f x = {0.0f, 0.0f, 0.0f, 0.0f}, y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int kb = 0; kb < DKT * 16 / M::kDeep; ++kb)
            M::mul(KTile::along(lds_k, i, kb), KTile::along(lds_q, wave, kb), x);
#pragma unroll
          for (int kb = 0; kb < 64 / M::kDeep; ++kb)
            M::mul(VTile::along(lds_v, i, kb), VTile::along(lds_d, wave, kb), y);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int d = 16 * (wave - i) + c - 4 * g4 - r;
            if (d > 0) sum = __builtin_fmaf(x[r] * y[r], float(d) * power.far[CH + d], sum);
          }
        }
      }
      // ---- through the states at the chunk's start
      v4f xs[MT], ys[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) xs[m] = ys[m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kb = 0; kb < KD; ++kb) {
        float fs[PE], ft[PE];
#pragma unroll
        for (int e = 0; e < PE; ++e) fs[e] = s[kb * PB + e / 4][e % 4], ft[e] = grow[kb * PB + e / 4][e % 4];
        Frag a[TERMS], b[TERMS];
        split<CT>(fs, a);
        split<CT>(ft, b);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const Frag f = KTile::along(lds_q, m, half * KD + kb);
#pragma unroll
          for (int t = 0; t < TERMS; ++t) {
            M::mul(a[t], f, xs[m]);
            M::mul(b[t], f, ys[m]);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const v4f x = xs[m], y = ys[m];
        // rows: channels 16 wave + 4 g + r; column: position 16 m + c (0 past the valid ones, as dy is)
        float dy[4];
        VTile::four(lds_d, m, wave, dy);
        const float far = float(16 * m + c + 1);
        float one = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) one = __builtin_fmaf(dy[r], __builtin_fmaf(far, x[r], y[r]), one);
        sum = __builtin_fmaf(power.rise[16 * m + c], one, sum);
      }
      total += double(sum);
    }

    // ---- both states to the chunk's end
    const Decay whole(gd * float(valid));
#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        grow[a][r] = whole(__builtin_fmaf(float(valid), s[a][r], grow[a][r]));
        s[a][r] = whole(s[a][r]);
      }
#pragma unroll
    for (int kb = 0; kb < kBlocks; ++kb) {
      const Frag f = VTile::across(lds_v, wave, kb);
      float x[PE], y[PE];
      unpack<CT>(f, x);
#pragma unroll
      for (int e = 0; e < PE; ++e) {
        const int t = kb * M::kDeep + (e / 4) * 16 + 4 * g4 + e % 4;
        x[e] *= power.fall[CH - valid + t];
        y[e] = x[e] * float(valid - 1 - t);
      }
      Frag vs[TERMS], vt[TERMS];
      split<CT>(x, vs);
      split<CT>(y, vt);
#pragma unroll
      for (int a = 0; a < TA; ++a) {
        const Frag k = KTile::across(lds_k, half * TA + a, kb);
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
          M::mul(k, vs[t], s[a]);
          M::mul(k, vt[t], grow[a]);
        }
      }
    }
  }

  if constexpr (LOCAL) {
#pragma unroll
    for (int a = 0; a < TA; ++a) {
      kept[run * kept_step + 2 * a * 64] = __builtin_bit_cast(float4, s[a]);
      kept[run * kept_step + (2 * a + 1) * 64] = __builtin_bit_cast(float4, grow[a]);
    }
  } else {
    total *= double(p.scale_y);
    if (pass.dstate && run == g.runs - 1) {
      const float* ds = pass.dstate + nh * p.dk * p.dv;
      float sum = 0.0f;
#pragma unroll
      for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int32_t i = row0 + 16 * a + r;
          if (i < p.dk && j < p.dv) sum = __builtin_fmaf(ds[int64_t(i) * p.dv + j], grow[a][r], sum);
        }
      total += double(sum);
    }
    const float one = group_sum<64>(float(total));
    if (lane == 0) red[every] = one;
    __syncthreads();
    if (threadIdx.x == 0) {
      float sum = red[0];
#pragma unroll
      for (int w = 1; w < 4 * Sh::kSplit; ++w) sum += red[w];
      pass.sums[blockIdx.x] = sum;
    }
  }
}

// Along the runs, in place, as la_join_kernel; the two states of a row of 16 lie side by side.
template <int DT>
__global__ __launch_bounds__(256) void la_decay_join_kernel(DecayPass<DT> pass, LaGeo g, int64_t heads, int32_t per,
                                                            int32_t chunk) {
  const int32_t slots = g.runs - 1, half = per / 2;
  const int64_t total = heads * half;
  for (int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x; id < total; id += int64_t(gridDim.x) * 256) {
    const int64_t nh = id / half;
    const int32_t i = int32_t(id - nh * half);
    const int64_t n = nh / g.h, hd = nh - n * g.h;
    const int32_t len = valid_len(g.lengths, n, g.l);
    const float gd = rate(g.log_decay[hd]);
    float4* at = pass.a.kept + nh * slots * per + (i >> 6) * 128 + (i & 63);
    v4f h = {0.0f, 0.0f, 0.0f, 0.0f}, t = h;
    for (int32_t k = 0; k < slots; ++k, at += per) {
      const int32_t lo = k * g.run * chunk, hi = (k + 1) * g.run * chunk;
      const int32_t valid = (hi < len ? hi : len) - lo;
      const float count = float(valid < 0 ? 0 : valid);
      const RunDecay d(gd * count);
      const v4f s = __builtin_bit_cast(v4f, at[0]), grow = __builtin_bit_cast(v4f, at[64]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        t[r] = d(__builtin_fmaf(count, h[r], t[r])) + grow[r];
        h[r] = d(h[r]) + s[r];
      }
      at[0] = __builtin_bit_cast(float4, h);
      at[64] = __builtin_bit_cast(float4, t);
    }
  }
}

}  // namespace seq
}  // namespace cnhwc
