// Host-side argument checks shared by the sequence operators.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

#include "cnhwc_seq.h"

namespace cnhwc {
namespace seq {

inline bool aligned(const void* p, uint64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool dtype_ok(int32_t dt) { return dt == CNHWC_F32 || dt == CNHWC_F16 || dt == CNHWC_BF16; }
inline bool extent_ok(int64_t v) { return v >= 1 && v < (1ll << 31); }

// Strides of an [n, l, c] tensor with unit channel stride: >= 0, and no offset
// past 2^60 (extents are below 2^31, so no product here wraps).
inline bool strides_ok(int64_t n, int64_t l, int64_t c, const int64_t (&s)[2]) {
  constexpr int64_t kMax = 1ll << 60;
  const int64_t ext[2] = {n, l};
  int64_t end = c;
  for (int i = 0; i < 2; ++i) {
    if (ext[i] == 1) continue;  // never multiplied by more than 0
    if (s[i] < 0 || s[i] > kMax / ext[i]) return false;
    end += (ext[i] - 1) * s[i];
  }
  return end <= kMax;
}

// n * l * c of a dense tensor stays below 2^60.
inline bool dense_ok(int64_t n, int64_t l, int64_t c) {
  return static_cast<unsigned __int128>(n) * static_cast<uint64_t>(l) * static_cast<uint64_t>(c) < (1ull << 60);
}

// Elements from the first to one past the last of a strided tensor.
inline uint64_t span(int64_t n, int64_t l, int64_t c, const int64_t (&s)[2]) {
  return uint64_t((n > 1 ? (n - 1) * s[0] : 0) + (l > 1 ? (l - 1) * s[1] : 0) + c);
}

// Workgroups of a kernel that walks over its work with the grid's stride: at
// most 2^20, so that the threads of the launch stay within 32 bits.
inline dim3 grid_of(int64_t blocks) { return dim3(unsigned(blocks < (1 << 20) ? blocks : (1 << 20))); }

// The buffers of one call: present where required, aligned, and no output
// overlapping any other buffer.
class Buffers {
 public:
  void in(const void* p, uint64_t bytes, uint64_t align, bool required) { add(p, bytes, align, required, false); }
  void out(const void* p, uint64_t bytes, uint64_t align, bool required) { add(p, bytes, align, required, true); }
  bool ok() const {
    if (bad_) return false;
    for (int i = 0; i < n_; ++i)
      for (int j = i + 1; j < n_; ++j)
        if ((b_[i].out || b_[j].out) && b_[i].lo < b_[j].hi && b_[j].lo < b_[i].hi) return false;
    return true;
  }

 private:
  struct One { uintptr_t lo, hi; bool out; };
  void add(const void* p, uint64_t bytes, uint64_t align, bool required, bool out) {
    if (!p) {
      bad_ = bad_ || required;
      return;
    }
    if (!aligned(p, align) || n_ == kMax) {
      bad_ = true;
      return;
    }
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    b_[n_++] = {lo, lo + bytes, out};
  }
  static constexpr int kMax = 24;
  One b_[kMax];
  int n_ = 0;
  bool bad_ = false;
};

}  // namespace seq
}  // namespace cnhwc
