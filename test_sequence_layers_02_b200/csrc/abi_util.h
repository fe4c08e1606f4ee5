// Argument checks shared by the C-ABI entry points (host code only).
#pragma once

#include <cstddef>
#include <cstdint>

namespace ttt {
namespace abi {

inline bool misaligned(const void* p) {
  return p && (reinterpret_cast<uintptr_t>(p) & 15u) != 0;
}

// Is p off an `align`-byte boundary (a power of two)?
inline bool misaligned_to(const void* p, size_t align) {
  return p && (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0;
}

// Do the byte ranges [a, a + na) and [b, b + nb) intersect? (null or empty: no)
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

struct Span {
  const void* p;
  size_t n;
};

// Does any output meet an input or another output?
template <int NI, int NO>
bool any_overlap(const Span (&in)[NI], const Span (&out)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlaps(out[i].p, out[i].n, in[j].p, in[j].n)) return true;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
  }
  return false;
}

// A strided tensor: up to three outer dimensions (sizes n, element strides s)
// of contiguous rows of `row` elements of `elt` bytes.
struct Strided {
  long long n[3], s[3];
  long long row;
  size_t elt;

  bool empty() const { return n[0] * n[1] * n[2] * row == 0; }

  // Bytes from the first to behind the last element.
  size_t extent() const {
    if (empty()) return 0;
    long long last = row - 1;
    for (int i = 0; i < 3; ++i) last += (n[i] - 1) * s[i];
    return (size_t)(last + 1) * elt;
  }

  bool negative() const { return s[0] < 0 || s[1] < 0 || s[2] < 0; }

  // Could two of its elements share an address? (Outputs may not.) Dimensions
  // taken from the smallest stride up, each has to step over the one before.
  bool self_overlap() const {
    if (empty()) return false;
    int o[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (s[o[j]] > s[o[j + 1]]) { const int t = o[j]; o[j] = o[j + 1]; o[j + 1] = t; }
    long long span = row;
    for (int i = 0; i < 3; ++i) {
      if (n[o[i]] <= 1) continue;
      if (s[o[i]] < span) return true;
      span += (n[o[i]] - 1) * s[o[i]];
    }
    return false;
  }

  // Are the strides whole multiples of `by` elements?
  bool multiple_of(long long by) const {
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && s[i] % by != 0) return false;
    return true;
  }
};

}  // namespace abi
}  // namespace ttt
