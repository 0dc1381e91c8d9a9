// Argument checks that the C entries of the token and trunk operators share.
#pragma once
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <utility>

#include "../../include/cbr.h"

namespace cbr {

// Row counts and strides up to 2^40, and an axis' steps times its stride up to 2^58 elements: a tensor's
// axes together stay within 2^62 bytes.
constexpr int64_t kMaxExtent = int64_t(1) << 40, kMaxReach = int64_t(1) << 58;

inline bool known_dtype(int32_t t) { return t == CBR_F16 || t == CBR_BF16 || t == CBR_F32; }
inline size_t elt(int32_t t) { return t == CBR_F32 ? 4 : 2; }
inline bool off(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }
inline bool extent(int64_t v) { return v >= 0 && v <= kMaxExtent; }
inline bool finite(float v) { return std::isfinite(v); }

inline bool in_reach(int64_t stride, int64_t steps) { return steps <= 1 || stride <= kMaxReach / (steps - 1); }

// A row stride: at least the row (any value will do where there is one row at most).
inline bool row_stride(int64_t s, int64_t width, int64_t rows) {
  return extent(s) && (rows <= 1 || s >= width) && in_reach(s, rows);
}

// An output that is an input must be it exactly.
inline bool same_or_apart(const void* out, int64_t out_stride, const void* in, int64_t in_stride, int64_t rows) {
  return out != in || !in || rows <= 1 || out_stride == in_stride;
}

// The heads of an output [batch][tokens][heads][width] must not share memory: taken by their strides, each
// axis of several steps steps past all that the smaller ones reach.
inline bool distinct(const int64_t* s, int64_t batch, int64_t tokens, int64_t heads, int64_t width) {
  std::pair<int64_t, int64_t> axes[3] = {{s[0], batch}, {s[1], tokens}, {s[2], heads}};   // stride, steps
  std::sort(axes, axes + 3);
  int64_t reach = width;
  for (const auto& [stride, steps] : axes) {
    if (steps <= 1) continue;
    if (stride < reach) return false;
    reach += stride * (steps - 1);
  }
  return true;
}

inline bool same(const int64_t* a, const int64_t* b) { return a[0] == b[0] && a[1] == b[1] && a[2] == b[2]; }

}  // namespace cbr
