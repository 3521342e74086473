// Host-side description of strided tensors and exact overlap tests, shared by
// the operators that take strides.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace mbd_host {

// Three strided dimensions (element strides) over dense runs of `run` elements.
struct Region {
  uintptr_t p;
  int64_t bytes;      // of one element
  int64_t n[3], s[3];
  int64_t run;

  bool empty() const { return !p || run <= 0 || n[0] <= 0 || n[1] <= 0 || n[2] <= 0; }
  int64_t span() const {   // bytes from the first to behind the last element
    int64_t e = run;
    for (int i = 0; i < 3; ++i) e += (n[i] - 1) * s[i];
    return e * bytes;
  }
};

inline Region dense_region(const void* p, int64_t elements, int64_t bytes) {
  return Region{(uintptr_t)p, bytes, {1, 1, 1}, {0, 0, 0}, elements};
}

// Whether a region's own elements are all different: each stride, from the
// smallest up, steps over everything below it.
inline bool distinct(const Region& r) {
  int64_t n[3], s[3];
  int m = 0;
  for (int i = 0; i < 3; ++i)
    if (r.n[i] > 1) {
      n[m] = r.n[i];
      s[m++] = r.s[i];
    }
  for (int i = 0; i < m; ++i)
    for (int j = i + 1; j < m; ++j)
      if (s[j] < s[i]) {
        std::swap(s[i], s[j]);
        std::swap(n[i], n[j]);
      }
  int64_t below = r.run;
  for (int i = 0; i < m; ++i) {
    if (s[i] < below) return false;
    below += (n[i] - 1) * s[i];
  }
  return true;
}

// delta = sum_i x_i s_i + c for some |x_i| < n_i and -lo < c < hi, over
// dimensions in descending order of stride.
inline bool reachable(int64_t delta, const int64_t* n, const int64_t* s, int m, int64_t lo, int64_t hi) {
  if (m == 0) return delta > -lo && delta < hi;
  if (s[0] <= 0) return reachable(delta, n + 1, s + 1, m - 1, lo, hi);
  int64_t rest = std::max(lo, hi);
  for (int i = 1; i < m; ++i) rest += (n[i] - 1) * s[i];
  int64_t a = (delta - rest) / s[0] - 1, b = (delta + rest) / s[0] + 1;
  a = std::max(a, -(n[0] - 1));
  b = std::min(b, n[0] - 1);
  for (int64_t i = a; i <= b; ++i)
    if (reachable(delta - i * s[0], n + 1, s + 1, m - 1, lo, hi)) return true;
  return false;
}

// Whether two regions share memory: exact for regions of the same strides and
// element size (slices of one tensor), by their spans otherwise.
inline bool share(const Region& x, const Region& y) {
  if (x.empty() || y.empty()) return false;
  if (!(x.p < y.p + (uintptr_t)y.span() && y.p < x.p + (uintptr_t)x.span())) return false;
  const int64_t d = (int64_t)(y.p - x.p);
  bool same = x.bytes == y.bytes && d % x.bytes == 0 && distinct(x) && distinct(y);
  for (int i = 0; i < 3; ++i) same = same && x.n[i] == y.n[i] && (x.s[i] == y.s[i] || x.n[i] == 1);
  if (!same) return true;
  int64_t n[3] = {x.n[0], x.n[1], x.n[2]}, s[3] = {x.s[0], x.s[1], x.s[2]};
  for (int i = 0; i < 3; ++i)
    if (n[i] == 1) s[i] = 0;
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (s[j] > s[i]) {
        std::swap(s[i], s[j]);
        std::swap(n[i], n[j]);
      }
  // y's element = x's element:  d / bytes = (lattice difference) + (x's channel - y's channel)
  return reachable(d / x.bytes, n, s, 3, y.run, x.run);
}

}  // namespace mbd_host
