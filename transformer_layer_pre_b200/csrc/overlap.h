// overlap.h — whether two strided tensors share memory (host side).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace tlp {

// Rows of `width` contiguous bytes at `at` plus any sum of i * stride (bytes),
// 0 <= i < count, over its dimensions: strides positive, largest first.
struct ByteRows {
  int64_t at, width;
  int dims;
  struct Dim { int64_t stride, count; } dim[3];

  ByteRows(const void* p, int64_t bytes) : at((int64_t) reinterpret_cast<uintptr_t>(p)), width(bytes), dims(0) {}

  // (batch, token, head, head_dim) entries of es bytes by element strides
  ByteRows(const void* p, int64_t sb, int B, int64_t st, int S, int64_t sh, int nh, int d, int es)
      : ByteRows(p, (int64_t)d * es) {
    // the stride of a dimension of one entry means nothing and may hold anything
    Dim x[3] = {{B > 1 ? sb * es : 0, B}, {S > 1 ? st * es : 0, S}, {nh > 1 ? sh * es : 0, nh}};
    std::sort(x, x + 3, [](const Dim& l, const Dim& r) { return l.stride < r.stride; });
    for (const Dim& e : x) {
      if (e.count == 1) continue;
      if (dims == 0 && e.stride == width) width *= e.count;   // rows that touch are one
      else dim[dims++] = e;
    }
    std::reverse(dim, dim + dims);
  }
  int64_t span(int from) const {
    int64_t s = width;
    for (int k = from; k < dims; ++k) s += dim[k].stride * (dim[k].count - 1);
    return s;
  }
};

// Whether a byte of x from its dimension kx on, moved to ax, is one of y from ky
// on, moved to ay.  Exact: a dimension is split into its entries, of which only
// those within the other tensor's span are looked at, and two of the same
// stride into the distances between their entries, so that views of one packed
// buffer take a few steps each.  Tensors of different strides that lie within
// one another take up to a step per row; `left` bounds the steps, after which
// they count as overlapping.
inline bool meet(const ByteRows& x, int kx, int64_t ax, const ByteRows& y, int ky, int64_t ay, int& left) {
  if (ax >= ay + y.span(ky) || ay >= ax + x.span(kx)) return false;
  if ((kx == x.dims && ky == y.dims) || --left <= 0) return true;
  auto down = [](int64_t a, int64_t b) { return a >= 0 ? a / b : -((-a + b - 1) / b); };   // floor(a / b)
  const int64_t sx = kx < x.dims ? x.dim[kx].stride : 0, sy = ky < y.dims ? y.dim[ky].stride : 0;
  if (sx == sy) {
    // entry i of x against entry j of y: distance i - j
    const int64_t lo = std::max(1 - y.dim[ky].count, down(ay - ax - x.span(kx + 1), sx) + 1);
    const int64_t hi = std::min(x.dim[kx].count - 1, down(ay + y.span(ky + 1) - ax - 1, sx));
    for (int64_t i = lo; i <= hi; ++i)
      if (meet(x, kx + 1, ax + i * sx, y, ky + 1, ay, left)) return true;
  } else if (sx > sy) {
    const int64_t lo = std::max<int64_t>(0, down(ay - ax - x.span(kx + 1), sx) + 1);
    const int64_t hi = std::min(x.dim[kx].count - 1, down(ay + y.span(ky) - ax - 1, sx));
    for (int64_t i = lo; i <= hi; ++i)
      if (meet(x, kx + 1, ax + i * sx, y, ky, ay, left)) return true;
  } else {
    return meet(y, ky, ay, x, kx, ax, left);
  }
  return false;
}

inline bool overlap(const ByteRows& x, const ByteRows& y) {
  int left = 1 << 16;
  return meet(x, 0, x.at, y, 0, y.at, left);
}

}  // namespace tlp
