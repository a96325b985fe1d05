// Whether arrays with strides share memory: host code, for the calls whose result may not lie over an operand.
#pragma once
#include <algorithm>

namespace tileq {

// Memory of an array: mats matrices, stride bytes apart, of rows of `width` bytes, ld bytes apart (none where rows is 0).
struct Memory {
  const void *base;
  long long width, rows = 1, ld = 0, mats = 1, stride = 0;
  long long matrix() const { return (rows - 1) * ld + width; }
  long long bytes() const { return (mats - 1) * stride + matrix(); }
};
inline long long div_down(long long v, long long m) { return v >= 0 ? v / m : -((-v + m - 1) / m); }

// Do bytes [lo, hi), counted from m's base, hold any of m's?
inline bool touches(const Memory &m, long long lo, long long hi) {
  // the first matrix and row that end behind lo
  const long long first = m.mats > 1 ? std::max(div_down(lo - m.matrix(), m.stride) + 1, 0ll) : 0;
  for (long long i = first; i < m.mats && i * m.stride < hi; ++i) {
    const long long l = lo - i * m.stride, h = hi - i * m.stride;
    const long long row = m.rows > 1 ? std::max(div_down(l - m.width, m.ld) + 1, 0ll) : 0;
    if (row < m.rows && row * m.ld < h && row * m.ld + m.width > l) return true;
  }
  return false;
}

// Do two arrays share a byte?  Exactly: columns of the same rows (a gate beside its up projection) are not shared.
inline bool share(Memory a, Memory b) {
  if (!a.base || !b.base || !a.rows || !b.rows) return false;
  for (Memory *m : {&a, &b})  // matrices in one piece are one
    if (m->mats > 1 && m->stride == m->rows * m->ld) m->rows *= m->mats, m->mats = 1;
  const long long d = static_cast<const char *>(b.base) - static_cast<const char *>(a.base);
  if (d >= a.bytes() || -d >= b.bytes()) return false;
  if (a.mats == 1 && b.mats == 1 && a.rows > 1 && b.rows > 1 && a.ld == b.ld) {
    const long long at = d - div_down(d, a.ld) * a.ld;  // where b's rows start in a's
    return at < a.width || at + b.width > a.ld;
  }
  // rows of other lengths between each other: one by one, of the array that has fewer
  const bool swap = b.mats * b.rows < a.mats * a.rows;
  const Memory &few = swap ? b : a, &many = swap ? a : b;
  const long long off = swap ? d : -d;  // few's base from many's
  for (long long i = 0; i < few.mats; ++i)
    for (long long r = 0; r < few.rows; ++r) {
      const long long lo = off + i * few.stride + r * few.ld;
      if (touches(many, lo, lo + few.width)) return true;
    }
  return false;
}

}  // namespace tileq
