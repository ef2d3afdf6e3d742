// ts_overlap.h -- whether arrays of a call share memory, as far as their addresses and
// strides say (host only, no CUDA).
#pragma once

#include <algorithm>
#include <cstdint>

namespace ts_host {

// The bytes of an array of rows (none for NULL).
struct Span {
  uintptr_t from, to;     // of the first element, behind the last
  uintptr_t pitch, wide;  // from row to row (0: one row), and of a row
  // Whether two arrays share bytes.  Columns of one buffer side by side do not; arrays
  // of different pitch that lie within one another count as if they did.
  bool meets(const Span &o) const {
    if (from >= o.to || o.from >= to) return false;
    if (!pitch || pitch != o.pitch) return true;
    const uintptr_t shift = (o.from >= from ? o.from - from : pitch - (from - o.from) % pitch) % pitch;
    return shift < wide || shift + o.wide > pitch;
  }
};
inline Span rows_span(const void *p, int64_t rows, int64_t dim, int64_t stride, int64_t es) {
  if (!p || rows < 1) return {0, 0, 0, 0};
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const uintptr_t pitch = rows > 1 ? static_cast<uintptr_t>(stride * es) : 0, wide = static_cast<uintptr_t>(dim * es);
  return {at, at + static_cast<uintptr_t>(rows - 1) * pitch + wide, pitch, wide};
}

// Heads [rows][heads] of `wide` bytes at byte strides `row` and `head` (neither negative;
// that of an axis of one entry says nothing).
struct Heads {
  uintptr_t from;
  int64_t rows, heads, row, head, wide;

  static Heads of(const void *p, int64_t rows, int64_t heads, int64_t row, int64_t head, int64_t dim, int64_t es) {
    return {reinterpret_cast<uintptr_t>(p), p ? rows : 0, heads, row * es, head * es, dim * es};
  }
  bool none() const { return rows < 1 || heads < 1; }
  __int128 end() const {
    return static_cast<__int128>(from) + static_cast<__int128>(rows - 1) * row + static_cast<__int128>(heads - 1) * head + wide;
  }
  // Whether its heads lie on one another.  The larger stride has to hold all that lies
  // along the smaller one (others could interleave without sharing anything; they count
  // as if they did).
  bool meets_itself() const {
    if (none()) return false;
    struct { int64_t count, stride; } axis[2] = {{rows, row}, {heads, head}};
    if (axis[0].count < 2 || (axis[1].count > 1 && axis[1].stride < axis[0].stride)) std::swap(axis[0], axis[1]);
    __int128 extent = wide;
    for (const auto &x : axis) {
      if (x.count < 2) continue;
      if (x.stride < extent) return true;
      extent += static_cast<__int128>(x.count - 1) * x.stride;
    }
    return false;
  }
  // Whether two arrays with heads of one width share bytes: exactly where they have the
  // same strides; else, columns of rows of one pitch side by side do not, and what lies
  // within one another counts as if it did.
  bool meets(const Heads &o) const {
    if (none() || o.none() || from >= o.end() || o.from >= end()) return false;
    const __int128 most = static_cast<__int128>(1) << 60;
    if (end() - from > most || o.end() - o.from > most) return true;
    const bool many_rows = rows > 1 && o.rows > 1, many_heads = heads > 1 && o.heads > 1;
    if (many_rows && row == o.row && row > 0 && !by_row().meets(o.by_row())) return false;
    if ((many_rows && row != o.row) || (many_heads && head != o.head) || wide != o.wide) return true;
    // rows i and heads j apart (of those that there are): nearer than a head's width?
    const int64_t step = rows > 1 ? row : o.rows > 1 ? o.row : 0, head_step = heads > 1 ? head : o.head;
    const int64_t apart = static_cast<int64_t>(o.from - from);
    for (int64_t j = 1 - heads; j < o.heads; ++j) {
      const int64_t at = apart + j * head_step;
      int64_t i = 0;
      if (step > 0) i = std::min(std::max((at < 0 ? step / 2 - at : -step / 2 - at) / step, 1 - rows), o.rows - 1);
      const int64_t off = at + i * step;
      if (off < wide && -off < wide) return true;
    }
    return false;
  }
  // Its rows, as far as all heads reach.
  Span by_row() const {
    return {from, static_cast<uintptr_t>(end()), static_cast<uintptr_t>(row), static_cast<uintptr_t>((heads - 1) * head + wide)};
  }
};

}  // namespace ts_host
