// rows.h -- host checks of the tensors that rotary and cache calls read and write by strides:
// whether an output shares an element with another tensor of the call, and whether its own
// rows lie apart.
#pragma once

#include <algorithm>
#include <cstdint>

#include "common.cuh"

namespace sdpa {

// The rows of a rotary call's tensor: places in elements, dimensions batch, head, position.
struct RopeRows {
  long long base, end;  // first element, and one past the last
  long long st[3];
  int ext[3], D;
};
inline RopeRows rope_rows(const void* ptr, const long long* st, int B, int H, int S, int D) {
  RopeRows r{(long long)(reinterpret_cast<uintptr_t>(ptr) / 2), 0, {st[0], st[1], st[2]}, {B, H, S}, D};
  r.end = r.base + D;
  for (int j = 0; j < 3; ++j)
    if (r.ext[j] > 1) r.end += st[j] * (r.ext[j] - 1);
  return r;
}
inline bool same_rows(const RopeRows& a, const RopeRows& b) {
  bool same = a.base == b.base;
  for (int j = 0; j < 3; ++j) same = same && a.ext[j] == b.ext[j] && (a.ext[j] == 1 || a.st[j] == b.st[j]);
  return same;
}
// Whether rows `delta` apart come within D of one another by up to `back[j]` steps back and
// `on[j]` steps on of the strides st, descending: of each only those few are tried that the smaller
// ones can make up for.
inline bool steps_meet(const long long* st, const int* back, const int* on, int n, long long D, long long delta) {
  if (n == 0) return delta < D && -delta < D;
  long long reach = D;
  for (int j = 1; j < n; ++j) reach += st[j] * std::max(back[j], on[j]);
  const long long lo = std::max(floor_div(-delta - reach, st[0]), -(long long)back[0]);
  const long long hi = std::min(floor_div(reach - delta, st[0]) + 1, (long long)on[0]);
  for (long long k = lo; k <= hi; ++k)
    if (steps_meet(st + 1, back + 1, on + 1, n - 1, D, delta + k * st[0])) return true;
  return false;
}
// Whether an output y shares an element with x: exact for tensors that step alike (slices of
// one projection), and taken to be so for others whose places interleave.
inline bool rows_meet(const RopeRows& x, const RopeRows& y) {
  if (x.end <= y.base || y.end <= x.base) return false;
  long long st[3];
  int back[3], on[3], n = 0;
  for (int j = 0; j < 3; ++j) {
    if (x.ext[j] == 1 && y.ext[j] == 1) continue;
    if (x.ext[j] > 1 && y.ext[j] > 1 && x.st[j] != y.st[j]) return true;
    const long long s = y.ext[j] > 1 ? y.st[j] : x.st[j];
    if (s <= 0) return true;
    int at = n++;
    for (; at > 0 && st[at - 1] < s; --at) st[at] = st[at - 1], back[at] = back[at - 1], on[at] = on[at - 1];
    st[at] = s;
    back[at] = x.ext[j] - 1;
    on[at] = y.ext[j] - 1;
  }
  return steps_meet(st, back, on, n, x.D, y.base - x.base);
}

// Whether output rows of D elements, ext[j] steps of st[j], lie apart: taken by ascending
// stride, each dimension has to step over everything that the smaller ones span.
inline bool rows_apart(const long long (&st)[3], int B, int H, int S, int D) {
  long long span = D, ext[3] = {B, H, S};
  for (int pass = 0; pass < 3; ++pass) {
    int low = -1;
    for (int j = 0; j < 3; ++j)
      if (ext[j] > 1 && (low < 0 || st[j] < st[low])) low = j;
    if (low < 0) break;
    if (st[low] < span || st[low] > (1ll << 40)) return false;
    span += st[low] * (ext[low] - 1);
    ext[low] = 1;
  }
  return true;
}

}  // namespace sdpa
