// Whether the arrays of a call share memory (internal, on the host): an array
// that a call writes must lie apart from its others, and no two of its own
// elements in one place.
#pragma once

#include <cstddef>
#include <cstdint>

namespace sv {

// Runs of `run` bytes, st[d] bytes apart along each of up to three axes.
struct Span {
  long at = 0, size = 0, run = 0;  // first byte; from there to the last one's end; run 0: no array
  int dims = 0;
  long n[3], st[3];                // strides above 0, the largest first
  bool repeats = false;            // an axis whose elements are all one
};

// No memory is as long as this: a larger stride counts as it, so that no sum overflows.
constexpr long kFar = 1l << 42;

inline Span dense(const void* p, long bytes) {
  Span s;
  if (p) {
    s.at = (long)reinterpret_cast<uintptr_t>(p);
    s.size = s.run = bytes;
  }
  return s;
}

// [n0, n1, n2, run] of `elem` bytes each, strides in elements.
inline Span strided(const void* p, const int64_t* st, long n0, long n1, long n2, long run, int elem) {
  Span s = dense(p, run * elem);
  const long n[3] = {n0, n1, n2};
  for (int d = 0; p && d < 3; ++d) {
    if (n[d] <= 1) continue;
    const long far = kFar / elem, step = (st[d] < 0 ? st[d] < -far ? far : -st[d] : st[d] > far ? far : st[d]) * elem;
    if (step == 0) {
      s.repeats = true;
      continue;
    }
    if (st[d] < 0) s.at -= (n[d] - 1) * step;
    s.size += (n[d] - 1) * step;
    int i = s.dims++;
    for (; i > 0 && s.st[i - 1] < step; --i) s.st[i] = s.st[i - 1], s.n[i] = s.n[i - 1];
    s.st[i] = step;
    s.n[i] = n[d];
  }
  return s;
}

// A stride and how often it may be taken.
struct Steps {
  long st, lo, hi;
};

inline long floor_div(long a, long b) { return a / b - (a % b < 0); }

// Whether gap + sum of c_i st_i comes into [lo, hi] for whole c_i of their
// ranges.  The strides fall, so where axes nest (a row's bytes lie inside the
// stride of the axis above) one or two c_i of each are tried.  `left` bounds the
// search: what it does not settle counts as reached.
inline bool reaches(const Steps* t, int n, long gap, long lo, long hi, int* left) {
  if (--*left < 0) return true;
  if (n == 0) return lo <= gap && gap <= hi;
  long least = 0, most = 0;  // of the smaller strides
  for (int i = 1; i < n; ++i) least += t[i].lo * t[i].st, most += t[i].hi * t[i].st;
  long c0 = -floor_div(gap + most - lo, t->st), c1 = floor_div(hi - gap - least, t->st);
  if (c0 < t->lo) c0 = t->lo;
  if (c1 > t->hi) c1 = t->hi;
  if (n == 1) return c0 <= c1;
  for (long c = c0; c <= c1; ++c)
    if (reaches(t + 1, n - 1, gap + c * t->st, lo, hi, left)) return true;
  return false;
}

constexpr int kSearch = 1 << 16;

inline bool meet(const Span& a, const Span& b) {
  if (!a.run || !b.run || a.at >= b.at + b.size || b.at >= a.at + a.size) return false;
  Steps t[6];
  int n = 0;
  // b's runs less a's, equal strides as one
  for (int i = 0, j = 0; i < a.dims || j < b.dims; ++n) {
    const long x = i < a.dims ? a.st[i] : 0, y = j < b.dims ? b.st[j] : 0;
    t[n] = Steps{x > y ? x : y, 0, 0};
    for (; i < a.dims && a.st[i] == t[n].st; ++i) t[n].lo -= a.n[i] - 1;
    for (; j < b.dims && b.st[j] == t[n].st; ++j) t[n].hi += b.n[j] - 1;
  }
  int left = kSearch;
  return reaches(t, n, b.at - a.at, 1 - b.run, a.run - 1, &left);
}

// Whether two of an array's own elements lie in one place.
inline bool folds(const Span& a) {
  if (!a.run) return false;
  if (a.repeats) return true;
  long inner = a.run;  // bytes that a step along the next axis has to pass
  int d = a.dims;
  for (; d > 0 && a.st[d - 1] >= inner; --d) inner += (a.n[d - 1] - 1) * a.st[d - 1];
  if (d == 0) return false;
  for (int top = 0; top < a.dims; ++top) {  // the first axis along which they differ
    Steps t[3];
    for (int i = top; i < a.dims; ++i) t[i] = Steps{a.st[i], i == top ? 1l : 1 - a.n[i], a.n[i] - 1};
    int left = kSearch;
    if (reaches(t + top, a.dims - top, 0, 1 - a.run, a.run - 1, &left)) return true;
  }
  return false;
}

inline bool same(const Span& a, const Span& b) {
  bool r = a.at == b.at && a.size == b.size && a.run == b.run && a.dims == b.dims && a.repeats == b.repeats;
  for (int d = 0; r && d < a.dims; ++d) r = a.st[d] == b.st[d] && a.n[d] == b.n[d];
  return r;
}

// The arrays of one call.
class Arrays {
 public:
  int read(const Span& x) { return add(x, false, -1); }
  // `in`: the array that it may be, in place.
  int write(const Span& x, int in = -1) { return add(x, true, in); }
  // Whether what is written lies apart from all else.
  bool apart() const {
    for (int i = 0; i < n_; ++i) {
      if (!written_[i]) continue;
      if (folds(x_[i])) return false;
      for (int j = 0; j < n_; ++j)
        if (j != i && (j < i || !written_[j]) && !(in_[i] == j && same(x_[i], x_[j])) && meet(x_[i], x_[j])) return false;
    }
    return true;
  }

 private:
  int add(const Span& x, bool written, int in) {
    x_[n_] = x;
    written_[n_] = written;
    in_[n_] = in;
    return n_++;
  }
  Span x_[16];
  bool written_[16];
  int in_[16];
  int n_ = 0;
};

}  // namespace sv
