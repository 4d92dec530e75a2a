// Do two strided arrays share a byte? Host arithmetic, free of HIP so that the
// tests can check it with a plain C++ compiler.
#pragma once

#include <algorithm>
#include <cstdint>
#include <initializer_list>

namespace sk {

// Runs of `width` bytes at at + sum of index * step, over three indices.
struct Span {
  uintptr_t at = 0;  // 0: no array
  int64_t step[3] = {0, 0, 0}, count[3] = {1, 1, 1}, width = 0;

  Span(const void* p, int64_t bytes) : at((uintptr_t)p), width(bytes) {}
  // stride: of three indices, in elements of `size` bytes
  Span(const void* p, const int64_t* stride, int64_t n0, int64_t n1, int64_t n2, int64_t elements, int64_t size)
      : at((uintptr_t)p), count{n0, n1, n2}, width(elements * size) {
    for (int i = 0; i < 3; ++i) step[i] = stride[i] * size;
  }
  bool empty() const { return at == 0 || width <= 0 || count[0] <= 0 || count[1] <= 0 || count[2] <= 0; }
  __int128 end() const {
    __int128 e = (__int128)at + width;
    for (int i = 0; i < 3; ++i) e += (__int128)step[i] * (count[i] - 1);
    return e;
  }
};

// Exact: a byte is shared where at_a + sum x_i s_i and at_b + sum y_i t_i differ
// by less than a run. The terms of one step are joined (all whole multiples in an
// interval) and the rest is searched from the largest step down, cutting off
// what the smaller terms can not reach; nested layouts of one buffer take a few
// nodes. Past kNodes of them (layouts that share no step, deep inside each
// other) the answer is "yes".
class Meeting {
 public:
  static bool of(const Span& a, const Span& b) {
    if (a.empty() || b.empty() || a.end() <= (Wide)b.at || b.end() <= (Wide)a.at) return false;
    Meeting m;
    for (int i = 0; i < 3; ++i) {
      m.add(a.step[i], 0, a.count[i] - 1);
      m.add(b.step[i], 1 - b.count[i], 0);
    }
    std::sort(m.terms, m.terms + m.n, [](const Term& x, const Term& y) { return x.step > y.step; });
    m.under = -(Wide)a.width;
    m.over = b.width;
    return m.reach(0, (Wide)a.at - (Wide)b.at);
  }

 private:
  typedef __int128 Wide;
  struct Term {
    int64_t step, lo, hi;
  };
  static constexpr int kNodes = 4096;
  Term terms[6];
  int n = 0, nodes = 0;
  Wide under, over;  // a difference of a's and b's run between these: they share a byte

  void add(int64_t step, int64_t lo, int64_t hi) {
    if (step == 0 || lo == hi) return;
    for (int i = 0; i < n; ++i)
      if (terms[i].step == step) {
        terms[i].lo += lo;
        terms[i].hi += hi;
        return;
      }
    terms[n++] = Term{step, lo, hi};
  }
  static Wide floor_div(Wide x, Wide y) { return x >= 0 ? x / y : -((-x + y - 1) / y); }
  bool reach(int i, Wide v) {
    if (++nodes > kNodes) return true;
    if (i == n) return v > under && v < over;
    Wide least = 0, most = 0;  // of the terms behind this one
    for (int k = i + 1; k < n; ++k) {
      least += (Wide)terms[k].step * terms[k].lo;
      most += (Wide)terms[k].step * terms[k].hi;
    }
    const Wide s = terms[i].step;
    // under < v + z s + most and v + z s + least < over
    const Wide lo = std::max<Wide>(terms[i].lo, floor_div(under - v - most, s) + 1);
    const Wide hi = std::min<Wide>(terms[i].hi, -floor_div(-(over - v - least), s) - 1);
    for (Wide z = lo; z <= hi; ++z)
      if (reach(i + 1, v + z * s)) return true;
    return false;
  }
};

// Does an array that a call writes share a byte with one that it reads, or with
// another that it writes? Arrays whose ranges are apart, as nearly all are, cost
// two compares a pair. At most 16 arrays.
inline bool any_meet(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  struct Range {
    const Span* s;
    __int128 from, end;
  } all[16];
  int n = 0, outputs = 0;
  auto add = [&](const Span& s) {
    if (!s.empty()) all[n++] = Range{&s, (__int128)s.at, s.end()};
  };
  for (const Span& s : written) add(s);
  outputs = n;
  for (const Span& s : read) add(s);
  for (int i = 0; i < outputs; ++i)
    for (int k = i + 1; k < n; ++k)
      if (all[i].from < all[k].end && all[k].from < all[i].end && Meeting::of(*all[i].s, *all[k].s)) return true;
  return false;
}

}  // namespace sk
