// Host-only driver for overlap.h: reads lines of two arrays, each "at step0 step1
// step2 count0 count1 count2 width", and prints 1 where they share a byte.
#include <cstdio>

#include "overlap.h"

static bool read(sk::Span& s) {
  unsigned long long at;
  long long x[7];
  if (std::scanf("%llu", &at) != 1) return false;
  for (long long& v : x)
    if (std::scanf("%lld", &v) != 1) return false;
  s.at = (uintptr_t)at;
  for (int i = 0; i < 3; ++i) {
    s.step[i] = x[i];
    s.count[i] = x[3 + i];
  }
  s.width = x[6];
  return true;
}

int main() {
  sk::Span a(nullptr, 0), b(nullptr, 0);
  while (read(a) && read(b)) std::printf("%d\n", sk::Meeting::of(a, b) ? 1 : 0);
  return 0;
}
