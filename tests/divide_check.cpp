// Host check of csrc/divide.h: prints "ok" if every quotient is that of a division.
#include <cstdint>
#include <cstdio>

#include "divide.h"

static bool check(int64_t d) {
  const sk::attn::Divide by(d);
  const int64_t most = (int64_t(1) << 31) - 1;
  auto one = [&](int64_t x) { return x < 0 || x > most || by((uint32_t)x) == (uint32_t)(x / (d < 1 ? 1 : d)); };
  for (int64_t x = 0; x < 3000; ++x)
    if (!one(x) || !one(most - x)) return false;
  // both sides of multiples, where a quotient changes
  for (int64_t k = 1; k < 3000; ++k)
    for (int64_t off = -1; off <= 1; ++off)
      if (!one(k * d + off) || !one(most / d * d - k * d + off)) return false;
  return true;
}

int main() {
  for (int64_t d = 1; d < 5000; ++d)
    if (!check(d)) return std::printf("wrong for %lld\n", (long long)d), 1;
  for (int l = 12; l < 31; ++l)
    for (int64_t off = -3; off <= 3; ++off)
      if (!check((int64_t(1) << l) + off)) return std::printf("wrong for 2^%d %+lld\n", l, (long long)off), 1;
  if (!check((int64_t(1) << 31) - 1)) return std::printf("wrong for 2^31 - 1\n"), 1;
  std::printf("ok\n");
  return 0;
}
