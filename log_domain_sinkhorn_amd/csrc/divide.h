// Division by a number that a launch fixes. The host part is free of HIP so that the
// tests can check it with a plain C++ compiler.
#pragma once

#include <cstdint>

#ifndef __HIP__
#define SK_HOST_DEVICE
#else
#define SK_HOST_DEVICE __host__ __device__
#endif

namespace sk {
namespace attn {

// x / d for 0 <= x < 2^31 by a product: with 2^(l - 1) < d <= 2^l, mul = floor(2^(31 + l)
// / d) + 1 exceeds 2^(31 + l) / d by at most 1, which moves x mul / 2^(31 + l) by less
// than 1 / d, too little to pass the next whole number. (A division takes about 30
// instructions, in 64 bits 130.)
struct Divide {
  uint32_t mul = 0, shift = 0;  // mul 0: by 1

  Divide() = default;
  explicit Divide(int64_t d) {
    if (d <= 1) return;
    int l = 1;
    while ((int64_t(1) << l) < d) ++l;
    mul = (uint32_t)((uint64_t(1) << (31 + l)) / (uint64_t)d + 1);
    shift = (uint32_t)(l - 1);
  }
  SK_HOST_DEVICE uint32_t operator()(uint32_t x) const {
    return mul ? (uint32_t)(((uint64_t)x * mul) >> 32) >> shift : x;
  }
};

}  // namespace attn
}  // namespace sk
