// What the C entry points of the attention operators and of the caches share on
// the host: errors, launch plans, workspaces.
#pragma once

#include <algorithm>

#include "internal.h"

namespace sk {
namespace attn {

template <class F>
int guarded(F&& body) {
  try {
    set_last_error("");
    return body();
  } catch (const Failure& f) {
    set_last_error(f.msg);
    return f.code;
  } catch (...) {
    set_last_error("unexpected exception");
    return SINKHORN_ERR_HIP;
  }
}

inline void require(bool ok, const char* what) {
  if (!ok) fail(SINKHORN_ERR_INVALID_ARG, what);
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Splits of the streamed side, `steps` tiles of it, for `blocks` workgroups of
// which about `slots` run at a time (the chip holds more at up to 64 16-bit
// columns, and fewer of the weight's own pass in fp32 above 64): the number with
// the least time in units of one step, counting rounds of workgroups, two steps to
// begin and end each, and the join (`join` steps and a little per split: a join
// takes 4 to 7 us, a step of 64 keys at 128 rows about 2 in 16-bit types and 6 in
// fp32, of few rows about 1). `fine`: at least four rounds, so that sequences of
// different lengths even out.
inline int32_t splits(int64_t blocks, int64_t steps, int64_t slots, double join, bool fine) {
  if (blocks <= 0 || steps <= 1 || blocks >= 4 * slots) return 1;
  const int64_t most = std::min<int64_t>(steps, 512);
  int32_t best = 1;
  double least = 0.0;
  for (int64_t n = 1; n <= most; ++n) {
    const double rounds = (double)ceil_div(blocks * n, slots);
    const double cost = rounds * (double)(ceil_div(steps, n) + 2) + (n > 1 ? join + 0.02 * (double)n : 0.0);
    if (n == 1 || cost < least) {
      least = cost;
      best = (int32_t)n;
    }
  }
  if (fine && best > 1) {
    const int64_t n = std::min<int64_t>(ceil_div(4 * slots, blocks), std::max<int64_t>(1, steps / 8));
    if (n > best) best = (int32_t)n;
  }
  return best;
}

// Workspace layout: consecutive pieces of 256-byte multiples.
struct Space {
  int64_t bytes = 0;
  int64_t take(int64_t n) {
    const int64_t at = bytes;
    bytes += ceil_div(n, 256) * 256;
    return at;
  }
};

}  // namespace attn
}  // namespace sk
