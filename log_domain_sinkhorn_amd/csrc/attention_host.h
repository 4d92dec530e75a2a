// What the C entry points of the attention operators and of the caches share on
// the host: errors, launch plans, workspaces.
#pragma once

#include <algorithm>

#include "attention.h"

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

inline int64_t elem_size(const sinkhorn_attention* a) { return a->dtype == SINKHORN_F32 ? 4 : 2; }

inline void check(const sinkhorn_attention* a) {
  require(a != nullptr, "null attention description");
  require(a->dtype == SINKHORN_F32 || a->dtype == SINKHORN_F16 || a->dtype == SINKHORN_BF16, "unknown dtype");
  require(a->batch >= 0 && a->len_q >= 0 && a->len_k >= 0, "negative size");
  require(a->heads_q >= 1 && a->heads_kv >= 1 && a->heads_q % a->heads_kv == 0,
          "heads_q must be a multiple of heads_kv");
  if (a->heads_q > 8192) fail(SINKHORN_ERR_UNSUPPORTED, "more than 8192 heads");
  require(a->d >= 1 && a->dv >= 1, "head widths must be >= 1");
  if (a->d > kMaxD || a->dv > kMaxD) fail(SINKHORN_ERR_UNSUPPORTED, "head widths above 128");
  require(a->len_q * (a->heads_q / a->heads_kv) < (int64_t(1) << 31) && a->len_q < (int64_t(1) << 31) &&
              a->len_k < (int64_t(1) << 31),
          "lengths must be below 2^31");
  require(std::isfinite(a->scale) && a->scale > 0.0 && std::isfinite((float)(a->scale * kLog2e)) &&
              (float)a->scale > 0.0f,
          "scale must be finite and > 0");
  for (int i = 0; i < 3; ++i)
    require(a->q_stride[i] >= 0 && a->k_stride[i] >= 0 && a->v_stride[i] >= 0 && a->out_stride[i] >= 0 &&
                a->dout_stride[i] >= 0 && a->dq_stride[i] >= 0 && a->dk_stride[i] >= 0 && a->dv_stride[i] >= 0,
            "negative stride");
  require(a->bias_stride[0] >= 0 && a->bias_stride[1] >= 0, "negative stride");
}

inline Shape make_shape(const sinkhorn_attention* a) {
  Shape S{};
  S.batch = a->batch;
  S.hq = a->heads_q;
  S.hkv = a->heads_kv;
  S.group = a->heads_q / a->heads_kv;
  S.d = a->d;
  S.dv = a->dv;
  S.lq = a->len_q;
  S.lk = a->len_k;
  S.rows = a->len_q * S.group;
  S.group_mul = S.group > 1 ? (uint32_t)(((uint64_t(1) << 32) + S.group - 1) / S.group) : 0;
  for (int i = 0; i < 3; ++i) {
    S.qs[i] = a->q_stride[i];
    S.ks[i] = a->k_stride[i];
    S.vs[i] = a->v_stride[i];
  }
  S.bias = a->key_bias;
  S.bs[0] = a->bias_stride[0];
  S.bs[1] = a->bias_stride[1];
  S.qlen = a->query_lengths;
  S.klen = a->key_lengths;
  S.scale = (float)a->scale;
  S.scale_lo = (float)(a->scale - (double)S.scale);
  S.c = (float)(a->scale * kLog2e);
  return S;
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
