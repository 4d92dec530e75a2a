// C ABI of the rotary positions and of appending to a paged cache: argument
// checks and launch plans. The kernels are in rotate.h, instantiated per element
// type.
#include <initializer_list>

#include "overlap.h"
#include "pages.h"
#include "rotate.h"

namespace sk {
namespace attn {

extern template void rotate<__bf16>(RotateArgs&, int, hipStream_t);
extern template void rotate<_Float16>(RotateArgs&, int, hipStream_t);
extern template void rotate<float>(RotateArgs&, int, hipStream_t);
extern template void rotate_grad<__bf16>(RotateArgs&, int, int32_t, hipStream_t);
extern template void rotate_grad<_Float16>(RotateArgs&, int, int, hipStream_t);
extern template void rotate_grad<float>(RotateArgs&, int, int, hipStream_t);

namespace {

// The weights' gradients from the workgroups' sums: one workgroup per tensor and four
// columns, thread t adding up rows t, t + 256, ...; then a tree over the threads.
__global__ __launch_bounds__(256) void k_weight_join(RotateArgs A, float* dq, float* dk) {
  __shared__ f32x4 s[256];
  const int which = blockIdx.x & 1, col = 4 * (blockIdx.x >> 1), tid = threadIdx.x;
  float* const out = which ? dk : dq;
  if (!out) return;
  f32x4 x = {0, 0, 0, 0};
  for (int n = (which ? A.part[0].end : 0) + tid; n < A.part[which].end; n += 256) {
    const f32x4 y = *(const f32x4*)(A.sums + (int64_t)n * kMaxD + col);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] += y[e];
  }
  s[tid] = x;
  for (int k = 128; k > 0; k >>= 1) {
    __syncthreads();
    if (tid < k)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[tid][e] += s[tid + k][e];
  }
  __syncthreads();
  if (tid < 4 && col + tid < A.d) out[col + tid] = s[0][tid];
}

int64_t elem_size(int32_t dtype) { return dtype == SINKHORN_F32 ? 4 : 2; }

void check(const sinkhorn_rotation* r) {
  require(r != nullptr, "null rotation description");
  require(r->dtype == SINKHORN_F32 || r->dtype == SINKHORN_F16 || r->dtype == SINKHORN_BF16, "unknown dtype");
  require(r->batch >= 0 && r->len >= 0, "negative size");
  require(r->heads_q >= 0 && r->heads_kv >= 0 && r->heads_q + (int64_t)r->heads_kv >= 1, "no heads");
  if (r->heads_q > 8192 || r->heads_kv > 8192) fail(SINKHORN_ERR_UNSUPPORTED, "more than 8192 heads");
  require(r->d >= 1, "head widths must be >= 1");
  if (r->d > kMaxD) fail(SINKHORN_ERR_UNSUPPORTED, "head widths above 128");
  require(r->rotated >= 0 && r->rotated <= r->d && r->rotated % 2 == 0, "rotated must be even and at most d");
  require(r->rotated == 0 || (std::isfinite(r->gain) && std::isfinite((float)r->gain)), "gain must be finite");
  require(!r->norm || (std::isfinite(r->eps) && std::isfinite((float)r->eps) && r->eps >= 0.0), "eps must be finite and >= 0");
  require(r->weight_dtype == SINKHORN_F32 || r->weight_dtype == r->dtype, "weights must be fp32 or of the tensors' type");
  require(r->batch * (__int128)r->len < (int64_t(1) << 31), "batch * len must be below 2^31");
  require(r->rotated == 0 || r->frequencies != nullptr, "null frequencies");
  for (int i = 0; i < 3; ++i)
    require(r->q_stride[i] >= 0 && r->k_stride[i] >= 0 && r->q_out_stride[i] >= 0 && r->k_out_stride[i] >= 0 &&
                r->dq_stride[i] >= 0 && r->dk_stride[i] >= 0,
            "negative stride");
  require(r->position_stride >= 0, "negative stride");
}

Span heads_of(const sinkhorn_rotation* r, const void* p, const int64_t* stride, int32_t heads, int32_t width) {
  return Span(p, stride, r->batch, r->len, heads, width, elem_size(r->dtype));
}
Span weight_of(const sinkhorn_rotation* r, const void* p) { return Span(p, r->d * elem_size(r->weight_dtype)); }
Span positions_of(const sinkhorn_rotation* r) {
  const int64_t stride[3] = {r->position_stride, 0, 0};
  return Span(r->positions, stride, r->batch, 1, 1, r->len, 4);
}
Span per_entry(const sinkhorn_rotation* r, const void* p) { return Span(p, 4 * (int64_t)r->batch); }
Span frequencies_of(const sinkhorn_rotation* r) { return Span(r->rotated ? r->frequencies : nullptr, 4 * (int64_t)r->rotated); }

// The array `out` is written in the places that `in` is read from.
bool in_place(const void* out, const int64_t* out_stride, const void* in, const int64_t* in_stride) {
  return out == in && out_stride[0] == in_stride[0] && out_stride[1] == in_stride[1] && out_stride[2] == in_stride[2];
}

void set(HeadRows& r, const void* src, const int64_t* ss, void* dst, const int64_t* ds, const void* weight, int32_t heads) {
  r.src = src;
  r.dst = dst;
  r.weight = weight;
  r.heads = heads;
  for (int i = 0; i < 3; ++i) {
    r.ss[i] = ss[i];
    r.ds[i] = ds[i];
  }
}

// The widest chunk that every array allows.
struct Unit {
  int64_t size;
  int e;
  explicit Unit(const sinkhorn_rotation* r) : size(elem_size(r->dtype)), e((int)(16 / elem_size(r->dtype))) {
    // both elements of a pair in a chunk, or in two chunks of one lane
    const int32_t turn = r->interleaved ? r->rotated : r->rotated / 2;
    while (r->d % e != 0 || turn % e != 0) e /= 2;
  }
  void fit(const void* p, const int64_t* stride, int32_t width) {
    while (e > 1 && !rows_aligned(p, stride, width, size, e * size)) e /= 2;
  }
};

RotateArgs arguments(const sinkhorn_rotation* r) {
  RotateArgs A{};
  A.batch = r->batch;
  A.len = A.steps = (int32_t)r->len;
  A.d = r->d;
  A.half = r->rotated / 2;
  A.interleaved = r->interleaved != 0;
  A.norm = r->norm != 0;
  A.weight_f32 = r->weight_dtype == SINKHORN_F32;
  A.gain = (float)r->gain;
  A.sign = 1.0f;
  A.eps = (float)r->eps;
  A.inv_d = 1.0f / (float)r->d;
  A.freq = r->frequencies;
  A.positions = r->positions;
  A.position_stride = r->position_stride;
  A.lengths = r->lengths;
  return A;
}

void run(const sinkhorn_rotation* r, RotateArgs& A, int e, hipStream_t st) {
  if (r->dtype == SINKHORN_BF16)
    rotate<__bf16>(A, e, st);
  else if (r->dtype == SINKHORN_F16)
    rotate<_Float16>(A, e, st);
  else
    rotate<float>(A, e, st);
}

// Workgroups of the backward pass with a norm: as many as the chip holds at a time,
// three a compute unit (16384 tokens x 40 heads of 128 bf16: 768 103 us, 1024 110, 1536
// 103; 8192 x 40 of 64 29.6, 32.6, 31.7), fewer where a wave would not find four heads;
// two at least, one for each tensor.
int32_t grad_blocks(const sinkhorn_rotation* r) {
  const int64_t n = ceil_div(r->batch * r->len * (r->heads_q + r->heads_kv), 16);
  return (int32_t)(n < 2 ? 2 : (n > 768 ? 768 : n));
}
int64_t grad_space(const sinkhorn_rotation* r) { return r->norm ? (int64_t)grad_blocks(r) * kMaxD * 4 : 0; }

}  // namespace
}  // namespace attn
}  // namespace sk

using namespace sk;
using namespace sk::attn;

extern "C" {

int sinkhorn_rotary_frequencies(int32_t rotated, double base, double factor, double original_length, double low,
                                double high, double* out) {
  return guarded([&] {
    require(rotated >= 0 && rotated % 2 == 0, "rotated must be even");
    require(out != nullptr || rotated == 0, "null pointer");
    require(std::isfinite(base) && base > 0.0 && std::isfinite(factor) && factor > 0.0, "base and factor must be finite and > 0");
    require(std::isfinite(original_length) && original_length >= 0.0, "original_length must be finite and >= 0");
    require(original_length == 0.0 || (std::isfinite(low) && std::isfinite(high) && low < high), "low must be below high");
    for (int32_t i = 0; i < rotated / 2; ++i) {
      const double f = std::pow(base, -2.0 * i / rotated);
      double keep = 0.0;  // the part that is not slowed down
      if (original_length > 0.0) {
        const double turns = original_length * f / 6.283185307179586477;
        keep = (turns - low) / (high - low);
        keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      }
      out[i] = f * (keep + (1.0 - keep) / factor);
    }
    return SINKHORN_OK;
  });
}

int sinkhorn_rotate_heads(const sinkhorn_rotation* r, const void* q, const void* k, const void* q_weight,
                          const void* k_weight, void* q_out, void* k_out, void* stream) {
  return guarded([&] {
    check(r);
    if (r->batch == 0 || r->len == 0) return SINKHORN_OK;
    require((r->heads_q == 0 || (q && q_out)) && (r->heads_kv == 0 || (k && k_out)), "null pointer");
    const bool qsame = in_place(q_out, r->q_out_stride, q, r->q_stride), ksame = in_place(k_out, r->k_out_stride, k, r->k_stride);
    require(!any_meet({heads_of(r, q_out, r->q_out_stride, r->heads_q, r->d), heads_of(r, k_out, r->k_out_stride, r->heads_kv, r->d)},
                      {heads_of(r, qsame ? nullptr : q, r->q_stride, r->heads_q, r->d),
                       heads_of(r, ksame ? nullptr : k, r->k_stride, r->heads_kv, r->d), weight_of(r, q_weight),
                       weight_of(r, k_weight), positions_of(r), per_entry(r, r->lengths), frequencies_of(r)}),
            "an output overlaps another argument");
    RotateArgs A = arguments(r);
    set(A.part[0], q, r->q_stride, q_out, r->q_out_stride, q_weight, r->heads_q);
    set(A.part[1], k, r->k_stride, k_out, r->k_out_stride, k_weight, r->heads_kv);
    Unit u(r);
    if (r->heads_q) u.fit(q, r->q_stride, r->d), u.fit(q_out, r->q_out_stride, r->d);
    if (r->heads_kv) u.fit(k, r->k_stride, r->d), u.fit(k_out, r->k_out_stride, r->d);
    run(r, A, u.e, (hipStream_t)stream);
    return SINKHORN_OK;
  });
}

int sinkhorn_rotation_workspace(const sinkhorn_rotation* r, int64_t* bytes) {
  return guarded([&] {
    check(r);
    require(bytes != nullptr, "null pointer");
    *bytes = grad_space(r);
    return SINKHORN_OK;
  });
}

int sinkhorn_rotate_heads_grad(const sinkhorn_rotation* r, const void* dq_out, const void* dk_out, const void* q,
                               const void* k, const void* q_weight, const void* k_weight, void* dq, void* dk,
                               float* dq_weight, float* dk_weight, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&] {
    check(r);
    const bool rows = r->batch > 0 && r->len > 0;
    require(r->norm || (!dq_weight && !dk_weight), "gradients of weights need a norm");
    require((dq_weight == nullptr || r->heads_q > 0) && (dk_weight == nullptr || r->heads_kv > 0),
            "a weight's gradient without its tensor");
    require(!rows || ((r->heads_q == 0 || (dq_out && dq && (q || !r->norm))) &&
                      (r->heads_kv == 0 || (dk_out && dk && (k || !r->norm)))),
            "null pointer");
    if (!r->norm && !rows) return SINKHORN_OK;
    const int64_t need = grad_space(r);
    require(need == 0 || (workspace != nullptr && workspace_bytes >= need), "workspace too small (sinkhorn_rotation_workspace)");
    require((uintptr_t)workspace % 16 == 0, "workspace must be 16-byte aligned");
    const bool qsame = in_place(dq, r->dq_stride, dq_out, r->q_out_stride), ksame = in_place(dk, r->dk_stride, dk_out, r->k_out_stride);
    require(!any_meet({heads_of(r, dq, r->dq_stride, r->heads_q, r->d), heads_of(r, dk, r->dk_stride, r->heads_kv, r->d),
                       Span(dq_weight, 4 * (int64_t)r->d), Span(dk_weight, 4 * (int64_t)r->d), Span(workspace, need)},
                      {heads_of(r, qsame ? nullptr : dq_out, r->q_out_stride, r->heads_q, r->d),
                       heads_of(r, ksame ? nullptr : dk_out, r->k_out_stride, r->heads_kv, r->d),
                       heads_of(r, r->norm ? q : nullptr, r->q_stride, r->heads_q, r->d),
                       heads_of(r, r->norm ? k : nullptr, r->k_stride, r->heads_kv, r->d), weight_of(r, q_weight),
                       weight_of(r, k_weight), positions_of(r), per_entry(r, r->lengths), frequencies_of(r)}),
            "an output or the workspace overlaps another argument");
    const hipStream_t st = (hipStream_t)stream;
    RotateArgs A = arguments(r);
    A.sign = -1.0f;
    Unit u(r);
    if (r->heads_q) u.fit(dq_out, r->q_out_stride, r->d), u.fit(dq, r->dq_stride, r->d);
    if (r->heads_kv) u.fit(dk_out, r->k_out_stride, r->d), u.fit(dk, r->dk_stride, r->d);
    if (!r->norm) {
      set(A.part[0], dq_out, r->q_out_stride, dq, r->dq_stride, nullptr, r->heads_q);
      set(A.part[1], dk_out, r->k_out_stride, dk, r->dk_stride, nullptr, r->heads_kv);
      run(r, A, u.e, st);
      return SINKHORN_OK;
    }
    if (r->heads_q) u.fit(q, r->q_stride, r->d);
    if (r->heads_kv) u.fit(k, r->k_stride, r->d);
    set(A.part[0], q, r->q_stride, dq, r->dq_stride, q_weight, r->heads_q);
    set(A.part[1], k, r->k_stride, dk, r->dk_stride, k_weight, r->heads_kv);
    A.part[0].dy = dq_out;
    A.part[1].dy = dk_out;
    for (int i = 0; i < 3; ++i) {
      A.part[0].ys[i] = r->q_out_stride[i];
      A.part[1].ys[i] = r->k_out_stride[i];
    }
    A.sums = (float*)workspace;
    const int32_t blocks = grad_blocks(r);
    if (r->dtype == SINKHORN_BF16)
      rotate_grad<__bf16>(A, u.e, blocks, st);
    else if (r->dtype == SINKHORN_F16)
      rotate_grad<_Float16>(A, u.e, blocks, st);
    else
      rotate_grad<float>(A, u.e, blocks, st);
    if (dq_weight || dk_weight) {
      hipLaunchKernelGGL(k_weight_join, grid1(2 * ceil_div(r->d, 4), 256), dim3(256), 0, st, A, dq_weight, dk_weight);
      SK_LAUNCH_CHECK();
    }
    return SINKHORN_OK;
  });
}

int sinkhorn_cache_append(const sinkhorn_rotation* r, const sinkhorn_pages* c, const void* q, const void* k, const void* v,
                          const int64_t* v_stride, const void* q_weight, const void* k_weight, void* q_out, void* k_cache,
                          void* v_cache, int32_t* lengths_out, void* stream) {
  return guarded([&] {
    check(r);
    check_pages(c);
    require(r->heads_kv >= 1, "no key heads");
    if (r->batch == 0) return SINKHORN_OK;
    const bool rows = r->len > 0, places = c->table_len > 0 && c->pages > 0;
    require(v_stride != nullptr && c->lengths && lengths_out, "null pointer");
    require(!rows || (k && v && (r->heads_q == 0 || (q && q_out))), "null pointer");
    require(!places || (k_cache && v_cache), "null pointer");
    // a token looks its place up before it knows that there are no pages
    require(!(places || (rows && c->table_len > 0)) || c->page_table, "null page table");
    for (int i = 0; i < 3; ++i) require(v_stride[i] >= 0, "negative stride");
    const bool qsame = in_place(q_out, r->q_out_stride, q, r->q_stride);
    const int64_t size = elem_size(r->dtype), table[3] = {c->table_stride, 0, 0};
    require(!any_meet({heads_of(r, q_out, r->q_out_stride, r->heads_q, r->d),
                       Span(k_cache, c->k_stride, c->pages, c->page_size, r->heads_kv, r->d, size),
                       Span(v_cache, c->v_stride, c->pages, c->page_size, r->heads_kv, c->dv, size), per_entry(r, lengths_out)},
                      {heads_of(r, qsame ? nullptr : q, r->q_stride, r->heads_q, r->d), heads_of(r, k, r->k_stride, r->heads_kv, r->d),
                       heads_of(r, v, v_stride, r->heads_kv, c->dv), weight_of(r, q_weight), weight_of(r, k_weight),
                       positions_of(r), per_entry(r, r->lengths), frequencies_of(r),
                       Span(c->page_table, table, r->batch, 1, 1, c->table_len, 4), per_entry(r, c->lengths)}),
            "an output overlaps another argument");
    RotateArgs A = arguments(r);
    set(A.part[0], q, r->q_stride, q_out, r->q_out_stride, q_weight, r->heads_q);
    set(A.part[1], k, r->k_stride, k_cache, c->k_stride, k_weight, r->heads_kv);
    set(A.part[2], v, v_stride, v_cache, c->v_stride, nullptr, r->heads_kv);
    A.dv = c->dv;
    A.steps = rows ? A.len : 1;
    A.P = paging(c);
    A.lengths_out = lengths_out;
    Unit u(r);
    if (rows) {
      if (r->heads_q) u.fit(q, r->q_stride, r->d), u.fit(q_out, r->q_out_stride, r->d);
      u.fit(k, r->k_stride, r->d), u.fit(k_cache, c->k_stride, r->d);
      u.fit(v, v_stride, c->dv), u.fit(v_cache, c->v_stride, c->dv);
    }
    run(r, A, u.e, (hipStream_t)stream);
    return SINKHORN_OK;
  });
}

}  // extern "C"
