// C ABI of the attention operators: argument checks, launch plans and
// workspaces. The kernels are in attend.h (forward), attend_grad.h (backward)
// and attend_mass.h (gathered weight), instantiated per element type.
#include <algorithm>
#include <initializer_list>

#include "attend.h"
#include "attend_grad.h"
#include "attend_mass.h"
#include "attention_host.h"
#include "overlap.h"

namespace sk {
namespace attn {

extern template void attend<__bf16>(const AttendArgs&, bool, const MassArgs*, hipStream_t);
extern template void attend<_Float16>(const AttendArgs&, bool, const MassArgs*, hipStream_t);
extern template void attend<float>(const AttendArgs&, bool, const MassArgs*, hipStream_t);
extern template void attend_grad<__bf16>(const GradArgs&, hipStream_t);
extern template void attend_grad<_Float16>(const GradArgs&, hipStream_t);
extern template void attend_grad<float>(const GradArgs&, hipStream_t);
extern template void attend_mass<__bf16>(const MassArgs&, hipStream_t);
extern template void attend_mass<_Float16>(const MassArgs&, hipStream_t);
extern template void attend_mass<float>(const MassArgs&, hipStream_t);

namespace {

void copy3(int64_t* dst, const int64_t* src) {
  for (int i = 0; i < 3; ++i) dst[i] = src[i];
}

// ---------------------------------------------------------------- plans
// An operand that the kernels can not load 16 bytes a lane from is first
// copied: rows at other addresses or of other widths, and strides with which a
// tile could span 2^31 bytes. A copy is [batch][length][heads][width] with the
// width rounded up to 16 bytes and zero behind d.
struct Operand {
  const void* p = nullptr;
  int64_t stride[3] = {0, 0, 0};
  int64_t len = 0;
  int32_t heads = 0, d = 0, dp = 0;
  bool copy = false;
  int64_t at = 0;  // place of the copy in the workspace
};

// group: heads that a tile takes side by side (rows of q and dout that share a
// key head; 1 for keys). The stride of others only moves the tile's base.
Operand operand(const sinkhorn_attention* a, const void* p, const int64_t* stride, int64_t len, int32_t heads,
                int32_t group, int32_t d, Space& ws) {
  const int64_t size = elem_size(a);
  Operand o;
  o.p = p;
  for (int i = 0; i < 3; ++i) o.stride[i] = stride[i];
  o.len = len;
  o.heads = heads;
  o.d = d;
  o.dp = (int32_t)(ceil_div(d * size, 16) * 16 / size);
  o.copy = !rows_aligned(p, stride, d, size, 16) || stride[1] >= (int64_t(1) << 23) / size ||
           (group > 1 && stride[2] >= (int64_t(1) << 30) / size / group);
  if (o.copy) o.at = ws.take(size * a->batch * len * heads * o.dp);
  return o;
}
Operand rows_operand(const sinkhorn_attention* a, const void* p, const int64_t* stride, int32_t d, Space& ws) {
  return operand(a, p, stride, a->len_q, a->heads_q, a->heads_q / a->heads_kv, d, ws);
}
Operand keys_operand(const sinkhorn_attention* a, const void* p, const int64_t* stride, int32_t d, Space& ws) {
  return operand(a, p, stride, a->len_k, a->heads_kv, 1, d, ws);
}

struct MassPlan {
  int64_t tiles, rows_pad;
  int32_t nsplit;
  int64_t stat_off, part_off;
};

struct AttendPlan {
  bool many;     // 128 rows per workgroup (else all rows in tiles of 32)
  bool partial;  // through partial results and k_join
  bool scores;   // the scores are kept for the gathered weight
  int32_t nsplit;
  int64_t tiles;
  int64_t score_ld;
  Operand q, k, v;
  int64_t o_off, ml_off, score_off;
  MassPlan mass;  // where the weight takes its own pass
  int64_t bytes;
};


bool wide(const sinkhorn_attention* a) { return a->d > 64 || a->dv > 64; }
// steps of the streamed side that a join costs
double join_steps(const sinkhorn_attention* a) { return a->dtype == SINKHORN_F32 ? 1.0 : 3.0; }

MassPlan plan_weight(const sinkhorn_attention* a, Space& ws) {
  MassPlan p{};
  const int64_t pairs = (int64_t)a->batch * a->heads_kv;
  const int64_t rows = a->len_q * (a->heads_q / a->heads_kv);
  p.tiles = ceil_div(a->len_k, 128);
  p.nsplit = splits(pairs * p.tiles, ceil_div(rows, 64), 768, join_steps(a), false);
  p.rows_pad = ceil_div(rows, 64) * 64;
  p.stat_off = ws.take(8 * pairs * p.rows_pad);
  if (p.nsplit > 1) p.part_off = ws.take(4 * p.nsplit * pairs * a->len_k);
  return p;
}

void use_plan(const MassPlan& p, char* ws, MassArgs& M) {
  M.tiles = p.tiles;
  M.rows_pad = p.rows_pad;
  M.nsplit = p.nsplit;
  M.stat = (f32x2*)(ws + p.stat_off);
  M.part = p.nsplit > 1 ? (float*)(ws + p.part_off) : nullptr;
}

AttendPlan plan_attend(const sinkhorn_attention* a, const void* q, const void* k, const void* v, bool mass) {
  AttendPlan p{};
  Space ws;
  const bool f32 = a->dtype == SINKHORN_F32;
  const int64_t pairs = (int64_t)a->batch * a->heads_kv;
  const int64_t rows = a->len_q * (a->heads_q / a->heads_kv);
  p.many = rows > 32;
  p.tiles = ceil_div(rows, p.many ? 128 : 32);
  const int64_t keys = p.many ? 64 : 32 * few_waves((wide(a) ? 128 : 64) * elem_size(a));  // of a tile
  const int64_t steps = ceil_div(a->len_k, keys);
  const int64_t slots = !p.many || (f32 && wide(a)) ? 256 : 512;
  p.nsplit = splits(pairs * p.tiles, steps, slots, p.many ? join_steps(a) : 7.0, !p.many);
  p.partial = p.nsplit > 1;
  p.scores = mass && !p.many;
  p.q = rows_operand(a, q, a->q_stride, a->d, ws);
  p.k = keys_operand(a, k, a->k_stride, a->d, ws);
  p.v = keys_operand(a, v, a->v_stride, a->dv, ws);
  const int64_t after_copies = ws.bytes;
  if (p.partial) {
    p.o_off = ws.take(4 * p.nsplit * pairs * rows * ceil_div(a->dv, 4) * 4);
    p.ml_off = ws.take(8 * p.nsplit * pairs * rows);
  }
  if (p.scores) {
    p.score_ld = ceil_div(a->len_k, keys) * keys;
    p.score_off = ws.take(4 * pairs * rows * p.score_ld);
  } else if (mass) {
    // the forward pass is done with its partial results by then
    Space two;
    two.bytes = after_copies;
    p.mass = plan_weight(a, two);
    ws.bytes = std::max(ws.bytes, two.bytes);
  }
  p.bytes = ws.bytes;
  return p;
}

struct GradPlan {
  int64_t tiles_q, tiles_kv, rows_pad;
  int32_t split_q, split_kv;
  Operand q, k, v, dout;
  int64_t stat_off, pq_off, pk_off, pv_off, bytes;
};

GradPlan plan_grad(const sinkhorn_attention* a, const void* q, const void* k, const void* v, const void* dout) {
  GradPlan p{};
  Space ws;
  const bool f32 = a->dtype == SINKHORN_F32;
  const int64_t pairs = (int64_t)a->batch * a->heads_kv;
  const int64_t rows = a->len_q * (a->heads_q / a->heads_kv);
  const int64_t step = f32 && wide(a) ? 32 : 64;
  p.tiles_q = ceil_div(rows, 128);
  p.tiles_kv = ceil_div(a->len_k, 128);
  p.rows_pad = ceil_div(rows, 64) * 64;
  p.split_q = splits(pairs * p.tiles_q, ceil_div(a->len_k, step), f32 && wide(a) ? 256 : 512, join_steps(a), false);
  p.split_kv = f32 || wide(a) ? splits(pairs * p.tiles_kv, ceil_div(rows, 32), 256, 4 * join_steps(a), false)
                              : splits(pairs * p.tiles_kv, ceil_div(rows, 64), 512, 2 * join_steps(a), false);
  p.q = rows_operand(a, q, a->q_stride, a->d, ws);
  p.k = keys_operand(a, k, a->k_stride, a->d, ws);
  p.v = keys_operand(a, v, a->v_stride, a->dv, ws);
  p.dout = rows_operand(a, dout, a->dout_stride, a->dv, ws);
  const int64_t dp = ceil_div(a->d, 4) * 4, dvp = ceil_div(a->dv, 4) * 4;
  p.stat_off = ws.take(8 * pairs * p.rows_pad);
  if (p.split_q > 1) p.pq_off = ws.take(4 * p.split_q * pairs * rows * dp);
  if (p.split_kv > 1) {
    p.pk_off = ws.take(4 * p.split_kv * pairs * a->len_k * dp);
    p.pv_off = ws.take(4 * p.split_kv * pairs * a->len_k * dvp);
  }
  p.bytes = ws.bytes;
  return p;
}

struct WeightPlan {
  MassPlan m;
  Operand q, k;
  int64_t bytes;
};

WeightPlan plan_mass(const sinkhorn_attention* a, const void* q, const void* k) {
  WeightPlan p{};
  Space ws;
  p.q = rows_operand(a, q, a->q_stride, a->d, ws);
  p.k = keys_operand(a, k, a->k_stride, a->d, ws);
  p.m = plan_weight(a, ws);
  p.bytes = ws.bytes;
  return p;
}

// ---------------------------------------------------------------- copies
struct Copy {
  const void* src;
  int64_t stride[3];
  int64_t len, total;  // rows of a batch entry, 16-byte chunks of the copy
  int32_t heads, d, chunks;
  u32x4* dst;
};
struct Copies {
  Copy c[4];
};

// One 16-byte chunk of a copy per thread; blockIdx.y: the operand.
template <class U>
__global__ __launch_bounds__(256) void k_copy_rows(Copies all) {
  const Copy& o = all.c[blockIdx.y];
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= o.total) return;
  constexpr int EPC = 16 / (int)sizeof(U);
  const int64_t row = i / o.chunks;
  const int c = (int)(i - row * o.chunks) * EPC;
  const int64_t bl = row / o.heads, b = bl / o.len;
  const U* p = (const U*)o.src + b * o.stride[0] + (bl - b * o.len) * o.stride[1] + (row - bl * o.heads) * o.stride[2];
  union {
    U e[EPC];
    u32x4 u;
  } x;
#pragma unroll
  for (int e = 0; e < EPC; ++e) x.e[e] = c + e < o.d ? p[c + e] : (U)0;
  o.dst[i] = x.u;
}

// The operands as the kernels read them: addresses and strides, after the
// copies that they need (in one launch).
struct Placed {
  const Operand* o;
  const void** p;
  int64_t* stride;
};

void place(const sinkhorn_attention* a, std::initializer_list<Placed> operands, char* ws, hipStream_t st) {
  const int64_t size = elem_size(a);
  Copies all{};
  unsigned n = 0;
  int64_t most = 0;
  for (const Placed& x : operands) {
    const Operand& o = *x.o;
    *x.p = o.p;
    for (int i = 0; i < 3; ++i) x.stride[i] = o.stride[i];
    if (!o.copy || o.len == 0) continue;
    Copy& c = all.c[n++];
    c.src = o.p;
    for (int i = 0; i < 3; ++i) c.stride[i] = o.stride[i];
    c.len = o.len;
    c.heads = o.heads;
    c.d = o.d;
    c.chunks = (int32_t)(o.dp * size / 16);
    c.total = a->batch * o.len * o.heads * c.chunks;
    c.dst = (u32x4*)(ws + o.at);
    most = std::max(most, c.total);
    *x.p = ws + o.at;
    x.stride[0] = o.len * o.heads * o.dp;
    x.stride[1] = (int64_t)o.heads * o.dp;
    x.stride[2] = o.dp;
  }
  if (n == 0) return;
  dim3 grid = grid1(ceil_div(most, 256), 256);
  grid.y = n;
  if (size == 4)
    hipLaunchKernelGGL((k_copy_rows<uint32_t>), grid, dim3(256), 0, st, all);
  else
    hipLaunchKernelGGL((k_copy_rows<uint16_t>), grid, dim3(256), 0, st, all);
  SK_LAUNCH_CHECK();
}

// The contiguous fp32 outputs against each other and their inputs.
void check_mass(const sinkhorn_attention* a, const float* lse, const float* row_weight, const float* mass_in,
                const float* mass_out) {
  const int64_t rows = 4 * (int64_t)a->batch * a->len_q, mass = 4 * (int64_t)a->batch * a->heads_kv * a->len_k;
  const int64_t stat = rows * a->heads_q;
  require(mass_in == mass_out || apart(mass_in, mass, mass_out, mass), "mass_out overlaps mass_in without being it");
  require(apart(row_weight, rows, mass_out, mass) && apart(lse, stat, mass_out, mass), "mass_out overlaps another argument");
}

void check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return;
  require(ws != nullptr && have >= need, "workspace too small (sinkhorn_attention_workspace)");
  require((uintptr_t)ws % 16 == 0, "workspace must be 16-byte aligned");
}

// The arrays of a call, for the test that nothing is written that another
// workgroup may be reading: by elements, as outputs may lie between the rows of
// inputs (the halves of one buffer).
Span row_heads(const sinkhorn_attention* a, const void* p, const int64_t* stride, int32_t width) {
  return Span(p, stride, a->batch, a->len_q, a->heads_q, width, elem_size(a));
}
Span key_heads(const sinkhorn_attention* a, const void* p, const int64_t* stride, int32_t width) {
  return Span(p, stride, a->batch, a->len_k, a->heads_kv, width, elem_size(a));
}
Span bias_rows(const sinkhorn_attention* a) {
  const int64_t stride[3] = {a->bias_stride[0], a->bias_stride[1], 0};
  return Span(a->key_bias, stride, a->batch, a->heads_kv, 1, a->len_k, 4);
}
Span per_row(const sinkhorn_attention* a, const void* p) { return Span(p, 4 * (int64_t)a->batch * a->len_q); }
Span per_row_head(const sinkhorn_attention* a, const void* p) {
  return Span(p, 4 * (int64_t)a->batch * a->heads_q * a->len_q);
}
Span per_key(const sinkhorn_attention* a, const void* p) {
  return Span(p, 4 * (int64_t)a->batch * a->heads_kv * a->len_k);
}
Span per_entry(const sinkhorn_attention* a, const void* p) { return Span(p, 4 * (int64_t)a->batch); }

void check_apart(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  require(!any_meet(written, read), "an output or the workspace overlaps another argument");
}

// ---------------------------------------------------------------- gathered weight
// Row statistics of k_mass (natural: as for mass_row).
__global__ __launch_bounds__(256) void k_mass_stat(MassArgs A, bool natural) {
  const Shape& S = A.S;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= (int64_t)S.batch * S.hkv * A.rows_pad) return;
  const int64_t pair = idx / A.rows_pad;
  const int b = (int)(pair / S.hkv);
  const f32x2 x = mass_row(A, b, (int)(pair - (int64_t)b * S.hkv), idx - pair * A.rows_pad, live_rows(S, b), natural);
  A.stat[idx] = f32x2{-x[0], x[1]};
}

__global__ __launch_bounds__(256) void k_mass_join(MassArgs A) {
  const Shape& S = A.S;
  const int64_t n = (int64_t)S.batch * S.hkv * S.lk;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float x = 0.0f;
  for (int s = 0; s < A.nsplit; ++s) x += A.part[s * n + i];
  A.mass_out[i] = (A.mass_in ? A.mass_in[i] : 0.0f) + x;
}

// From the scores of a forward pass whose keys were not split, and its lse.
__global__ __launch_bounds__(256) void k_mass_scores(MassArgs A) {
  const float lo = A.exact ? (float)(kLog2e - (double)(float)kLog2e) : 0.0f;
  weight_keys(A, blockIdx.x, lo, [&](f32x2* srow, int64_t, int b, int hk, int64_t nrows) {
    if (threadIdx.x >= 32) return;
    f32x2 x = mass_row(A, b, hk, threadIdx.x, nrows, false);
    srow[threadIdx.x] = x[0] == kInf ? f32x2{0.0f, 0.0f} : x;
  });
}

void run_mass(const sinkhorn_attention* a, MassArgs& A, hipStream_t st) {
  if (A.S.rows > 0) {
    hipLaunchKernelGGL(k_mass_stat, grid1(ceil_div((int64_t)A.S.batch * A.S.hkv * A.rows_pad, 256), 256), dim3(256), 0,
                       st, A, a->dtype == SINKHORN_F32);
    SK_LAUNCH_CHECK();
  }
  if (a->dtype == SINKHORN_BF16)
    attend_mass<__bf16>(A, st);
  else if (a->dtype == SINKHORN_F16)
    attend_mass<_Float16>(A, st);
  else
    attend_mass<float>(A, st);
  if (A.part) {
    hipLaunchKernelGGL(k_mass_join, grid1(ceil_div((int64_t)A.S.batch * A.S.hkv * A.S.lk, 256), 256), dim3(256), 0, st,
                       A);
    SK_LAUNCH_CHECK();
  }
}

}  // namespace
}  // namespace attn
}  // namespace sk

using namespace sk;
using namespace sk::attn;

extern "C" {

int sinkhorn_attention_workspace(const sinkhorn_attention* a, int32_t what, const void* q, const void* k, const void* v,
                                 const void* dout, int64_t* bytes) {
  return guarded([&] {
    check(a);
    require(bytes != nullptr, "null pointer");
    switch (what) {
      case SINKHORN_ATTEND: *bytes = plan_attend(a, q, k, v, false).bytes; break;
      case SINKHORN_ATTEND_MASS: *bytes = plan_attend(a, q, k, v, true).bytes; break;
      case SINKHORN_ATTEND_GRAD: *bytes = plan_grad(a, q, k, v, dout).bytes; break;
      case SINKHORN_ATTENTION_MASS: *bytes = plan_mass(a, q, k).bytes; break;
      default: fail(SINKHORN_ERR_INVALID_ARG, "unknown workspace kind");
    }
    return SINKHORN_OK;
  });
}

int sinkhorn_cross_attention(const sinkhorn_attention* a, const void* q, const void* k, const void* v, void* out,
                             float* lse, const float* row_weight, const float* mass_in, float* mass_out,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&] {
    check(a);
    if (a->batch == 0) return SINKHORN_OK;
    const bool keys = a->len_k > 0, rows = a->len_q > 0;
    require(!rows || (q && out && lse), "null pointer");
    require(!(rows && keys) || (k && v), "null pointer");
    require(mass_out != nullptr || (mass_in == nullptr && row_weight == nullptr),
            "mass_in and row_weight need mass_out");
    require(out == nullptr || (out != q && out != k && out != v), "output aliases an input");
    const bool mass = mass_out != nullptr && keys;
    check_mass(a, lse, row_weight, mass_in, mass_out);
    require(apart(lse, 4 * (int64_t)a->batch * a->heads_q * a->len_q, mass_in,
                  4 * (int64_t)a->batch * a->heads_kv * a->len_k) &&
                apart(lse, 4 * (int64_t)a->batch * a->heads_q * a->len_q, row_weight, 4 * (int64_t)a->batch * a->len_q),
            "lse overlaps an input");
    const AttendPlan p = plan_attend(a, q, k, v, mass);
    check_workspace(workspace, workspace_bytes, p.bytes);
    check_apart({row_heads(a, out, a->out_stride, a->dv), per_row_head(a, lse), per_key(a, mass_out),
                 Span(workspace, p.bytes)},
                {row_heads(a, q, a->q_stride, a->d), key_heads(a, k, a->k_stride, a->d),
                 key_heads(a, v, a->v_stride, a->dv), bias_rows(a), per_entry(a, a->query_lengths),
                 per_entry(a, a->key_lengths), per_row(a, row_weight),
                 per_key(a, mass_in == mass_out ? nullptr : mass_in)});
    const hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    AttendArgs A{};
    A.S = make_shape(a);
    if (rows) place(a, {{&p.q, &A.S.q, A.S.qs}, {&p.k, &A.S.k, A.S.ks}, {&p.v, &A.S.v, A.S.vs}}, ws, st);
    copy3(A.os, a->out_stride);
    A.out = out;
    A.lse = lse;
    A.dvp = (int32_t)(ceil_div(a->dv, 4) * 4);
    A.nsplit = p.nsplit;
    A.tiles = p.tiles;
    A.vec = rows_aligned(out, a->out_stride, a->dv, elem_size(a), 4 * elem_size(a));
    if (p.partial) {
      A.opart = (float*)(ws + p.o_off);
      A.mlpart = (f32x2*)(ws + p.ml_off);
    }
    if (p.scores) {
      A.scores = (float*)(ws + p.score_off);
      A.score_ld = p.score_ld;
    }
    MassArgs M{};
    M.S = A.S;
    M.lse = lse;
    M.weight = row_weight;
    M.mass_in = mass_in;
    M.mass_out = mass_out;
    M.scores = A.scores;
    M.score_ld = A.score_ld;
    M.exact = a->dtype == SINKHORN_F32;
    M.deal = (int64_t)a->batch * a->heads_kv * ceil_div(a->len_k, 1024) < 512;  // two workgroups a compute unit
    const MassArgs* with = p.scores && p.partial ? &M : nullptr;
    if (rows) {
      if (a->dtype == SINKHORN_BF16)
        attend<__bf16>(A, p.many, with, st);
      else if (a->dtype == SINKHORN_F16)
        attend<_Float16>(A, p.many, with, st);
      else
        attend<float>(A, p.many, with, st);
    }
    if (mass && p.scores && !(rows && with)) {
      hipLaunchKernelGGL(k_mass_scores, grid1(weight_blocks(M), 256), dim3(256), 0, st, M);
      SK_LAUNCH_CHECK();
    } else if (mass && !p.scores) {
      use_plan(p.mass, ws, M);
      run_mass(a, M, st);
    }
    return SINKHORN_OK;
  });
}

int sinkhorn_cross_attention_grad(const sinkhorn_attention* a, const void* q, const void* k, const void* v,
                                  const void* out, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&] {
    check(a);
    if (a->batch == 0) return SINKHORN_OK;
    const bool keys = a->len_k > 0, rows = a->len_q > 0;
    require(!rows || (q && out && lse && dout && dq), "null pointer");
    require(!keys || (dk && dv), "null pointer");
    require(!(rows && keys) || (k && v), "null pointer");
    for (void* o : {dq, dk, dv})
      require(o == nullptr || (o != q && o != k && o != v && o != out && o != dout), "output aliases an input");
    require((!keys || dk != dv) && (!(rows && keys) || (dq != dk && dq != dv)), "outputs alias each other");
    const GradPlan p = plan_grad(a, q, k, v, dout);
    check_workspace(workspace, workspace_bytes, p.bytes);
    check_apart({row_heads(a, dq, a->dq_stride, a->d), key_heads(a, dk, a->dk_stride, a->d),
                 key_heads(a, dv, a->dv_stride, a->dv), Span(workspace, p.bytes)},
                {row_heads(a, q, a->q_stride, a->d), key_heads(a, k, a->k_stride, a->d),
                 key_heads(a, v, a->v_stride, a->dv), row_heads(a, out, a->out_stride, a->dv),
                 row_heads(a, dout, a->dout_stride, a->dv), per_row_head(a, lse), bias_rows(a),
                 per_entry(a, a->query_lengths), per_entry(a, a->key_lengths)});
    const hipStream_t st = (hipStream_t)stream;
    const int64_t size = elem_size(a);
    char* ws = (char*)workspace;
    GradArgs A{};
    A.S = make_shape(a);
    copy3(A.os, a->out_stride);
    copy3(A.dos, a->dout_stride);
    if (rows && keys) {
      place(a, {{&p.q, &A.S.q, A.S.qs}, {&p.k, &A.S.k, A.S.ks}, {&p.v, &A.S.v, A.S.vs}, {&p.dout, &A.dout, A.dos}}, ws,
            st);
    } else {
      A.dout = dout;  // only its products with out, which is 0
    }
    copy3(A.dqs, a->dq_stride);
    copy3(A.dks, a->dk_stride);
    copy3(A.dvs, a->dv_stride);
    A.out = out;
    A.lse = lse;
    A.dq = dq;
    A.dk = dk;
    A.dv = dv;
    A.stat = (f32x2*)(ws + p.stat_off);
    A.rows_pad = p.rows_pad;
    A.dp = (int32_t)(ceil_div(a->d, 4) * 4);
    A.dvp = (int32_t)(ceil_div(a->dv, 4) * 4);
    A.split_q = p.split_q;
    A.split_kv = p.split_kv;
    A.tiles_q = p.tiles_q;
    A.tiles_kv = p.tiles_kv;
    if (p.split_q > 1) A.part_q = (float*)(ws + p.pq_off);
    if (p.split_kv > 1) {
      A.part_k = (float*)(ws + p.pk_off);
      A.part_v = (float*)(ws + p.pv_off);
    }
    A.vec_q = rows_aligned(dq, a->dq_stride, a->d, size, 4 * size);
    A.vec_k = rows_aligned(dk, a->dk_stride, a->d, size, 4 * size);
    A.vec_v = rows_aligned(dv, a->dv_stride, a->dv, size, 4 * size);
    A.out_vec = rows_aligned(out, A.os, a->dv, size, 16);
    if (a->dtype == SINKHORN_BF16)
      attend_grad<__bf16>(A, st);
    else if (a->dtype == SINKHORN_F16)
      attend_grad<_Float16>(A, st);
    else
      attend_grad<float>(A, st);
    return SINKHORN_OK;
  });
}

int sinkhorn_attention_mass(const sinkhorn_attention* a, const void* q, const void* k, const float* lse,
                            const float* row_weight, const float* mass_in, float* mass_out, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  return guarded([&] {
    check(a);
    if (a->batch == 0 || a->len_k == 0) return SINKHORN_OK;
    require(mass_out != nullptr, "null pointer");
    require(a->len_q == 0 || (q && k && lse), "null pointer");
    check_mass(a, lse, row_weight, mass_in, mass_out);
    const WeightPlan p = plan_mass(a, q, k);
    check_workspace(workspace, workspace_bytes, p.bytes);
    check_apart({per_key(a, mass_out), Span(workspace, p.bytes)},
                {row_heads(a, q, a->q_stride, a->d), key_heads(a, k, a->k_stride, a->d), bias_rows(a),
                 per_entry(a, a->query_lengths), per_entry(a, a->key_lengths), per_row_head(a, lse),
                 per_row(a, row_weight), per_key(a, mass_in == mass_out ? nullptr : mass_in)});
    const hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    MassArgs M{};
    M.S = make_shape(a);
    if (a->len_q > 0) place(a, {{&p.q, &M.S.q, M.S.qs}, {&p.k, &M.S.k, M.S.ks}}, ws, st);
    M.lse = lse;
    M.weight = row_weight;
    M.mass_in = mass_in;
    M.mass_out = mass_out;
    use_plan(p.m, ws, M);
    run_mass(a, M, st);
    return SINKHORN_OK;
  });
}

}  // extern "C"
