// C ABI of the attention operators: argument checks, launch plans and
// workspaces. The kernels are in attend.h (forward), attend_grad.h (backward)
// and attend_mass.h (gathered weight), instantiated per element type.
#include <initializer_list>

#include "attend.h"
#include "attend_grad.h"
#include "attend_mass.h"

namespace sk {
namespace attn {

extern template void attend<__bf16>(const AttendArgs&, bool, hipStream_t);
extern template void attend<_Float16>(const AttendArgs&, bool, hipStream_t);
extern template void attend<float>(const AttendArgs&, bool, hipStream_t);
extern template void attend_grad<__bf16>(const GradArgs&, bool, hipStream_t);
extern template void attend_grad<_Float16>(const GradArgs&, bool, hipStream_t);
extern template void attend_grad<float>(const GradArgs&, bool, hipStream_t);
extern template void attend_mass<__bf16>(const MassArgs&, bool, hipStream_t);
extern template void attend_mass<_Float16>(const MassArgs&, bool, hipStream_t);
extern template void attend_mass<float>(const MassArgs&, bool, hipStream_t);

namespace {

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

void require(bool ok, const char* what) {
  if (!ok) fail(SINKHORN_ERR_INVALID_ARG, what);
}

constexpr int64_t kFill = 512;  // workgroups that fill the chip: two for each of the 256 compute units

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Splits of the streamed side (`steps` tiles of it) for `blocks` workgroups:
// one when they fill the chip by themselves.
int32_t splits(int64_t blocks, int64_t steps) {
  if (blocks <= 0 || blocks * 2 > kFill || steps <= 1) return 1;
  const int64_t want = ceil_div(kFill, blocks);
  return (int32_t)(want < steps ? want : steps);
}

int64_t elem_size(const sinkhorn_attention* a) { return a->dtype == SINKHORN_F32 ? 4 : 2; }

void check(const sinkhorn_attention* a) {
  require(a != nullptr, "null attention description");
  require(a->dtype == SINKHORN_F32 || a->dtype == SINKHORN_F16 || a->dtype == SINKHORN_BF16, "unknown dtype");
  require(a->batch >= 0 && a->len_q >= 0 && a->len_k >= 0, "negative size");
  require(a->heads_q >= 1 && a->heads_kv >= 1 && a->heads_q % a->heads_kv == 0,
          "heads_q must be a multiple of heads_kv");
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

struct Operand {
  const void* p;
  const int64_t* stride;
  int64_t width;
};

// Bytes a lane may load to LDS at once from the rows of `ops`: 16, 4, or 2 for
// a row that is not a multiple of four bytes (loaded through registers), as for
// row strides of 2^23 bytes and more, with which a tile could span 2^31 bytes.
int32_t load_unit(std::initializer_list<Operand> ops, int64_t size) {
  bool by16 = true, by4 = true;
  for (const Operand& o : ops) {
    if (o.stride[1] * size >= (int64_t(1) << 23)) return 2;
    by16 = by16 && rows_aligned(o.p, o.stride, o.width, size, 16);
    by4 = by4 && rows_aligned(o.p, o.stride, o.width, size, 4);
  }
  return by16 ? 16 : (by4 ? 4 : 2);
}

Shape make_shape(const sinkhorn_attention* a, const void* q, const void* k, const void* v) {
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
  for (int i = 0; i < 3; ++i) {
    S.qs[i] = a->q_stride[i];
    S.ks[i] = a->k_stride[i];
    S.vs[i] = a->v_stride[i];
  }
  S.q = q;
  S.k = k;
  S.v = v;
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

void copy3(int64_t* dst, const int64_t* src) {
  for (int i = 0; i < 3; ++i) dst[i] = src[i];
}

// ---------------------------------------------------------------- plans
struct AttendPlan {
  bool many;       // 128 rows per workgroup (else all rows in tiles of 32)
  bool partial;    // through partial results and k_join
  bool scores;     // the scores are kept for the gathered weight
  int32_t nsplit;
  int64_t tiles;
  int64_t score_ld;
  int64_t ml_off, score_off, bytes;
};

AttendPlan plan_attend(const sinkhorn_attention* a, bool mass) {
  AttendPlan p{};
  const int64_t pairs = (int64_t)a->batch * a->heads_kv;
  const int64_t rows = a->len_q * (a->heads_q / a->heads_kv);
  p.many = rows > 32;
  p.tiles = ceil_div(rows, p.many ? 128 : 32);
  p.nsplit = splits(pairs * p.tiles, ceil_div(a->len_k, p.many || a->dtype == SINKHORN_F32 ? 64 : 128));
  p.partial = p.nsplit > 1;
  p.scores = mass && !p.many;
  const int64_t dvp = ceil_div(a->dv, 4) * 4;
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = off;
    off += ceil_div(bytes, 256) * 256;
    return at;
  };
  if (p.partial) {
    take(4 * p.nsplit * pairs * rows * dvp);
    p.ml_off = take(8 * p.nsplit * pairs * rows);
  }
  if (p.scores) {
    p.score_ld = ceil_div(a->len_k, 128) * 128;
    p.score_off = take(4 * pairs * rows * p.score_ld);
  }
  p.bytes = off;
  return p;
}

struct GradPlan {
  int64_t tiles_q, tiles_kv;
  int32_t split_q, split_kv;
  int64_t pq_off, pk_off, pv_off, bytes;
};

GradPlan plan_grad(const sinkhorn_attention* a) {
  GradPlan p{};
  const int64_t pairs = (int64_t)a->batch * a->heads_kv;
  const int64_t rows = a->len_q * (a->heads_q / a->heads_kv);
  p.tiles_q = ceil_div(rows, 128);
  p.tiles_kv = ceil_div(a->len_k, 128);
  p.split_q = splits(pairs * p.tiles_q, ceil_div(a->len_k, 64));
  p.split_kv = splits(pairs * p.tiles_kv, ceil_div(rows, 64));
  const int64_t dp = ceil_div(a->d, 4) * 4, dvp = ceil_div(a->dv, 4) * 4;
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = off;
    off += ceil_div(bytes, 256) * 256;
    return at;
  };
  take(8 * pairs * rows);
  if (p.split_q > 1) p.pq_off = take(4 * p.split_q * pairs * rows * dp);
  if (p.split_kv > 1) {
    p.pk_off = take(4 * p.split_kv * pairs * a->len_k * dp);
    p.pv_off = take(4 * p.split_kv * pairs * a->len_k * dvp);
  }
  p.bytes = off;
  return p;
}

struct MassPlan {
  int64_t tiles;
  int32_t nsplit;
  int64_t bytes;
};

MassPlan plan_mass(const sinkhorn_attention* a) {
  MassPlan p{};
  const int64_t pairs = (int64_t)a->batch * a->heads_kv;
  const int64_t rows = a->len_q * (a->heads_q / a->heads_kv);
  p.tiles = ceil_div(a->len_k, 128);
  p.nsplit = splits(pairs * p.tiles, ceil_div(rows, 64));
  p.bytes = p.nsplit > 1 ? 4 * p.nsplit * pairs * a->len_k : 0;
  return p;
}

void check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return;
  require(ws != nullptr && have >= need, "workspace too small (sinkhorn_attention_workspace)");
  require((uintptr_t)ws % 16 == 0, "workspace must be 16-byte aligned");
}

// ---------------------------------------------------------------- gathered weight
__global__ __launch_bounds__(256) void k_mass_join(MassArgs A) {
  const Shape& S = A.S;
  const int64_t n = (int64_t)S.batch * S.hkv * S.lk;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float x = 0.0f;
  for (int s = 0; s < A.nsplit; ++s) x += A.part[s * n + i];
  A.mass_out[i] = (A.mass_in ? A.mass_in[i] : 0.0f) + x;
}

// From the forward kernel's scores: rows <= 32, four keys a thread.
__global__ __launch_bounds__(256) void k_mass_scores(MassArgs A) {
  __shared__ f32x2 srow[32];
  const Shape& S = A.S;
  const int64_t chunks = (S.lk + 1023) / 1024;
  const int64_t pair = blockIdx.x / chunks;
  const int64_t j = (blockIdx.x - pair * chunks) * 1024 + 4 * threadIdx.x;
  const int b = (int)(pair / S.hkv), hk = (int)(pair - (int64_t)b * S.hkv);
  const int64_t nkeys = live_keys(S, b), nrows = live_rows(S, b);
  if (threadIdx.x < 32) srow[threadIdx.x] = mass_row(A, b, hk, threadIdx.x, nrows, A.exact);
  __syncthreads();
  f32x4 x = {0, 0, 0, 0};
  const float f = A.exact ? (float)kLog2e : 1.0f;
  if (j < nkeys) {
    // the forward kernel wrote whole tiles of the live keys
    const float* sc = A.scores + pair * S.rows * A.score_ld + j;
    for (int r = 0; r < (int)nrows; ++r) {
      const f32x4 t = *(const f32x4*)(sc + r * A.score_ld);
      const f32x2 st = srow[r];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = fmaf(st[1], ex2((t[e] - st[0]) * f), x[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (j + e < S.lk) {
      const int64_t i = pair * S.lk + j + e;
      A.mass_out[i] = (A.mass_in ? A.mass_in[i] : 0.0f) + (j + e < nkeys ? x[e] : 0.0f);
    }
}

void run_mass(const sinkhorn_attention* a, MassArgs& A, hipStream_t st) {
  const int64_t size = elem_size(a);
  const bool al = rows_aligned(A.S.q, a->q_stride, a->d, size, 16) && rows_aligned(A.S.k, a->k_stride, a->d, size, 16);
  if (a->dtype == SINKHORN_BF16)
    attend_mass<__bf16>(A, al, st);
  else if (a->dtype == SINKHORN_F16)
    attend_mass<_Float16>(A, al, st);
  else
    attend_mass<float>(A, al, st);
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

int sinkhorn_attention_workspace(const sinkhorn_attention* a, int32_t what, int64_t* bytes) {
  return guarded([&] {
    check(a);
    require(bytes != nullptr, "null pointer");
    switch (what) {
      case SINKHORN_ATTEND: *bytes = plan_attend(a, false).bytes; break;
      case SINKHORN_ATTEND_MASS: {
        const int64_t x = plan_attend(a, true).bytes, y = plan_mass(a).bytes;
        *bytes = x > y ? x : y;
        break;
      }
      case SINKHORN_ATTEND_GRAD: *bytes = plan_grad(a).bytes; break;
      case SINKHORN_ATTENTION_MASS: *bytes = plan_mass(a).bytes; break;
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
    const AttendPlan p = plan_attend(a, mass);
    const MassPlan mp = mass ? plan_mass(a) : MassPlan{};
    const int64_t need = mass && mp.bytes > p.bytes ? mp.bytes : p.bytes;
    check_workspace(workspace, workspace_bytes, need);
    const hipStream_t st = (hipStream_t)stream;
    const int64_t size = elem_size(a);
    char* ws = (char*)workspace;
    AttendArgs A{};
    A.S = make_shape(a, q, k, v);
    copy3(A.os, a->out_stride);
    A.out = out;
    A.lse = lse;
    A.dvp = (int32_t)(ceil_div(a->dv, 4) * 4);
    A.nsplit = p.nsplit;
    A.tiles = p.tiles;
    A.vec = rows_aligned(out, a->out_stride, a->dv, size, 4 * size);
    if (p.partial) {
      A.opart = (float*)ws;
      A.mlpart = (f32x2*)(ws + p.ml_off);
    }
    if (p.scores) {
      A.scores = (float*)(ws + p.score_off);
      A.score_ld = p.score_ld;
    }
    if (rows) {
      A.unit = load_unit({{q, a->q_stride, a->d}, {k, a->k_stride, a->d}, {v, a->v_stride, a->dv}}, size);
      if (a->dtype == SINKHORN_BF16)
        attend<__bf16>(A, p.many, st);
      else if (a->dtype == SINKHORN_F16)
        attend<_Float16>(A, p.many, st);
      else
        attend<float>(A, p.many, st);
    }
    if (mass) {
      MassArgs M{};
      M.S = A.S;
      M.lse = lse;
      M.weight = row_weight;
      M.mass_in = mass_in;
      M.mass_out = mass_out;
      if (p.scores) {
        M.scores = A.scores;
        M.score_ld = A.score_ld;
        M.exact = a->dtype == SINKHORN_F32;
        hipLaunchKernelGGL(k_mass_scores, grid1((int64_t)a->batch * a->heads_kv * ceil_div(a->len_k, 1024), 256),
                           dim3(256), 0, st, M);
        SK_LAUNCH_CHECK();
      } else {
        // the forward pass is done with the workspace by then
        M.tiles = mp.tiles;
        M.nsplit = mp.nsplit;
        M.part = mp.nsplit > 1 ? (float*)ws : nullptr;
        run_mass(a, M, st);
      }
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
    const GradPlan p = plan_grad(a);
    check_workspace(workspace, workspace_bytes, p.bytes);
    const int64_t size = elem_size(a);
    char* ws = (char*)workspace;
    GradArgs A{};
    A.S = make_shape(a, q, k, v);
    copy3(A.os, a->out_stride);
    copy3(A.dos, a->dout_stride);
    copy3(A.dqs, a->dq_stride);
    copy3(A.dks, a->dk_stride);
    copy3(A.dvs, a->dv_stride);
    A.out = out;
    A.dout = dout;
    A.lse = lse;
    A.dq = dq;
    A.dk = dk;
    A.dv = dv;
    A.stat = (f32x2*)ws;
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
    const bool al = rows_aligned(q, a->q_stride, a->d, size, 16) && rows_aligned(k, a->k_stride, a->d, size, 16) &&
                    rows_aligned(v, a->v_stride, a->dv, size, 16) &&
                    rows_aligned(dout, a->dout_stride, a->dv, size, 16);
    const hipStream_t st = (hipStream_t)stream;
    if (a->dtype == SINKHORN_BF16)
      attend_grad<__bf16>(A, al, st);
    else if (a->dtype == SINKHORN_F16)
      attend_grad<_Float16>(A, al, st);
    else
      attend_grad<float>(A, al, st);
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
    const MassPlan p = plan_mass(a);
    check_workspace(workspace, workspace_bytes, p.bytes);
    MassArgs M{};
    M.S = make_shape(a, q, k, nullptr);
    M.lse = lse;
    M.weight = row_weight;
    M.mass_in = mass_in;
    M.mass_out = mass_out;
    M.tiles = p.tiles;
    M.nsplit = p.nsplit;
    M.part = p.nsplit > 1 ? (float*)workspace : nullptr;
    run_mass(a, M, (hipStream_t)stream);
    return SINKHORN_OK;
  });
}

}  // extern "C"
