// C ABI of attention over a paged cache: argument checks, launch plan, workspace.
// The kernels are in attend_paged.h, instantiated per element type.
#include <algorithm>
#include <initializer_list>

#include "attend_paged.h"
#include "attention_host.h"
#include "overlap.h"

namespace sk {
namespace attn {

extern template void attend_paged<__bf16>(const PagedArgs&, bool, hipStream_t);
extern template void attend_paged<_Float16>(const PagedArgs&, bool, hipStream_t);
extern template void attend_paged<float>(const PagedArgs&, bool, hipStream_t);

namespace {

struct PagedPlan {
  bool many;
  int32_t nsplit;
  int64_t tiles, rows;
  int64_t o_off, ml_off, bytes;
};

// As plan_attend, for as many keys as the table has places for or the rows of a
// tile may see.
PagedPlan plan_paged(const sinkhorn_attention* a, const sinkhorn_pages* c, int64_t first, int64_t recent) {
  PagedPlan p{};
  const bool f32 = a->dtype == SINKHORN_F32, wide = a->d > 64 || a->dv > 64;
  const int64_t group = a->heads_q / a->heads_kv, pairs = (int64_t)a->batch * a->heads_kv;
  p.rows = a->len_q * group;
  p.many = p.rows > 32;
  p.tiles = ceil_div(p.rows, p.many ? 128 : 32);
  const int64_t size = elem_size(a), keys = p.many ? 64 : 32 * paged_waves((wide ? 128 : 64) * size);  // of a tile
  int64_t seen = c->table_len * (int64_t)c->page_size;
  if (recent > 0) {
    // the window of a tile's rows and the first keys, each with a tile cut at both ends
    const int64_t rows = std::min<int64_t>(a->len_q, (p.many ? 128 : 32) / group + 2);
    seen = std::min(seen, std::min(first, seen) + std::min(recent, seen) + rows + 2 * keys);
  }
  // a step of few rows takes 1.4 us, a join with its launch 4 to 5 (at 7 steps, as a
  // step of k_attend's tokens seems: 4 x 1000 keys x 8 heads of 64 14.9 -> 9.9 us, 32768 x
  // 8 of 128 46 -> 30.5)
  const int64_t slots = p.many ? (f32 && wide ? 256 : 512) : 256 * paged_groups((wide ? 128 : 64) * size);
  p.nsplit = splits(pairs * p.tiles, ceil_div(seen, keys), slots, f32 && p.many ? 1.0 : 3.0, !p.many);
  Space ws;
  if (p.nsplit > 1) {
    p.o_off = ws.take(4 * p.nsplit * pairs * p.rows * ceil_div(a->dv, 4) * 4);
    p.ml_off = ws.take(8 * p.nsplit * pairs * p.rows);
  }
  p.bytes = ws.bytes;
  return p;
}

void check_call(const sinkhorn_attention* a, const sinkhorn_pages* c, int64_t first, int64_t recent) {
  check(a);
  check_pages(c);
  require(a->dv == c->dv, "dv of the attention and of the cache differ");
  require(first >= 0 && recent >= 0, "first and recent must be >= 0");
  require(first == 0 || recent > 0, "first needs recent");
}

// Keys are loaded 16 bytes a lane, several slots at a time.
void check_rows(const void* p, const int64_t* stride, int64_t width, int64_t size, const char* what) {
  if (!rows_aligned(p, stride, width, size, 16)) fail(SINKHORN_ERR_UNSUPPORTED, what);
  if (stride[1] >= (int64_t(1) << 27) / size) fail(SINKHORN_ERR_UNSUPPORTED, "slots of a page 128 MB apart or more");
}

}  // namespace
}  // namespace attn
}  // namespace sk

using namespace sk;
using namespace sk::attn;

extern "C" {

int sinkhorn_paged_workspace(const sinkhorn_attention* a, const sinkhorn_pages* c, int64_t first, int64_t recent,
                             int64_t* bytes) {
  return guarded([&] {
    check_call(a, c, first, recent);
    require(bytes != nullptr, "null pointer");
    *bytes = plan_paged(a, c, first, recent).bytes;
    return SINKHORN_OK;
  });
}

int sinkhorn_paged_attention(const sinkhorn_attention* a, const sinkhorn_pages* c, int64_t first, int64_t recent,
                             const void* q, const void* k_cache, const void* v_cache, void* out, float* lse,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&] {
    check_call(a, c, first, recent);
    if (a->batch == 0 || a->len_q == 0) return SINKHORN_OK;
    require(q && out && lse && c->lengths, "null pointer");
    require(a->key_bias == nullptr && a->key_lengths == nullptr, "key_bias and key_lengths have no place here");
    const bool places = c->table_len > 0 && c->pages > 0;
    require(!places || (k_cache && v_cache && c->page_table), "null pointer");
    const int64_t size = elem_size(a);
    if (places) {
      check_rows(k_cache, c->k_stride, a->d, size, "keys of the cache are not whole, aligned units of 16 bytes");
      check_rows(v_cache, c->v_stride, a->dv, size, "values of the cache are not whole, aligned units of 16 bytes");
    }
    const PagedPlan p = plan_paged(a, c, first, recent);
    require(p.bytes == 0 || (workspace != nullptr && workspace_bytes >= p.bytes), "workspace too small (sinkhorn_paged_workspace)");
    require((uintptr_t)workspace % 16 == 0, "workspace must be 16-byte aligned");
    const int64_t table[3] = {c->table_stride, 0, 0};
    require(!any_meet({Span(out, a->out_stride, a->batch, a->len_q, a->heads_q, a->dv, size),
                       Span(lse, 4 * (int64_t)a->batch * a->heads_q * a->len_q), Span(workspace, p.bytes)},
                      {Span(q, a->q_stride, a->batch, a->len_q, a->heads_q, a->d, size),
                       Span(k_cache, c->k_stride, c->pages, c->page_size, a->heads_kv, a->d, size),
                       Span(v_cache, c->v_stride, c->pages, c->page_size, a->heads_kv, a->dv, size),
                       Span(c->page_table, table, a->batch, 1, 1, c->table_len, 4), Span(c->lengths, 4 * (int64_t)a->batch),
                       Span(a->query_lengths, 4 * (int64_t)a->batch)}),
            "an output or the workspace overlaps another argument");
    PagedArgs G{};
    AttendArgs& A = G.A;
    A.S = make_shape(a);
    A.S.q = q;
    A.S.k = k_cache;
    A.S.v = v_cache;
    A.S.klen = c->lengths;
    for (int i = 0; i < 3; ++i) {
      A.S.ks[i] = c->k_stride[i];
      A.S.vs[i] = c->v_stride[i];
      A.os[i] = a->out_stride[i];
    }
    A.out = out;
    A.lse = lse;
    A.dvp = (int32_t)(ceil_div(a->dv, 4) * 4);
    A.nsplit = p.nsplit;
    A.tiles = p.tiles;
    A.vec = rows_aligned(out, a->out_stride, a->dv, size, 4 * size);
    if (p.nsplit > 1) {
      A.opart = (float*)((char*)workspace + p.o_off);
      A.mlpart = (f32x2*)((char*)workspace + p.ml_off);
    }
    G.P = paging(c);
    if (!places) G.P.len = 0;  // no keys
    const int64_t most = INT32_MAX;
    G.first = (int32_t)std::min(first, most);
    G.recent = (int32_t)std::min(recent, most);
    G.rows = (int32_t)p.rows;
    G.tiles = (int32_t)p.tiles;
    G.per = (int32_t)(p.tiles * p.nsplit);
    G.by_group = Divide(A.S.group);
    G.by_heads = Divide(A.S.hkv);
    G.by_per = Divide(G.per);
    G.by_split = Divide(p.nsplit);
    G.qvec = rows_aligned(q, a->q_stride, a->d, size, 16);
    const hipStream_t st = (hipStream_t)stream;
    if (a->dtype == SINKHORN_BF16)
      attend_paged<__bf16>(G, p.many, st);
    else if (a->dtype == SINKHORN_F16)
      attend_paged<_Float16>(G, p.many, st);
    else
      attend_paged<float>(G, p.many, st);
    return SINKHORN_OK;
  });
}

}  // extern "C"
