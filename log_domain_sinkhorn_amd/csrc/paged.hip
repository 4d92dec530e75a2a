// C ABI of attention over a paged cache: argument checks, launch plan, workspace.
// The kernels are in attend_paged.h, instantiated per element type.
#include <algorithm>
#include <initializer_list>

#include "attend_paged.h"
#include "attention_host.h"
#include "overlap.h"

namespace sk {
namespace attn {

extern template void attend_paged<__bf16>(const PagedArgs&, PagedForm, hipStream_t);
extern template void attend_paged<_Float16>(const PagedArgs&, PagedForm, hipStream_t);
extern template void attend_paged<float>(const PagedArgs&, PagedForm, hipStream_t);

namespace {

struct PagedPlan {
  PagedForm form;
  int32_t nsplit;
  int64_t tiles, rows;
  int64_t o_off, ml_off, bytes;
};

// The forms of the kernel: 128 rows against 64 keys a step, or 32 rows against 32 keys
// of each wave. step: microseconds of a step with `slots` workgroups on the chip, by
// width (32, 64, 96, 128 columns), measured at 256 to 768 pairs of 4096 keys that share
// their pages; of the form that is alone on its compute unit at 8 and 32 pairs of 250
// to 2000 keys.
struct Form {
  PagedForm form;
  int64_t rows, keys, slots;
  double step;
};
Form form_of(const sinkhorn_attention* a, PagedForm form) {
  const bool f32 = a->dtype == SINKHORN_F32;
  const int w = head_width(a->d, a->dv) / 32 - 1;
  const int64_t bytes = row_width(32 * (w + 1)) * elem_size(a);
  static const double steps[3][2][4] = {{{1.5, 2.1, 1.9, 2.2}, {5.3, 9.1, 7.7, 10.1}},
                                        {{1.4, 1.4, 1.1, 1.2}, {1.8, 2.8, 3.8, 4.8}},
                                        {{1.6, 1.6, 2.2, 2.4}, {4.0, 6.0, 3.8, 4.8}}};
  const double step = steps[(int)form][f32][w];
  if (form == PagedForm::kMany) return Form{form, 128, 64, bytes <= 128 ? 768 : (bytes <= 256 ? 512 : 256), step};
  if (form == PagedForm::kAlone) return Form{form, 32, 32 * alone_waves(bytes), 256, step};
  return Form{form, 32, 32 * kPagedWaves, 256 * paged_groups(bytes), step};
}

// Microseconds of a call on the device: rounds of workgroups, each with 4 to begin and
// end, and the join: 4, and its partial results written and read at 4.5 TB/s. With fewer
// workgroups on a compute unit than it holds a step is shorter. The least calls take
// longer on the host, 12.5 and with a join's launch and workspace 16.5: what counts is
// the mean of a call that waits for the host and one that is replayed (32 pairs of 64
// columns bf16 over 1000 keys: split 9.9 and 16.6, not split 11.3 and 12.8).
double cost_of(const Form& f, int64_t tiles, int64_t steps, int64_t n, double partial) {
  const int64_t blocks = tiles * n, rounds = ceil_div(blocks, f.slots), most = f.slots / 256;
  const int64_t held = std::min(ceil_div(blocks, 256), most);
  const double step = f.step * (0.4 + 0.6 * (double)held / (double)most);
  const double device = (double)rounds * ((double)ceil_div(steps, n) * step + 4.0) + (n > 1 ? 4.0 + (double)n * partial / 2.25e6 : 0.0);
  return 0.5 * (device + std::max(device, n > 1 ? 16.5 : 12.5));
}

// The form and the number of splits of the keys that cost least, for as many keys as
// the table has places for or the rows of a tile may see. More than 32 rows of a pair
// take the form of few rows where its smaller tiles spread over more of the chip:
// 14 pairs of 170 rows against 2123 keys of 128 bf16 26.3 us of many rows, 20.7 of few;
// 24 x 180 against 199 of 96 13.3, 10.1; 10 x 3928 against 491 of 72 22.5, 43.7; over 40
// drawn chunks what this takes is 0.7% above the better one.
PagedPlan plan_paged(const sinkhorn_attention* a, const sinkhorn_pages* c, int64_t first, int64_t recent) {
  PagedPlan p{};
  const int64_t group = a->heads_q / a->heads_kv, pairs = (int64_t)a->batch * a->heads_kv;
  p.rows = a->len_q * group;
  const double partial = 4.0 * (double)(pairs * p.rows) * (double)(ceil_div(a->dv, 4) * 4 + 2);
  double least = 0.0;
  for (const PagedForm form : {PagedForm::kAlone, PagedForm::kFew, PagedForm::kMany}) {
    if (form == PagedForm::kMany && p.rows <= 32) continue;
    const Form f = form_of(a, form);
    const int64_t tiles = ceil_div(p.rows, f.rows);
    if (form == PagedForm::kAlone && pairs * tiles > f.slots) continue;
    int64_t seen = c->table_len * (int64_t)c->page_size;
    if (recent > 0) {
      // the window of a tile's rows and the first keys, each with a tile cut at both ends
      const int64_t rows = std::min<int64_t>(a->len_q, f.rows / group + 2);
      seen = std::min(seen, std::min(first, seen) + std::min(recent, seen) + rows + 2 * f.keys);
    }
    const int64_t steps = ceil_div(seen, f.keys), most = form == PagedForm::kAlone ? 1 : std::min<int64_t>(steps, 512);
    int64_t n = 1, best = 1;
    double cost = 0.0;
    do {  // the fewest splits for each number of steps
      const double x = cost_of(f, pairs * tiles, steps, n, partial);
      if (n == 1 || x < cost) {
        cost = x;
        best = n;
      }
      const int64_t each = ceil_div(steps, n);
      if (each <= 1) break;
      n = ceil_div(steps, each - 1);
    } while (n <= most);
    // tokens: at least four rounds where there are several, so that sequences of
    // different lengths even out
    if (p.rows <= 32 && best > 1)
      best = std::max(best, std::min(ceil_div(4 * f.slots, pairs * tiles), std::max<int64_t>(1, steps / 8)));
    if (p.tiles == 0 || cost < least) {
      least = cost;
      p.form = form;
      p.tiles = tiles;
      p.nsplit = (int32_t)best;
    }
  }
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
    G.pair_up = p.form == PagedForm::kMany && p.nsplit == 1 &&
                (int64_t)a->batch * a->heads_kv * p.tiles <= form_of(a, p.form).slots;
    G.qvec = rows_aligned(q, a->q_stride, a->d, size, 16);
    const hipStream_t st = (hipStream_t)stream;
    if (a->dtype == SINKHORN_BF16)
      attend_paged<__bf16>(G, p.form, st);
    else if (a->dtype == SINKHORN_F16)
      attend_paged<_Float16>(G, p.form, st);
    else
      attend_paged<float>(G, p.form, st);
    return SINKHORN_OK;
  });
}

}  // extern "C"
