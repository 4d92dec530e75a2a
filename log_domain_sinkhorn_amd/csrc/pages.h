// A paged cache as the host describes it and as the kernels see it.
#pragma once

#include "attention_host.h"
#include "divide.h"

namespace sk {
namespace attn {

struct Paging {
  const int32_t* table;
  const int32_t* lengths;  // keys of each entry
  int64_t stride, pages;
  int32_t size, len;  // of a page, of an entry's part of the table
  Divide page;        // of a key
};

// Keys of entry b, within what its table has places for.
__device__ __forceinline__ int32_t paged_keys(const Paging& P, int b) {
  const int32_t n = P.lengths[b], cap = P.len * P.size;
  return n < 0 ? 0 : (n > cap ? cap : n);
}

inline void check_pages(const sinkhorn_pages* c) {
  require(c != nullptr, "null cache description");
  require(c->page_size >= 8 && c->page_size % 8 == 0, "page_size must be a multiple of 8");
  require(c->table_len >= 0 && c->pages >= 0 && c->table_stride >= 0, "negative size");
  require(c->table_len * (int64_t)c->page_size < (int64_t(1) << 31) && c->pages < (int64_t(1) << 31),
          "places of a sequence, and pages, must be below 2^31");
  require(c->dv >= 1, "head widths must be >= 1");
  if (c->dv > 128) fail(SINKHORN_ERR_UNSUPPORTED, "head widths above 128");
  for (int i = 0; i < 3; ++i) require(c->k_stride[i] >= 0 && c->v_stride[i] >= 0, "negative stride");
}

inline Paging paging(const sinkhorn_pages* c) {
  Paging P{};
  P.table = c->page_table;
  P.lengths = c->lengths;
  P.stride = c->table_stride;
  P.pages = c->pages;
  P.size = c->page_size;
  P.len = c->table_len;
  P.page = Divide(P.size);
  return P;
}

}  // namespace attn
}  // namespace sk
