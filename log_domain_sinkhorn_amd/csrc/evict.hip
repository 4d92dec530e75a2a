// Eviction from a cache by gathered attention weight: of each (batch entry,
// key head)'s live keys keep the first ones, the recent ones and the heaviest
// of the rest, and move the kept rows of k, v and the weight to the front of
// the output buffers in their order.
//
// k_evict_select (one workgroup per pair) finds the keep-th largest weight by
// radix selection on the weights' bits taken as ordered integers (8 bits a
// pass, counts in LDS: integer sums, so the result is exact and does not depend
// on the order of threads). Keys that are kept in any case count as the highest;
// of those that equal the threshold the lowest indices are kept. It then counts
// the kept keys before every 256th one. Up to 65536 keys stay in registers as
// ordered integers over the passes. One compute unit's vector work bounds it, so
// all that can be done by others is: k_evict_move (one workgroup per 256 keys)
// takes the threshold and those counts, finds its kept keys' places and copies
// their rows, bound by memory (4 x 8 x 65536 keys to 16384, rows of 128 bf16: with
// the places found by k_evict_select that one took 78 us in place of 27; k_evict_move
// takes 112).
#include "attention.h"
#include "overlap.h"

namespace sk {
namespace attn {
namespace {

struct EvictArgs {
  int32_t batch, heads;
  int64_t len, cap;  // keys per pair in, rows per pair out (min(keep, len))
  int64_t keep, first, recent;
  const int32_t* klen;   // nullable
  const float* mass;     // [batch][heads][len]
  float* mass_out;       // [batch][heads][cap]
  int32_t* index_out;    // [batch][heads][cap]
  int32_t* lengths_out;  // [batch]
  const char* src[2];    // k, v
  char* dst[2];
  int64_t ss[2][3], ds[2][3];  // strides in bytes: batch, row, head
  int32_t width[2];            // row width in units of the copy
  uint32_t* limit;   // [pairs][2] threshold, and how many keys equal to it are kept
  uint32_t* before;  // [pairs][groups][2] kept for sure, and equal to the threshold, before a group
  int64_t groups;    // of kGroup keys
};

constexpr int kGroup = 256;  // keys of a workgroup of k_evict_move
constexpr int kSelThreads = 1024;
constexpr int kSelPer = 16;  // keys of a thread in a chunk
constexpr int kSelChunk = kSelThreads * kSelPer;
constexpr int kSelFew = 4;  // the same where all keys fit kSelThreads * kSelFew
// Copies of the counts, by lane: equal weights (keys that gathered none) would
// otherwise make a wave's additions to one counter wait for each other.
constexpr int kCopies = 8;

__device__ __forceinline__ int64_t evict_len(const EvictArgs& A, int b) {
  if (!A.klen) return A.len;
  const int64_t n = A.klen[b];
  return n < 0 ? 0 : (n > A.len ? A.len : n);
}

// Weights as ordered integers: a NaN is the lowest, -0 equals +0. Values below
// kLowest and above that of +infinity stand for no weight.
constexpr uint32_t kNone = 0u, kLowest = 2u, kAlways = 0xffffffffu;
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  const uint32_t v = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return x != x ? kLowest : v;
}

// Key j of n with weight x: the first `lo` and those from `hi` on are always kept.
__device__ __forceinline__ uint32_t key_value(float x, int j, int n, int lo, int hi) {
  return j >= n ? kNone : (j < lo || j >= hi ? kAlways : order_key(x));
}

// C: chunks of keys held in registers; 0: any number, read in each pass. P: keys of
// a thread in a chunk.
template <int C, int P>
__global__ __launch_bounds__(kSelThreads) void k_evict_select(EvictArgs A) {
  constexpr int kChunk = kSelThreads * P;
  constexpr int kSub = kChunk / kGroup, kOwn = 64 * P / kGroup;  // groups of a chunk, of a wave's part of it
  static_assert(kSub <= 64 && kOwn * kGroup == 64 * P, "a lane of one wave for each group");
  __shared__ uint32_t hist[256][kCopies];
  __shared__ uint32_t scount[2][kSub];
  __shared__ uint32_t sdigit, sbefore;
  const int64_t pair = blockIdx.x;
  const int b = (int)(pair / A.heads);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = (int)evict_len(A, b);
  const int keep = (int)(A.keep < A.len ? A.keep : A.len);
  const int left = n < keep ? n : keep;
  if (tid == 0 && pair == (int64_t)b * A.heads) A.lengths_out[b] = left;
  // in 64 bits: a step from below cap, itself below 2^31, can lead past 2^31
  for (int64_t j = left + tid; j < A.cap; j += kSelThreads) {
    A.index_out[pair * A.cap + j] = -1;
    A.mass_out[pair * A.cap + j] = 0.0f;
  }
  if (n <= keep) return;  // all kept
  const float* w = A.mass + pair * A.len;
  const int lo = (int)A.first, hi = n - (int)A.recent;
  // a wave's keys of a chunk: 64 P consecutive ones, 64 at a time
  const int base = wave * (64 * P) + lane;
  auto read = [&](int chunk, uint32_t (&u)[P]) {
    const int j0 = chunk * kChunk + base;
    float x[P];
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = j0 + 64 * i < n ? w[j0 + 64 * i] : 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) u[i] = key_value(x[i], j0 + 64 * i, n, lo, hi);
  };
  const int chunks = (n - 1) / kChunk + 1;
  uint32_t held[C > 0 ? C : 1][P];
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) read(c, held[c]);
  }
  // f(chunk, keys) for every chunk
  auto each = [&](auto&& f) {
    if constexpr (C > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c < chunks) f(c, held[c]);
    } else {
      for (int c = 0; c < chunks; ++c) {
        read(c, held[0]);
        f(c, held[0]);
      }
    }
  };
  uint32_t need = (uint32_t)keep;  // of the keys that agree with `prefix` in the bits of `mask`; fewer than there are
  uint32_t prefix = 0, mask = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256 * kCopies; i += kSelThreads) ((uint32_t*)hist)[i] = 0;
    __syncthreads();
    each([&](int, const uint32_t (&u)[P]) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if ((u[i] & mask) == prefix) atomicAdd(&hist[(u[i] >> shift) & 255u][lane % kCopies], 1u);
    });
    __syncthreads();
    if (tid < 64) {
      // four bins a lane from the top down: lane 0 holds bins 255 .. 252
      uint32_t c[4], s = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c[e] = 0;
#pragma unroll
        for (int k = 0; k < kCopies; ++k) c[e] += hist[255 - 4 * tid - e][k];
        s += c[e];
      }
      uint32_t inc = s;
#pragma unroll
      for (int x = 1; x < 64; x <<= 1) {
        const uint32_t y = __shfl_up(inc, x);
        if (lane >= x) inc += y;
      }
      uint32_t before = inc - s;  // keys in higher bins
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (before < need && need <= before + c[e]) {
          sdigit = 255 - 4 * tid - e;
          sbefore = before;
        }
        before += c[e];
      }
    }
    __syncthreads();
    prefix |= sdigit << shift;
    mask |= 255u << shift;
    need -= sbefore;
  }
  // keys above `prefix` are kept, and the first `need` of those equal to it
  if (tid == 0) {
    A.limit[2 * pair] = prefix;
    A.limit[2 * pair + 1] = need;
  }
  uint32_t nsel = 0, neq = 0;  // before this chunk (the first wave's)
  each([&](int chunk, const uint32_t (&u)[P]) {
#pragma unroll
    for (int g = 0; g < kOwn; ++g) {
      uint32_t s = 0, q = 0;
#pragma unroll
      for (int i = 4 * g; i < 4 * g + 4; ++i) {
        s += __popcll(__ballot(u[i] > prefix));
        q += __popcll(__ballot(u[i] == prefix));
      }
      if (lane == 0) {
        scount[0][kOwn * wave + g] = s;
        scount[1][kOwn * wave + g] = q;
      }
    }
    __syncthreads();
    if (wave == 0) {
      const uint32_t s = lane < kSub ? scount[0][lane] : 0, q = lane < kSub ? scount[1][lane] : 0;
      uint32_t is = s, iq = q;
#pragma unroll
      for (int x = 1; x < 64; x <<= 1) {
        const uint32_t ys = __shfl_up(is, x), yq = __shfl_up(iq, x);
        if (lane >= x) {
          is += ys;
          iq += yq;
        }
      }
      const int64_t group = (int64_t)chunk * kSub + lane;
      if (lane < kSub && group < A.groups) {
        A.before[2 * (pair * A.groups + group)] = nsel + is - s;
        A.before[2 * (pair * A.groups + group) + 1] = neq + iq - q;
      }
      nsel += __shfl(is, 63);
      neq += __shfl(iq, 63);
    }
    __syncthreads();
  });
}

// Copies the kept rows of a group of keys, a unit U a thread and step.
template <class U>
__global__ __launch_bounds__(kGroup) void k_evict_move(EvictArgs A) {
  __shared__ int src[kGroup];
  __shared__ uint32_t swave[2][kGroup / 64];
  const int64_t pair = blockIdx.x / A.groups;
  const int64_t group = blockIdx.x - pair * A.groups;
  const int b = (int)(pair / A.heads), hd = (int)(pair - (int64_t)b * A.heads);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = (int)evict_len(A, b), j0 = (int)(group * kGroup), j = j0 + tid;
  if (j0 >= n) return;
  const int keep = (int)(A.keep < A.len ? A.keep : A.len);
  const float x = j < n ? A.mass[pair * A.len + j] : 0.0f;
  bool kept = j < n;
  int first = j0, place = tid, count = n - j0 < kGroup ? n - j0 : kGroup;  // place of the first kept key, of this among them
  if (n > keep) {
    const uint32_t limit = A.limit[2 * pair], need = A.limit[2 * pair + 1];
    const uint32_t s0 = A.before[2 * (pair * A.groups + group)], q0 = A.before[2 * (pair * A.groups + group) + 1];
    const uint32_t u = key_value(x, j, n, (int)A.first, n - (int)A.recent);
    const uint64_t sel = __ballot(u > limit), eq = __ballot(u == limit);
    if (lane == 0) {
      swave[0][wave] = (uint32_t)__popcll(sel);
      swave[1][wave] = (uint32_t)__popcll(eq);
    }
    __syncthreads();
    uint32_t s = s0, q = q0, send = s0, qend = q0;
#pragma unroll
    for (int k = 0; k < kGroup / 64; ++k) {
      if (k < wave) {
        s += swave[0][k];
        q += swave[1][k];
      }
      send += swave[0][k];
      qend += swave[1][k];
    }
    const uint64_t below = (uint64_t(1) << lane) - 1;
    s += (uint32_t)__popcll(sel & below);
    q += (uint32_t)__popcll(eq & below);
    kept = u > limit || (u == limit && q < need);
    first = (int)(s0 + (q0 < need ? q0 : need));
    place = (int)(s + (q < need ? q : need)) - first;
    count = (int)(send + (qend < need ? qend : need)) - first;
  }
  if (kept) {
    src[place] = j;
    A.index_out[pair * A.cap + first + place] = j;
    A.mass_out[pair * A.cap + first + place] = x;
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int w = A.width[t];
    const char* from = A.src[t] + b * A.ss[t][0] + hd * A.ss[t][2];
    char* to = A.dst[t] + b * A.ds[t][0] + hd * A.ds[t][2] + first * A.ds[t][1];
    // a thread's column(s) and first row; four rows in flight
    const int wide = w < kGroup ? w : kGroup, step = kGroup / wide;
    const int r0 = tid / wide;
    if (r0 >= step) continue;
    for (int c = tid - r0 * wide; c < w; c += wide) {
      const U* p = (const U*)from + c;
      for (int r = r0; r < count; r += 4 * step) {
        U v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r + i * step < count) v[i] = __builtin_nontemporal_load((const U*)((const char*)p + src[r + i * step] * A.ss[t][1]));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r + i * step < count) __builtin_nontemporal_store(v[i], (U*)(to + (r + i * step) * A.ds[t][1]) + c);
      }
    }
  }
}

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

void check(const sinkhorn_cache* c) {
  require(c != nullptr, "null cache description");
  require(c->dtype == SINKHORN_F32 || c->dtype == SINKHORN_F16 || c->dtype == SINKHORN_BF16, "unknown dtype");
  require(c->batch >= 0 && c->heads >= 1 && c->len >= 0 && c->d >= 1 && c->dv >= 1, "bad sizes");
  require(c->len < (int64_t(1) << 31), "len must be below 2^31");
  require(c->keep >= 1 && c->first >= 0 && c->recent >= 0, "keep must be >= 1, first and recent >= 0");
  require(c->first <= c->keep && c->recent <= c->keep - c->first, "first + recent exceed keep");
  for (int i = 0; i < 3; ++i)
    require(c->k_stride[i] >= 0 && c->v_stride[i] >= 0 && c->k_out_stride[i] >= 0 && c->v_out_stride[i] >= 0,
            "negative stride");
}

int64_t space(const sinkhorn_cache* c) {
  return 8 * (int64_t)c->batch * c->heads * (1 + (c->len + kGroup - 1) / kGroup);
}

}  // namespace
}  // namespace attn
}  // namespace sk

using namespace sk;
using namespace sk::attn;

extern "C" {

int sinkhorn_cache_workspace(const sinkhorn_cache* c, int64_t* bytes) {
  return guarded([&] {
    check(c);
    require(bytes != nullptr, "null pointer");
    *bytes = space(c);
    return SINKHORN_OK;
  });
}

int sinkhorn_cache_evict(const sinkhorn_cache* c, const void* k, const void* v, const float* mass, void* k_out,
                         void* v_out, float* mass_out, int32_t* index_out, int32_t* lengths_out, void* workspace,
                         int64_t workspace_bytes, void* stream) {
  return guarded([&] {
    check(c);
    if (c->batch == 0) return SINKHORN_OK;
    require(lengths_out != nullptr, "null pointer");
    if (c->len > 0) {
      require(k && v && mass && k_out && v_out && mass_out && index_out, "null pointer");
      const int64_t pairs = (int64_t)c->batch * c->heads, in = 4 * pairs * c->len;
      const int64_t out = 4 * pairs * (c->keep < c->len ? c->keep : c->len), lengths = 4 * (int64_t)c->batch;
      require(k_out != k && k_out != v && v_out != v && v_out != k && k_out != v_out, "output aliases an input");
      // all of them are read by workgroups that run while others write (lengths_out in place of key_lengths, say)
      require(apart(mass, in, mass_out, out) && apart(mass, in, index_out, out) && apart(mass, in, lengths_out, lengths) &&
                  apart(c->key_lengths, lengths, lengths_out, lengths) && apart(c->key_lengths, lengths, mass_out, out) &&
                  apart(c->key_lengths, lengths, index_out, out) && apart(mass_out, out, index_out, out) &&
                  apart(mass_out, out, lengths_out, lengths) && apart(index_out, out, lengths_out, lengths),
              "an output overlaps an input or another output");
    }
    require(workspace_bytes >= space(c) && (space(c) == 0 || workspace != nullptr),
            "workspace too small (sinkhorn_cache_workspace)");
    require((uintptr_t)workspace % 16 == 0, "workspace must be 16-byte aligned");
    const int64_t size = c->dtype == SINKHORN_F32 ? 4 : 2;
    const int64_t cap = c->keep < c->len ? c->keep : c->len, pairs = (int64_t)c->batch * c->heads;
    require(!any_meet({Span(k_out, c->k_out_stride, c->batch, cap, c->heads, c->d, size),
                       Span(v_out, c->v_out_stride, c->batch, cap, c->heads, c->dv, size), Span(mass_out, 4 * pairs * cap),
                       Span(index_out, 4 * pairs * cap), Span(lengths_out, 4 * (int64_t)c->batch),
                       Span(workspace, space(c))},
                      {Span(k, c->k_stride, c->batch, c->len, c->heads, c->d, size),
                       Span(v, c->v_stride, c->batch, c->len, c->heads, c->dv, size), Span(mass, 4 * pairs * c->len),
                       Span(c->key_lengths, 4 * (int64_t)c->batch)}),
            "an output or the workspace overlaps another argument");
    EvictArgs A{};
    A.batch = c->batch;
    A.heads = c->heads;
    A.len = c->len;
    A.cap = cap;
    A.keep = c->keep;
    A.first = c->first;
    A.recent = c->recent;
    A.klen = c->key_lengths;
    A.mass = mass;
    A.mass_out = mass_out;
    A.index_out = index_out;
    A.lengths_out = lengths_out;
    const void* src[2] = {k, v};
    void* dst[2] = {k_out, v_out};
    const int64_t* sst[2] = {c->k_stride, c->v_stride};
    const int64_t* dst_s[2] = {c->k_out_stride, c->v_out_stride};
    const int64_t width[2] = {c->d, c->dv};
    // the widest unit that divides every address of both copies
    int64_t unit = 16;
    for (int t = 0; t < 2; ++t)
      while (unit > size) {
        bool ok = (uintptr_t)src[t] % unit == 0 && (uintptr_t)dst[t] % unit == 0 && width[t] * size % unit == 0;
        for (int i = 0; i < 3; ++i) ok = ok && sst[t][i] * size % unit == 0 && dst_s[t][i] * size % unit == 0;
        if (ok) break;
        unit /= 2;
      }
    for (int t = 0; t < 2; ++t) {
      A.src[t] = (const char*)src[t];
      A.dst[t] = (char*)dst[t];
      A.width[t] = (int32_t)(width[t] * size / unit);
      for (int i = 0; i < 3; ++i) {
        A.ss[t][i] = sst[t][i] * size;
        A.ds[t][i] = dst_s[t][i] * size;
      }
    }
    const hipStream_t st = (hipStream_t)stream;
    A.groups = (c->len + kGroup - 1) / kGroup;
    A.limit = (uint32_t*)workspace;
    A.before = (uint32_t*)workspace + 2 * pairs;
    const dim3 all = grid1(pairs, kSelThreads);
    // The smallest form that holds all keys in registers, spread over all waves; none
    // does above 65536. k_evict_select of 32 pairs, us, forms in this order:
    //   4096 keys 7.4, 11.1, 13.0, 16.3 |  4097 and 16384 -, 11.0, 13.5, 16.7
    //   16385 -, -, 18.2, 25.3 | 65536 -, -, 26.9, 45.6 | 65537 -, -, -, 54.6
    if (c->len <= kSelThreads * kSelFew)
      hipLaunchKernelGGL((k_evict_select<1, kSelFew>), all, dim3(kSelThreads), 0, st, A);
    else if (c->len <= kSelChunk)
      hipLaunchKernelGGL((k_evict_select<1, kSelPer>), all, dim3(kSelThreads), 0, st, A);
    else if (c->len <= 4 * kSelChunk)
      hipLaunchKernelGGL((k_evict_select<4, kSelPer>), all, dim3(kSelThreads), 0, st, A);
    else
      hipLaunchKernelGGL((k_evict_select<0, kSelPer>), all, dim3(kSelThreads), 0, st, A);
    SK_LAUNCH_CHECK();
    if (A.cap == 0) return SINKHORN_OK;
    const dim3 grid = grid1(pairs * A.groups, kGroup);
    switch (unit) {
      case 16: hipLaunchKernelGGL((k_evict_move<u32x4>), grid, dim3(kGroup), 0, st, A); break;
      case 8: hipLaunchKernelGGL((k_evict_move<u32x2>), grid, dim3(kGroup), 0, st, A); break;
      case 4: hipLaunchKernelGGL((k_evict_move<uint32_t>), grid, dim3(kGroup), 0, st, A); break;
      default: hipLaunchKernelGGL((k_evict_move<uint16_t>), grid, dim3(kGroup), 0, st, A); break;
    }
    SK_LAUNCH_CHECK();
    return SINKHORN_OK;
  });
}

}  // extern "C"
