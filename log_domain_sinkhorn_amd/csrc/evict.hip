// Eviction from a cache by gathered attention weight: of each (batch entry,
// key head)'s live keys keep the first ones, the recent ones and the heaviest
// of the rest, and move the kept rows of k, v and the weight to the front of
// the output buffers in their order.
//
// k_evict_select (one workgroup per pair) finds the keep-th largest weight by
// radix selection on the weights' bits taken as ordered integers (8 bits a
// pass, counts in LDS: integer sums, so the result is exact and does not depend
// on the order of threads), then writes the kept indices in order; keys that
// equal the threshold are taken from the lowest index up. Keys that are kept
// in any case count as the highest. Up to 65536 keys stay in registers as such
// integers over the passes; reading and converting them in each pass took 104 us
// in place of 2x us at 65536 keys.
// k_evict_move copies the rows. The copy is bound by memory.
#include "attention.h"

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
  int64_t blocks_per_pair;
};

constexpr int kSelThreads = 1024;
constexpr int kSelPer = 16;  // keys of a thread in a chunk
constexpr int kSelChunk = kSelThreads * kSelPer;
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

// C: chunks of keys held in registers; 0: any number, read in each pass.
template <int C>
__global__ __launch_bounds__(kSelThreads) void k_evict_select(EvictArgs A) {
  __shared__ uint32_t hist[256][kCopies];
  __shared__ uint32_t swave[2][kSelThreads / 64];
  __shared__ uint32_t sdigit, sbefore;
  const int64_t pair = blockIdx.x;
  const int b = (int)(pair / A.heads);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = (int)evict_len(A, b);
  const int keep = (int)(A.keep < A.len ? A.keep : A.len);
  const int left = n < keep ? n : keep;
  const float* w = A.mass + pair * A.len;
  int32_t* idx = A.index_out + pair * A.cap;
  float* mo = A.mass_out + pair * A.cap;
  if (tid == 0 && pair == (int64_t)b * A.heads) A.lengths_out[b] = left;
  for (int j = left + tid; j < (int)A.cap; j += kSelThreads) {
    idx[j] = -1;
    mo[j] = 0.0f;
  }
  if (n <= keep) {
    for (int j = tid; j < n; j += kSelThreads) {
      idx[j] = j;
      mo[j] = w[j];
    }
    return;
  }
  const int lo = (int)A.first, hi = n - (int)A.recent;
  // a wave's keys of a chunk: 1024 consecutive ones, 64 at a time
  const int base = wave * (64 * kSelPer) + lane;
  auto read = [&](int chunk, uint32_t (&u)[kSelPer]) {
    const int j0 = chunk * kSelChunk + base;
    float x[kSelPer];
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) x[i] = j0 + 64 * i < n ? w[j0 + 64 * i] : 0.0f;
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      const int j = j0 + 64 * i;
      u[i] = j >= n ? kNone : (j < lo || j >= hi ? kAlways : order_key(x[i]));
    }
  };
  const int chunks = (n - 1) / kSelChunk + 1;
  uint32_t held[C > 0 ? C : 1][kSelPer];
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
    each([&](int, const uint32_t (&u)[kSelPer]) {
#pragma unroll
      for (int i = 0; i < kSelPer; ++i)
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
  uint32_t nsel = 0, neq = 0;  // kept for sure, and equal, before this chunk
  each([&](int chunk, const uint32_t (&u)[kSelPer]) {
    uint64_t sel[kSelPer], eq[kSelPer];
    uint32_t csel = 0, ceq = 0;
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      sel[i] = __ballot(u[i] > prefix);
      eq[i] = __ballot(u[i] == prefix);
      csel += __popcll(sel[i]);
      ceq += __popcll(eq[i]);
    }
    if (lane == 0) {
      swave[0][wave] = csel;
      swave[1][wave] = ceq;
    }
    __syncthreads();
    uint32_t s = nsel, q = neq;  // kept, and equal, before this wave's keys
#pragma unroll
    for (int k = 0; k < kSelThreads / 64; ++k) {
      if (k < wave) {
        s += swave[0][k];
        q += swave[1][k];
      }
      nsel += swave[0][k];
      neq += swave[1][k];
    }
    const uint64_t below = (uint64_t(1) << lane) - 1;
    const int j0 = chunk * kSelChunk + base;
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      const uint32_t es = s + __popcll(sel[i] & below), ee = q + __popcll(eq[i] & below);
      if (((sel[i] >> lane) & 1) || (((eq[i] >> lane) & 1) && ee < need)) {
        const uint32_t pos = es + (ee < need ? ee : need);
        if (pos < (uint32_t)keep) {
          idx[pos] = j0 + 64 * i;
          mo[pos] = w[j0 + 64 * i];
        }
      }
      s += __popcll(sel[i]);
      q += __popcll(eq[i]);
    }
    __syncthreads();
  });
}

// Copies the kept rows: UNIT bytes a thread and step, 32 rows per workgroup.
template <class U>
__global__ __launch_bounds__(256) void k_evict_move(EvictArgs A) {
  const int64_t pair = blockIdx.x / A.blocks_per_pair;
  const int64_t r0 = (blockIdx.x - pair * A.blocks_per_pair) * 32;
  const int b = (int)(pair / A.heads), hd = (int)(pair - (int64_t)b * A.heads);
  const int64_t n = evict_len(A, b);
  const int64_t left = n < A.cap ? n : A.cap;
  const int rows = left - r0 < 32 ? (int)(left - r0) : 32;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int w = A.width[t];
    const char* src = A.src[t] + b * A.ss[t][0] + hd * A.ss[t][2];
    char* dst = A.dst[t] + b * A.ds[t][0] + hd * A.ds[t][2];
    for (int i = threadIdx.x; i < rows * w; i += 256) {
      const int r = i / w, c = i - r * w;
      const int64_t j = A.index_out[pair * A.cap + r0 + r];
      ((U*)(dst + (r0 + r) * A.ds[t][1]))[c] = ((const U*)(src + j * A.ss[t][1]))[c];
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

}  // namespace
}  // namespace attn
}  // namespace sk

using namespace sk;
using namespace sk::attn;

extern "C" int sinkhorn_cache_evict(const sinkhorn_cache* c, const void* k, const void* v, const float* mass,
                                    void* k_out, void* v_out, float* mass_out, int32_t* index_out,
                                    int32_t* lengths_out, void* stream) {
  return guarded([&] {
    require(c != nullptr, "null cache description");
    require(c->dtype == SINKHORN_F32 || c->dtype == SINKHORN_F16 || c->dtype == SINKHORN_BF16, "unknown dtype");
    require(c->batch >= 0 && c->heads >= 1 && c->len >= 0 && c->d >= 1 && c->dv >= 1, "bad sizes");
    require(c->len < (int64_t(1) << 31), "len must be below 2^31");
    require(c->keep >= 1 && c->first >= 0 && c->recent >= 0, "keep must be >= 1, first and recent >= 0");
    require(c->first <= c->keep && c->recent <= c->keep - c->first, "first + recent exceed keep");
    for (int i = 0; i < 3; ++i)
      require(c->k_stride[i] >= 0 && c->v_stride[i] >= 0 && c->k_out_stride[i] >= 0 && c->v_out_stride[i] >= 0,
              "negative stride");
    if (c->batch == 0) return SINKHORN_OK;
    require(lengths_out != nullptr, "null pointer");
    if (c->len > 0) {
      require(k && v && mass && k_out && v_out && mass_out && index_out, "null pointer");
      require(k_out != k && v_out != v && k_out != v_out && mass_out != mass, "output aliases an input");
    }
    const int64_t size = c->dtype == SINKHORN_F32 ? 4 : 2;
    EvictArgs A{};
    A.batch = c->batch;
    A.heads = c->heads;
    A.len = c->len;
    A.cap = c->keep < c->len ? c->keep : c->len;
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
    const int64_t pairs = (int64_t)c->batch * c->heads;
    const dim3 all = grid1(pairs, kSelThreads);
    if (c->len <= kSelChunk)
      hipLaunchKernelGGL((k_evict_select<1>), all, dim3(kSelThreads), 0, st, A);
    else if (c->len <= 4 * kSelChunk)
      hipLaunchKernelGGL((k_evict_select<4>), all, dim3(kSelThreads), 0, st, A);
    else
      hipLaunchKernelGGL((k_evict_select<0>), all, dim3(kSelThreads), 0, st, A);
    SK_LAUNCH_CHECK();
    if (A.cap == 0) return SINKHORN_OK;
    A.blocks_per_pair = (A.cap + 31) / 32;
    const dim3 grid = grid1(pairs * A.blocks_per_pair, 256);
    switch (unit) {
      case 16: hipLaunchKernelGGL((k_evict_move<u32x4>), grid, dim3(256), 0, st, A); break;
      case 8: hipLaunchKernelGGL((k_evict_move<u32x2>), grid, dim3(256), 0, st, A); break;
      case 4: hipLaunchKernelGGL((k_evict_move<uint32_t>), grid, dim3(256), 0, st, A); break;
      default: hipLaunchKernelGGL((k_evict_move<uint16_t>), grid, dim3(256), 0, st, A); break;
    }
    SK_LAUNCH_CHECK();
    return SINKHORN_OK;
  });
}
