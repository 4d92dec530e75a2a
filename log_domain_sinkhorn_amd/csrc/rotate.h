// Rotary positions with a norm of each head, and the same on the way into a
// paged cache.
//
// A group of LPH lanes holds one head at a time, a lane two chunks of E elements
// (16 bytes each where the layout allows it) whose pairs it has both elements of:
// chunks u and u + rotated / (2 E) for pairs half of the rotated part apart, any two
// for neighbours. So the rotation is in registers, the norm takes one sum
// over the group's lanes, and a lane's E angles serve all heads of its token: the
// angles are formed in 64 bits, reduced to a quarter turn there, and their sine and
// cosine are Taylor sums in fp32 (about 40 operations an angle against 14 bytes
// and more of traffic for each head that uses it).
//
// Bound by memory: each element is read once and written once.
#pragma once

#include <algorithm>

#include "attention.h"
#include "attention_host.h"
#include "pages.h"

namespace sk {
namespace attn {

// The heads of one tensor: q, k, or v, which is appended as it is.
struct HeadRows {
  const void* src;
  void* dst;
  const void* weight;    // of the norm, nullable
  const void* dy;        // backward: gradient of the result
  int64_t ss[3], ds[3], ys[3];  // elements: batch, row, head; ds of a cache: page, slot, head
  int32_t heads;
  int32_t groups;  // log2 of the lane groups that share a token's heads
  int32_t end;     // its workgroups end here (and start where the tensor's before it end)
};

struct RotateArgs {
  HeadRows part[3];  // q, k, v
  int32_t batch, len, d, dv;
  int32_t steps;   // rows of a batch entry that are visited: len, at least one where lengths are written
  Divide by_steps;
  int32_t half;    // pairs of a head
  bool interleaved, norm, weight_f32;
  float gain, sign, eps, inv_d;  // sign: -1 turns back; 1 / d
  const double* freq;
  const int32_t* positions;  // nullable
  int64_t position_stride;
  const int32_t* lengths;  // nullable
  Paging P;
  int32_t* lengths_out;  // null: no cache
  float* sums;           // backward: [workgroups][128] partial sums of the weights' gradients
};

// E elements as they lie in memory.
template <class T, int E>
struct Raw {
  typedef T V __attribute__((ext_vector_type(E)));
  __device__ __forceinline__ static float get(const V& v, int e) { return (float)v[e]; }
  __device__ __forceinline__ static void set(V& v, int e, float x) { v[e] = (T)x; }
};
template <class T>
struct Raw<T, 1> {
  typedef T V;
  __device__ __forceinline__ static float get(const V& v, int) { return (float)v; }
  __device__ __forceinline__ static void set(V& v, int, float x) { v = (T)x; }
};
template <class T, int E>
__device__ __forceinline__ void widen(const typename Raw<T, E>::V& v, float (&x)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = Raw<T, E>::get(v, e);
}
template <class T, int E>
__device__ __forceinline__ typename Raw<T, E>::V narrow(const float (&x)[E]) {
  typename Raw<T, E>::V v;
#pragma unroll
  for (int e = 0; e < E; ++e) Raw<T, E>::set(v, e, x[e]);
  return v;
}

// Results of calls that move more than the last cache holds are written past it: written
// into it they drive out each other and what is still to be read. 16384 tokens x 40 heads
// of 128 bf16 (336 MB) 71 -> 58 us, with the backward pass 172 -> 145, a call and the next
// reader of its results 95 either way, at 640 MB 204 -> 184; calls of 154 and 234 MB lose,
// 28 -> 41 and with the reader 66 -> 70.
template <bool PAST, class V>
__device__ __forceinline__ void put(V* p, const V& x) {
  if constexpr (PAST)
    __builtin_nontemporal_store(x, p);
  else
    *p = x;
}

// cos and sin of `turns` whole turns. The reduction to x quarter turns, |x| <= 1/2,
// is exact in 64 bits; sine and cosine of x pi / 2 by their Taylor sums, whose
// first terms left out are below 2e-9 and 2e-10.
__device__ __forceinline__ void cos_sin(double turns, float& c, float& s) {
  const double f = turns - rint(turns);
  const double n = rint(4.0 * f);
  const float x = (float)fma(4.0, f, -n);
  const int quarter = (int)n;
  constexpr double h = 1.57079632679489661923;  // pi / 2
  constexpr double h2 = h * h;
  const float z = x * x;
  const float sn = x * fmaf(fmaf(fmaf(fmaf(z, (float)(h2 * h2 * h2 * h2 * h / 362880), (float)(-h2 * h2 * h2 * h / 5040)),
                                      z, (float)(h2 * h2 * h / 120)), z, (float)(-h2 * h / 6)), z, (float)h);
  const float cs = fmaf(fmaf(fmaf(fmaf(fmaf(z, (float)(-h2 * h2 * h2 * h2 * h2 / 3628800), (float)(h2 * h2 * h2 * h2 / 40320)),
                                       z, (float)(-h2 * h2 * h2 / 720)), z, (float)(h2 * h2 / 24)), z, (float)(-h2 / 2)), z, 1.0f);
  const float a = quarter & 1 ? sn : cs, b = quarter & 1 ? cs : sn;
  c = (quarter + 1) & 2 ? -a : a;
  s = quarter & 2 ? -b : b;
}

// A lane's part of the heads of width d. PAIRS: neighbours turn together (for chunks
// of one element as for pairs apart, with other places). The first chunks of a
// group's lanes lie side by side, and so do the second ones, but for a step where the
// rotated part ends: a load or store of the group is one run of bytes, or two (with a
// lane's chunks side by side 16384 tokens x 40 heads of 128 bf16, neighbours, take 74 us
// in place of 65.5).
template <int E, int LPH, bool PAIRS>
struct Lane {
  int at[2];      // first element of its chunks
  bool has[2];    // are they within the head?
  bool turns[2];  // are they rotated?

  // u: the lane's place in its group; half: rotated pairs
  __device__ __forceinline__ Lane(int u, int half, int d) {
    const int n = half / E;  // lanes whose chunks are rotated, for pairs apart
    if constexpr (PAIRS) {
      at[0] = E > 1 ? u * E : 2 * u;
      at[1] = E > 1 ? (u + LPH) * E : 2 * u + 1;
    } else {
      at[0] = (u < n ? u : u + n) * E;
      at[1] = (u < n ? u + n : u + LPH) * E;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      has[k] = at[k] < d;
      turns[k] = PAIRS ? at[k] < 2 * half : u < n;
    }
  }
};

// (x, y) turned by the lane's angles: element pairs (x[e], y[e]), or with PAIRS
// neighbours in x, then in y.
template <int E, int LPH, bool PAIRS>
__device__ __forceinline__ void turn(float (&x)[E], float (&y)[E], const float (&c)[E], const float (&s)[E],
                                     const Lane<E, LPH, PAIRS>& l) {
  if constexpr (PAIRS && E > 1) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float(&z)[E] = k ? y : x;
      if (l.turns[k])
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          const float a = z[2 * e], b = z[2 * e + 1], cs = c[k * E / 2 + e], sn = s[k * E / 2 + e];
          z[2 * e] = fmaf(a, cs, -(b * sn));
          z[2 * e + 1] = fmaf(a, sn, b * cs);
        }
    }
  } else if (l.turns[0]) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float a = x[e], b = y[e];
      x[e] = fmaf(a, c[e], -(b * s[e]));
      y[e] = fmaf(a, s[e], b * c[e]);
    }
  }
}

// A lane's frequencies in turns per position.
template <int E, int LPH, bool PAIRS>
__device__ __forceinline__ void lane_frequencies(const RotateArgs& A, const Lane<E, LPH, PAIRS>& l, int u, double (&w)[E]) {
  constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
  constexpr int kFirst = PAIRS && E > 1 ? E / 2 : E;  // of the first chunk
  const double* const f0 = A.freq + (PAIRS && E > 1 ? l.at[0] / 2 : u * E);
#pragma unroll
  for (int e = 0; e < E; ++e) w[e] = 0.0;
  if (l.turns[0])
#pragma unroll
    for (int e = 0; e < kFirst; ++e) w[e] = f0[e] * kTurn;
  if (l.turns[1])
#pragma unroll
    for (int e = kFirst; e < E; ++e) w[e] = A.freq[l.at[1] / 2 + e - kFirst] * kTurn;
}
template <int E, int LPH, bool PAIRS>
__device__ __forceinline__ void lane_angles(const RotateArgs& A, const Lane<E, LPH, PAIRS>& l, const double (&w)[E], double p,
                                            float (&c)[E], float (&s)[E]) {
  if (!l.turns[0]) return;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    cos_sin(p * w[e], c[e], s[e]);
    c[e] *= A.gain;
    s[e] *= A.gain * A.sign;
  }
}

template <class T, int E, int LPH, bool PAIRS>
__device__ __forceinline__ void lane_weight(const RotateArgs& A, const void* weight, const Lane<E, LPH, PAIRS>& l, int i, float (&x)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = l.at[i] + e;
    x[e] = !weight || !l.has[i] ? 1.0f : (A.weight_f32 ? ((const float*)weight)[c] : (float)((const T*)weight)[c]);
  }
}

// Sum over the LPH lanes of a group.
template <int LPH>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int k = LPH / 2; k > 0; k >>= 1) x += __shfl_xor(x, k, 64);
  return x;
}

__device__ __forceinline__ int live_tokens(const RotateArgs& A, int b) {
  if (!A.lengths) return A.len;
  const int n = A.lengths[b];
  return n < 0 ? 0 : (n > A.len ? A.len : n);
}

// 1 / sqrt(mean + eps) from a head's sum of squares. fp32: rounded in full; else
// to about one step of fp32.
template <class T>
__device__ __forceinline__ float inverse_rms(const RotateArgs& A, float sum) {
  const float x = fmaf(sum, A.inv_d, A.eps);
  if constexpr (sizeof(T) == 4)
    return 1.0f / sqrtf(x);
  else
    return __builtin_amdgcn_rsqf(x);
}

// Forward (and the backward pass without a norm: the rotation the other way). A
// workgroup takes one of the tensors; a token's heads are dealt to 1 << groups lane
// groups, neighbours to neighbours, and U heads of a group are loaded before the
// first is used.
template <class T, int E, int LPH, int U, bool PAIRS, bool PAST>
__global__ __launch_bounds__(256) void k_rotate(RotateArgs A) {
  typedef typename Raw<T, E>::V V;
  const int which = (int)blockIdx.x < A.part[0].end ? 0 : ((int)blockIdx.x < A.part[1].end ? 1 : 2);
  const HeadRows& R = A.part[which];
  const bool value = which == 2, cache = A.lengths_out && which != 0;
  const int lane = threadIdx.x % LPH;
  const int64_t item = (int64_t)(blockIdx.x - (which ? A.part[which - 1].end : 0)) * (256 / LPH) + threadIdx.x / LPH;
  const int64_t token = item >> R.groups;
  const int g = (int)(item & ((1 << R.groups) - 1));
  if (token >= (int64_t)A.batch * A.steps) return;
  const int b = (int)A.by_steps((uint32_t)token), i = (int)token - b * A.steps;
  const int ntokens = live_tokens(A, b);
  const bool live = i < ntokens;
  const Lane<E, LPH, PAIRS> l(lane, value ? 0 : A.half, value ? A.dv : A.d);
  int64_t place = i;
  int64_t to = b * R.ds[0] + i * R.ds[1];
  if (A.lengths_out) {
    const int before = paged_keys(A.P, b);
    const int64_t j = (int64_t)before + i, cap = (int64_t)A.P.len * A.P.size;
    const int64_t after = (int64_t)before + ntokens;
    if (which == 1 && i == 0 && g == 0 && lane == 0) A.lengths_out[b] = (int)(after < cap ? after : cap);
    place = j;
    if (cache) {
      if (!live || j >= cap) return;
      const uint32_t page = A.P.page((uint32_t)j);
      const int64_t id = A.P.table[b * A.P.stride + page];
      if (id < 0 || id >= A.P.pages) return;
      to = id * R.ds[0] + (j - (int64_t)page * A.P.size) * R.ds[1];
    } else if (i >= A.len) {
      return;  // no rows at all
    }
  }
  float c[E], s[E];
  if (l.turns[0]) {
    double w[E];
    lane_frequencies(A, l, lane, w);
    if (A.positions) place = A.positions[b * A.position_stride + i];
    lane_angles(A, l, w, (double)place, c, s);
  }
  const bool norm = A.norm && !value;
  const bool turned[2] = {live && (norm || l.turns[0]), live && (norm || l.turns[1])};  // else as it is
  float weight[2][E];
  if (norm) {
    lane_weight<T>(A, R.weight, l, 0, weight[0]);
    lane_weight<T>(A, R.weight, l, 1, weight[1]);
  }
  const T* const src = (const T*)R.src + b * R.ss[0] + i * R.ss[1];
  T* const dst = (T*)R.dst + to;
  for (int h0 = g; h0 < R.heads; h0 += U << R.groups) {
    V raw[U][2];
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const int h = h0 + (n << R.groups);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        raw[n][k] = V{};
        if (live && h < R.heads && l.has[k]) raw[n][k] = *(const V*)(src + h * R.ss[2] + l.at[k]);
      }
    }
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const int h = h0 + (n << R.groups);
      if (h >= R.heads) break;
      float x[2][E];
      widen<T, E>(raw[n][0], x[0]);
      widen<T, E>(raw[n][1], x[1]);
      if (norm) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < E; ++e) sum = fmaf(x[k][e], x[k][e], sum);
        const float r = inverse_rms<T>(A, group_sum<LPH>(sum));
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < E; ++e) x[k][e] = x[k][e] * r * weight[k][e];
      }
      turn(x[0], x[1], c, s, l);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (l.has[k]) put<PAST>((V*)(dst + h * R.ds[2] + l.at[k]), turned[k] ? narrow<T, E>(x[k]) : raw[n][k]);
    }
  }
}

// Backward with a norm: with g = the rotation undone on the result's gradient,
// xh = x r, r = 1 / rms, u = g w:  dx = r (u - xh mean(u xh)),  dw = sum g xh.
// A workgroup takes rows of one tensor; a lane adds up the weight's gradient of its
// chunks over all that it meets; groups of a wave, waves and workgroups are then added
// in a fixed order.
template <class T, int E, int LPH, int U, bool PAIRS, bool PAST>
__global__ __launch_bounds__(256) void k_rotate_grad(RotateArgs A) {
  typedef typename Raw<T, E>::V V;
  __shared__ float sw[4][kMaxD];
  const int which = (int)blockIdx.x < A.part[0].end ? 0 : 1, first = which ? A.part[0].end : 0;
  const HeadRows& R = A.part[which];
  const int lane = threadIdx.x % LPH, wave = threadIdx.x >> 6;
  const Lane<E, LPH, PAIRS> l(lane, A.half, A.d);
  double w[E];
  lane_frequencies(A, l, lane, w);
  float acc[2][E], weight[2][E];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    lane_weight<T>(A, R.weight, l, k, weight[k]);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[k][e] = 0.0f;
  }
  const int64_t items = ((int64_t)A.batch * A.len) << R.groups, step = (int64_t)(R.end - first) * (256 / LPH);
  for (int64_t item = (int64_t)(blockIdx.x - first) * (256 / LPH) + threadIdx.x / LPH; item < items; item += step) {
    const uint32_t token = (uint32_t)(item >> R.groups);
    const int g = (int)(item & ((1 << R.groups) - 1));
    const int b = (int)A.by_steps(token), i = (int)token - b * A.len;
    const bool live = i < live_tokens(A, b);
    const T* const src = (const T*)R.src + b * R.ss[0] + i * R.ss[1];
    const T* const dy = (const T*)R.dy + b * R.ys[0] + i * R.ys[1];
    T* const dst = (T*)R.dst + b * R.ds[0] + i * R.ds[1];
    float c[E], s[E];
    lane_angles(A, l, w, (double)(A.positions ? A.positions[b * A.position_stride + i] : i), c, s);
    for (int h0 = g; h0 < R.heads; h0 += U << R.groups) {
      V rx[U][2], ry[U][2];
#pragma unroll
      for (int n = 0; n < U; ++n) {
        const int h = h0 + (n << R.groups);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          rx[n][k] = ry[n][k] = V{};
          if (live && h < R.heads && l.has[k]) {
            rx[n][k] = *(const V*)(src + h * R.ss[2] + l.at[k]);
            ry[n][k] = *(const V*)(dy + h * R.ys[2] + l.at[k]);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < U; ++n) {
        const int h = h0 + (n << R.groups);
        if (h >= R.heads) break;
        float x[2][E], y[2][E];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          widen<T, E>(rx[n][k], x[k]);
          widen<T, E>(ry[n][k], y[k]);
        }
        turn(y[0], y[1], c, s, l);
        float sum = 0.0f, dot = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            sum = fmaf(x[k][e], x[k][e], sum);
            dot = fmaf(y[k][e] * weight[k][e], x[k][e], dot);
          }
        const float r = inverse_rms<T>(A, group_sum<LPH>(sum));
        const float m = group_sum<LPH>(dot) * A.inv_d * r * r;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (live) acc[k][e] = fmaf(y[k][e], x[k][e] * r, acc[k][e]);
            x[k][e] = live ? r * fmaf(-m, x[k][e], y[k][e] * weight[k][e]) : 0.0f;
          }
          if (l.has[k]) put<PAST>((V*)(dst + h * R.ds[2] + l.at[k]), narrow<T, E>(x[k]));
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float x = acc[k][e];
#pragma unroll
      for (int z = LPH; z < 64; z <<= 1) x += __shfl_xor(x, z, 64);
      if ((threadIdx.x & 63) < LPH && l.has[k]) sw[wave][l.at[k] + e] = x;
    }
  __syncthreads();
  const int col = threadIdx.x;
  if (col < A.d) A.sums[(int64_t)blockIdx.x * kMaxD + col] = (sw[0][col] + sw[1][col]) + (sw[2][col] + sw[3][col]);
}

// ---------------------------------------------------------------- launches
// f(chunk, lanes, pairs): elements of a chunk (e: as many as 16 bytes hold, and the
// layout and the pairs allow), lanes for heads of up to 64 or 128 elements, neighbours.
template <class T, class F>
void by_chunk(int e, int width, bool interleaved, F&& f) {
  using std::integral_constant;
  auto go = [&](auto chunk) {
    constexpr int E = decltype(chunk)::value;
    auto wide = [&](auto pairs) {
      if (width <= kMaxD / 2)
        f(chunk, integral_constant<int, 32 / E>{}, pairs);
      else
        f(chunk, integral_constant<int, 64 / E>{}, pairs);
    };
    if (interleaved)
      wide(std::true_type{});
    else
      wide(std::false_type{});
  };
  if (e == 8) {
    if constexpr (sizeof(T) == 2) go(integral_constant<int, 8>{});
  } else if (e == 4) {
    go(integral_constant<int, 4>{});
  } else if (e == 2) {
    go(integral_constant<int, 2>{});
  } else {
    go(integral_constant<int, 1>{});
  }
}

// Lane groups of a token (log2): up to four heads share their token's angles, fewer
// where that leaves a compute unit fewer than 256 lanes (with 1024 as the bound more
// groups make the same angles: 6978 tokens x 16 heads of 32 bf16 13.1 us in place of 7.5,
// 635 x 45 of 96 9.9 of 6.9; 16384 x 40 of 128 takes four heads either way).
inline int32_t rotate_groups(int64_t tokens, int32_t heads, int32_t lanes) {
  int32_t g = 0;
  while ((1 << g) < (heads + 3) / 4) ++g;
  while ((1 << g) < heads && (tokens << g) * lanes < (int64_t)256 * 256) ++g;
  return g;
}

// Do `arrays` read or written for each of q, k and v hold more than the last cache, 256 MB?
// (Chunks of less than 16 bytes stay with plain stores, which join them in the caches.)
inline bool beyond_cache(const RotateArgs& A, int arrays, size_t size) {
  const int64_t row = (int64_t)(A.part[0].heads + A.part[1].heads) * A.d + (int64_t)A.part[2].heads * A.dv;
  return (int64_t)A.batch * A.len * row * arrays * (int64_t)size > (int64_t(1) << 28);
}

// Instantiated once per element type (rotate_*.hip). e: elements of a chunk.
template <class T>
void rotate(RotateArgs& A, int e, hipStream_t st) {
  A.by_steps = Divide(A.steps);
  const bool past = beyond_cache(A, 2, sizeof(T));
  by_chunk<T>(e, A.d > A.dv ? A.d : A.dv, A.interleaved, [&](auto chunk, auto lanes, auto pairs) {
    constexpr int E = decltype(chunk)::value, L = decltype(lanes)::value;
    constexpr bool P = decltype(pairs)::value;
    const int64_t tokens = (int64_t)A.batch * A.steps;
    int64_t blocks = 0;
    for (HeadRows& R : A.part) {
      if (R.heads > 0) {
        R.groups = rotate_groups(tokens, R.heads, L);
        blocks += ceil_div((tokens << R.groups) * L, 256);
      }
      R.end = (int32_t)std::min<int64_t>(blocks, INT32_MAX);
    }
    if (past && E * sizeof(T) == 16)
      hipLaunchKernelGGL((k_rotate<T, E, L, 4, P, E * sizeof(T) == 16>), grid1(blocks, 256), dim3(256), 0, st, A);
    else
      hipLaunchKernelGGL((k_rotate<T, E, L, 4, P, false>), grid1(blocks, 256), dim3(256), 0, st, A);
    SK_LAUNCH_CHECK();
  });
}

// blocks: workgroups for both tensors, dealt by their heads.
template <class T>
void rotate_grad(RotateArgs& A, int e, int32_t blocks, hipStream_t st) {
  A.by_steps = Divide(A.len);
  const bool past = beyond_cache(A, 3, sizeof(T));
  by_chunk<T>(e, A.d, A.interleaved, [&](auto chunk, auto lanes, auto pairs) {
    constexpr int E = decltype(chunk)::value, L = decltype(lanes)::value;
    constexpr bool P = decltype(pairs)::value;
    HeadRows &q = A.part[0], &k = A.part[1];
    for (HeadRows* R : {&q, &k}) R->groups = rotate_groups((int64_t)A.batch * A.len, R->heads, L);
    q.end = (int32_t)((int64_t)blocks * q.heads / (q.heads + k.heads));
    if (q.heads > 0 && q.end == 0) q.end = 1;
    if (k.heads > 0 && q.end == blocks) --q.end;
    k.end = blocks;
    if (past && E * sizeof(T) == 16)
      hipLaunchKernelGGL((k_rotate_grad<T, E, L, 2, P, E * sizeof(T) == 16>), grid1(blocks, 256), dim3(256), 0, st, A);
    else
      hipLaunchKernelGGL((k_rotate_grad<T, E, L, 2, P, false>), grid1(blocks, 256), dim3(256), 0, st, A);
    SK_LAUNCH_CHECK();
  });
}

}  // namespace attn
}  // namespace sk
