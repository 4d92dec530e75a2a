// Cross attention, forward: out = softmax(scale q.k + bias) v row by row, in
// one pass over the keys with a running maximum and sum, for the rows of one
// (batch entry, key head) pair.
//
// A wave holds 32 rows as the columns of transposed tiles: S^T = K Q^T (keys
// down, rows across), so a row's maximum and sum are over a lane's own
// registers and one exchange with the lane 32 away; the weights feed
// O^T = V^T P^T from their registers. WQ waves take different rows of the
// same keys and WK waves different keys of the same rows (joined through LDS
// at the end): 4 x 1 for many rows, 1 x 4 when one tile of 32 rows holds them
// all. The keys are split over workgroups when rows and heads alone do not fill
// the chip; k_join then joins the partial results.
#pragma once

#include "attention.h"

namespace sk {
namespace attn {

struct AttendArgs {
  Shape S;
  int64_t os[3];
  void* out;      // [batch][lq][hq][dv] by strides
  float* lse;     // [batch][hq][lq]
  float* opart;   // [split][batch * hkv][rows][dvp] unnormalized, nullable
  f32x2* mlpart;  // [split][batch * hkv][rows] running maximum (log2) and sum
  float* scores;  // [batch * hkv][rows][score_ld] scores in log2 units, nullable
  int64_t score_ld;
  int32_t dvp;     // dv rounded up to 4
  int32_t nsplit;  // splits of the keys
  int64_t tiles;   // row tiles per pair
  bool vec;        // out may be written four elements at a time
};

template <class T, int DP, int WQ, int WK, int NB, bool AL>
__global__ __launch_bounds__(64 * WQ * WK) void k_attend(AttendArgs A) {
  using TL = Tile<T, DP>;
  using V8 = typename Vec<T>::V8;
  constexpr int NT = 64 * WQ * WK;
  constexpr int KT = 32 * NB * WK;  // keys per tile
  constexpr int NS = DP / 16, NDB = DP / 32;
  constexpr int kTileBytes = KT * TL::RB;
  constexpr int kJoinBytes = WK > 1 ? WK * 32 * DP * 4 : 0;
  __shared__ __attribute__((aligned(16))) char sm[kJoinBytes > 2 * kTileBytes ? kJoinBytes : 2 * kTileBytes];
  __shared__ __attribute__((aligned(16))) float sterm[KT];
  __shared__ f32x2 sml[WK > 1 ? WK * 32 : 1];
  char* const sk_ = sm;
  char* const sv_ = sm + kTileBytes;

  const Shape& S = A.S;
  const int64_t pairs = (int64_t)S.batch * S.hkv;
  const int64_t item = xcd_item(pairs * A.tiles * A.nsplit);
  if (item >= pairs * A.tiles * A.nsplit) return;
  const int64_t pair = item / (A.tiles * A.nsplit);
  const int64_t rest = item - pair * (A.tiles * A.nsplit);
  const int64_t tile = rest / A.nsplit;
  const int split = (int)(rest - tile * A.nsplit);
  const int b = (int)(pair / S.hkv), hk = (int)(pair - (int64_t)b * S.hkv);

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = lane >> 5, r32 = lane & 31;
  const int wq = wave % WQ, wk = wave / WQ;

  const int64_t nkeys = live_keys(S, b), nrows = live_rows(S, b);
  const int64_t row0 = tile * (32 * WQ);
  const int64_t row = row0 + 32 * wq + r32;
  const bool live = row < nrows;
  const int64_t qi = row / S.group;
  const int qh = hk * S.group + (int)(row - qi * S.group);

  // this split's tiles of the live keys
  const int64_t ntiles = row0 < nrows ? (nkeys + KT - 1) / KT : 0;
  const int64_t per = (ntiles + A.nsplit - 1) / A.nsplit;
  const int64_t t0 = split * per, t1 = t0 + per < ntiles ? t0 + per : ntiles;

  const T* kbase = (const T*)S.k + b * S.ks[0] + hk * S.ks[2];
  const T* vbase = (const T*)S.v + b * S.vs[0] + hk * S.vs[2];
  const float* bias = S.bias ? S.bias + b * S.bs[0] + hk * S.bs[1] : nullptr;

  V8 qf[NS];
  {
    const T* qrow = (const T*)S.q + b * S.qs[0] + qi * S.qs[1] + qh * S.qs[2];
#pragma unroll
    for (int s = 0; s < NS; ++s) qf[s] = global_frag<T, AL>(qrow, live, s, h, S.d);
  }
  f32x16 o[NDB];
#pragma unroll
  for (int n = 0; n < NDB; ++n) o[n] = zero16();
  float m = -kInf, l = 0.0f;  // running maximum of the row; this lane's part of the sum

  Stage<T, DP, KT, NT, AL> xk, xv;
  float term = 0.0f;
  if (t0 < t1) {
    xk.load(kbase, S.ks[1], t0 * KT, nkeys, S.d, tid);
    xv.load(vbase, S.vs[1], t0 * KT, nkeys, S.dv, tid);
    if (tid < KT) term = column_term(bias, t0 * KT + tid, nkeys);
  }
  for (int64_t t = t0; t < t1; ++t) {
    // without a bias only a tile that the live keys end in has masked columns
    const bool masked = bias != nullptr || (t + 1) * KT > nkeys;
    __syncthreads();
    if (tid < KT) sterm[tid] = term;
    if (bias) {
      __syncthreads();
      xk.put_masked(sk_, sterm, tid);
      xv.put_masked(sv_, sterm, tid);
    } else {
      xk.put(sk_, tid);
      xv.put(sv_, tid);
    }
    __syncthreads();
    if (t + 1 < t1) {
      xk.load(kbase, S.ks[1], (t + 1) * KT, nkeys, S.d, tid);
      xv.load(vbase, S.vs[1], (t + 1) * KT, nkeys, S.dv, tid);
      if (tid < KT) term = column_term(bias, (t + 1) * KT + tid, nkeys);
    }
    f32x16 sc[NB];
    const int kb0 = wk * 32 * NB;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      sc[n] = zero16();
#pragma unroll
      for (int s = 0; s < NS; ++s)
        sc[n] = mma(TL::row_frag(sk_, kb0 + 32 * n + r32, s, h), qf[s], sc[n]);
    }
    float mx = -kInf;
    if (masked) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 ct = *(const f32x4*)&sterm[kb0 + 32 * n + 8 * g + 4 * h];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[n][4 * g + e] = fmaf(sc[n][4 * g + e], S.c, ct[e]);
            mx = fmaxf(mx, sc[n][4 * g + e]);
          }
        }
    } else {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          sc[n][e] *= S.c;
          mx = fmaxf(mx, sc[n][e]);
        }
    }
    if (A.scores && row < S.rows) {
      float* dst = A.scores + (pair * S.rows + row) * A.score_ld + t * KT + kb0;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *(f32x4*)(dst + 32 * n + 8 * g + 4 * h) =
              f32x4{sc[n][4 * g], sc[n][4 * g + 1], sc[n][4 * g + 2], sc[n][4 * g + 3]};
    }
    const float mn = fmaxf(m, half_max(mx));
    const float mu = mn == -kInf ? 0.0f : mn;  // a row with no live key yet: all weights 0
    const float a = ex2(m - mu);
    m = mn;
    l *= a;
#pragma unroll
    for (int n = 0; n < NDB; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[n][e] *= a;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        sc[n][e] = ex2(sc[n][e] - mu);
        l += sc[n][e];
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const V8 p = pack<T>(sc[n], s);
#pragma unroll
        for (int x = 0; x < NDB; ++x)
          o[x] = mma(TL::col_frag(sv_, kb0 + 32 * n + 16 * s, 32 * x, lane), p, o[x]);
      }
    }
  }
  l = half_sum(l);
  if (!live) {  // a row behind its sequence (its zero scores weigh nothing)
    m = -kInf;
    l = 0.0f;
#pragma unroll
    for (int n = 0; n < NDB; ++n) o[n] = zero16();
  }

  // the row's result, column group by column group: group index c4 of four
  // columns, value x (not divided by the sum)
  const bool part = A.opart != nullptr;
  if constexpr (WK > 1) {
    float* so = (float*)sm;  // [WK][DP][32]
    __syncthreads();
    if (h == 0) sml[wk * 32 + r32] = f32x2{m, l};
#pragma unroll
    for (int x = 0; x < NDB; ++x)
#pragma unroll
      for (int e = 0; e < 16; ++e) so[(wk * DP + 32 * x + 8 * (e >> 2) + 4 * h + (e & 3)) * 32 + r32] = o[x][e];
    __syncthreads();
    // thread: row tid % 32, column groups tid / 32, + NT / 32, ...
    const int64_t jrow = row0 + (tid & 31);
    float f[WK], mm = -kInf, ll = 0.0f;
#pragma unroll
    for (int w = 0; w < WK; ++w) mm = fmaxf(mm, sml[w * 32 + (tid & 31)][0]);
    const float mu = mm == -kInf ? 0.0f : mm;
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const f32x2 p = sml[w * 32 + (tid & 31)];
      f[w] = ex2(p[0] - mu);
      ll = fmaf(f[w], p[1], ll);
    }
    if (jrow >= S.rows) return;
    const int64_t ji = jrow / S.group;
    const int jh = hk * S.group + (int)(jrow - ji * S.group);
    // a NaN sum is kept; only an empty row is 0
    const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
    T* orow = (T*)A.out + b * A.os[0] + ji * A.os[1] + jh * A.os[2];
    float* prow = part ? A.opart + (((int64_t)split * pairs + pair) * S.rows + jrow) * A.dvp : nullptr;
#pragma unroll
    for (int it = 0; it < DP * 8 / NT; ++it) {
      const int c = 4 * ((tid >> 5) + it * (NT / 32));
      f32x4 x = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < WK; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = fmaf(f[w], so[(w * DP + c + e) * 32 + (tid & 31)], x[e]);
      if (part) {
        if (c < A.dvp) *(f32x4*)(prow + c) = x;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= inv;
        if (A.vec)
          store4<T, true>(orow, c, S.dv, x);
        else
          store4<T, false>(orow, c, S.dv, x);
      }
    }
    if (tid < 32) {
      if (part)
        A.mlpart[((int64_t)split * pairs + pair) * S.rows + jrow] = f32x2{mm, ll};
      else
        A.lse[((int64_t)b * S.hq + jh) * S.lq + ji] = ll == 0.0f ? -kInf : (mm + lg2(ll)) * (float)kLn2;
    }
  } else {
    if (row >= S.rows) return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    T* orow = (T*)A.out + b * A.os[0] + qi * A.os[1] + qh * A.os[2];
    const int64_t prow_i = ((int64_t)split * pairs + pair) * S.rows + row;
#pragma unroll
    for (int n = 0; n < NDB; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = 32 * n + 8 * g + 4 * h;
        f32x4 x = {o[n][4 * g], o[n][4 * g + 1], o[n][4 * g + 2], o[n][4 * g + 3]};
        if (part) {
          if (c < A.dvp) *(f32x4*)(A.opart + prow_i * A.dvp + c) = x;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] *= inv;
          if (A.vec)
            store4<T, true>(orow, c, S.dv, x);
          else
            store4<T, false>(orow, c, S.dv, x);
        }
      }
    if (h == 0) {
      if (part)
        A.mlpart[prow_i] = f32x2{m, l};
      else
        A.lse[((int64_t)b * S.hq + qh) * S.lq + qi] = l == 0.0f ? -kInf : (m + lg2(l)) * (float)kLn2;
    }
  }
}

// Joins the splits of a row: 32 lanes per row, four columns a lane.
template <class T>
__global__ __launch_bounds__(256) void k_join(AttendArgs A) {
  const Shape& S = A.S;
  const int64_t pairs = (int64_t)S.batch * S.hkv;
  const int64_t idx = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (idx >= pairs * S.rows) return;
  const int64_t pair = idx / S.rows, row = idx - pair * S.rows;
  const int c = 4 * (threadIdx.x & 31);
  const int b = (int)(pair / S.hkv), hk = (int)(pair - (int64_t)b * S.hkv);
  float mm = -kInf;
  for (int s = 0; s < A.nsplit; ++s) mm = fmaxf(mm, A.mlpart[s * pairs * S.rows + idx][0]);
  const float mu = mm == -kInf ? 0.0f : mm;
  float ll = 0.0f;
  f32x4 x = {0, 0, 0, 0};
  for (int s = 0; s < A.nsplit; ++s) {
    const f32x2 p = A.mlpart[s * pairs * S.rows + idx];
    const float f = ex2(p[0] - mu);
    ll = fmaf(f, p[1], ll);
    if (c < A.dvp) {
      const f32x4 o = *(const f32x4*)(A.opart + (s * pairs * S.rows + idx) * A.dvp + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = fmaf(f, o[e], x[e]);
    }
  }
  const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] *= inv;
  const int64_t qi = row / S.group;
  const int qh = hk * S.group + (int)(row - qi * S.group);
  T* orow = (T*)A.out + b * A.os[0] + qi * A.os[1] + qh * A.os[2];
  if (A.vec)
    store4<T, true>(orow, c, S.dv, x);
  else
    store4<T, false>(orow, c, S.dv, x);
  if (c == 0) A.lse[((int64_t)b * S.hq + qh) * S.lq + qi] = ll == 0.0f ? -kInf : (mm + lg2(ll)) * (float)kLn2;
}

// many: 128 rows per workgroup, else all rows in one tile of 32
template <class T, int DP, bool AL>
void attend_launch(const AttendArgs& A, bool many, hipStream_t st) {
  const int64_t blocks = xcd_blocks((int64_t)A.S.batch * A.S.hkv * A.tiles * A.nsplit);
  if (many)
    hipLaunchKernelGGL((k_attend<T, DP, 4, 1, 2, AL>), grid1(blocks, 256), dim3(256), 0, st, A);
  else
    hipLaunchKernelGGL((k_attend<T, DP, 1, 4, 1, AL>), grid1(blocks, 256), dim3(256), 0, st, A);
  SK_LAUNCH_CHECK();
}

// Instantiated once per element type (attend_*.hip).
template <class T>
void attend(const AttendArgs& A, bool many, bool aligned, hipStream_t st) {
  const bool wide = A.S.d > 64 || A.S.dv > 64;
  if (wide) {
    if (aligned)
      attend_launch<T, 128, true>(A, many, st);
    else
      attend_launch<T, 128, false>(A, many, st);
  } else {
    if (aligned)
      attend_launch<T, 64, true>(A, many, st);
    else
      attend_launch<T, 64, false>(A, many, st);
  }
  if (A.opart) {
    hipLaunchKernelGGL((k_join<T>), grid1(((int64_t)A.S.batch * A.S.hkv * A.S.rows + 7) / 8, 256), dim3(256), 0, st, A);
    SK_LAUNCH_CHECK();
  }
}

}  // namespace attn
}  // namespace sk
