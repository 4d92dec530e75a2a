// Cross attention, forward: out = softmax(scale q.k + bias) v row by row, in
// one pass over the keys with a running reference and sum, for the rows of one
// (batch entry, key head) pair.
//
// A wave holds 32 rows as the columns of transposed tiles: S^T = K Q^T (keys
// down, rows across), so a row's maximum and sum are over a lane's own
// registers and one exchange with the lane 32 away; the weights feed
// O^T = V^T P^T from their registers. WQ waves take different rows of the
// same keys and WK waves different keys of the same rows (joined through LDS
// at the end): 4 x 1 for many rows, 1 x 6, 3 or 2 (few_waves, by the bytes of a
// row) when one tile of 32 rows holds them all. The keys are split over workgroups when rows and heads alone do not fill
// the chip; k_join then joins the partial results.
//
// Tiles of keys lie in a ring of LDS buffers, filled by loads to LDS while an
// earlier one is computed on: one barrier per tile and no staging registers,
// which for many rows (two buffers) leaves two waves a SIMD whose matrix and
// vector work overlap. With few rows memory is the bound: three tiles of 48 KB,
// two of them in flight while one is computed on.
#pragma once

#include "attend_mass.h"
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
  float* scores;  // [batch * hkv][score_ld / 32][rows][32] scores (fp32: natural, else log2 units), nullable
  int64_t score_ld;
  int32_t dvp;     // dv rounded up to 4
  int32_t nsplit;  // splits of the keys
  int64_t tiles;   // row tiles per pair
  bool vec;        // out may be written four elements at a time
};

// Few rows: waves of a workgroup, each with 32 keys of a tile, and tiles in LDS
// for rows of `bytes` bytes: 144 KB, two thirds of it in flight; for the widest
// rows, of which three tiles do not fit, 128 KB and half of it.
constexpr int few_waves(int64_t bytes) { return bytes <= 128 ? 6 : (bytes <= 256 ? 3 : 2); }
constexpr int few_depth(int64_t bytes) { return bytes <= 256 ? 3 : 2; }

template <class T, int W, int WQ, int WK, int NB, int D, int OCC>
__global__ __launch_bounds__(64 * WQ * WK, OCC) void k_attend(
    AttendArgs A) {
  constexpr int DP = row_width(W);
  using TL = Tile<T, DP>;
  using V8 = typename Vec<T>::V8;
  constexpr int NT = 64 * WQ * WK;
  constexpr int KT = 32 * NB * WK;  // keys per tile
  constexpr int NS = W / 16, NDB = W / 32;
  // fp32: scores in natural units, rounded once, and 2^(log2e s - m) with the
  // product inside an fma: a weight is off by what its score's own rounding
  // makes it. 16-bit types: log2 units from the start, one operation less.
  constexpr bool kExact = sizeof(T) == 4;
  constexpr float kTerm = kExact ? 1.0f : (float)kLog2e;
  constexpr bool AHEAD = WK == 1 && TL::RB == 128;
  static_assert(WK == 1 || (WQ == 1 && NB == 1), "few rows: one tile of 32, a wave's own 32 keys");
  using KeyT = KeyTiles<T, DP, KT, NT, D, (WK > 1), true>;  // few rows: each key is read by one workgroup
  constexpr int kJoinBytes = WK > 1 ? WK * 32 * W * 4 : 0;
  union Memory {
    typename KeyT::Shared keys;
    float join[kJoinBytes / 4 + 1];  // [WK][W][32]
  };
  __shared__ Memory sm;
  __shared__ f32x2 sml[WK > 1 ? WK * 32 : 1];

  const Shape& S = A.S;
  const int64_t pairs = (int64_t)S.batch * S.hkv;
  const int64_t item = xcd_item(pairs, A.tiles * A.nsplit);
  if (item < 0) return;
  int64_t pair = item / (A.tiles * A.nsplit);
  const int64_t rest = item - pair * (A.tiles * A.nsplit);
  const int64_t tile = rest / A.nsplit;
  const int split = (int)(rest - tile * A.nsplit);
  const int pos = (int)(pair / S.hkv), hk = (int)(pair - (int64_t)pos * S.hkv);
  const int b = batch_entry(S, pos);
  pair = (int64_t)b * S.hkv + hk;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r32 = lane & 31;
  const int wq = wave % WQ, wk = wave / WQ;

  const int64_t nkeys = live_keys(S, b), nrows = live_rows(S, b);
  const int64_t row0 = tile * (32 * WQ);
  const int64_t row = row0 + 32 * wq + r32;
  const bool live_row = row < nrows;
  const int64_t qi = row / S.group;
  const int qh = hk * S.group + (int)(row - qi * S.group);

  // this split's tiles of the live keys
  const int64_t ntiles = row0 < nrows ? (nkeys + KT - 1) / KT : 0;
  const int64_t per = (ntiles + A.nsplit - 1) / A.nsplit;
  const int64_t t0 = split * per, t1 = t0 + per < ntiles ? t0 + per : ntiles;

  KeyT keys(sm.keys, S, b, hk, t0, t1, nkeys, kTerm, wave, lane);
  keys.begin();

  V8 qf[NS];
  {
    const T* qrow = (const T*)S.q + b * S.qs[0] + qi * S.qs[1] + qh * S.qs[2];
#pragma unroll
    for (int s = 0; s < NS; ++s) qf[s] = global_frag<T>(qrow, live_row && t0 < t1, s, h, S.d);
  }
  loads_done();
  f32x16 o[NDB];
#pragma unroll
  for (int n = 0; n < NDB; ++n) o[n] = zero16();
  float m = -kInf, l = 0.0f;  // the row's reference (log2 units) and this lane's part of the sum

  if constexpr (WK == 1 && OCC == 2) one_ahead();
  for (int it = 0; it < keys.count; ++it) {
    // each of the last two tiles stored its scores with an instruction at least
    keys.template next<(D > 2 ? 2 : 0)>(it, D > 2 && A.scores && it >= 2);
    const char* const tk = keys.ktile(it);
    const char* const tv = keys.vtile(it);
    const int kb0 = 32 * NB * wk;
    f32x16 sc[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) sc[n] = zero16();
    if constexpr (AHEAD) {
      // all fragments on their way before the first product: left alone, the
      // compiler reads one or two ahead and each product waits for LDS (512 x
      // 2000 x 16 heads of 64 x 8, fp16: 42.9 -> 41.6 us; of 128 columns no gain)
      V8 kf[NS][NB];
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int n = 0; n < NB; ++n) kf[s][n] = TL::row_frag(tk, kb0 + 32 * n + r32, s, h);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int n = 0; n < NB; ++n) sc[n] = mma(kf[s][n], qf[s], sc[n]);
    } else {
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int n = 0; n < NB; ++n) sc[n] = s + 2 < NS ? mma(TL::row_frag(tk, kb0 + 32 * n + r32, s, h), qf[s], sc[n])
                           : mma_first(TL::row_frag(tk, kb0 + 32 * n + r32, s, h), qf[s], sc[n], S.d - 16 * s);
    }
    float f = kExact ? (float)kLog2e : S.c;  // to log2 units
    if (kExact || keys.masked(it)) {
      const float* const term = keys.term(it);
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 ct = *(const f32x4*)&term[kb0 + 32 * n + 8 * g + 4 * h];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = sc[n][4 * g + e];
            sc[n][4 * g + e] = kExact ? fmaf(x, S.scale, fmaf(x, S.scale_lo, ct[e])) : fmaf(x, S.c, ct[e]);
          }
        }
      if (!kExact) f = 1.0f;
    }
    if constexpr (WK > 1) {
      if (A.scores) {
        // Through this wave's own rows of the k tile, which it is done with, so
        // that a row's 32 scores go out as one 128-byte line (361 -> 349 us at
        // 16 x 8 x 32768 keys against four 32-byte pieces of a line each).
        const float u = kExact ? 1.0f : f;
        char* const mine = const_cast<char*>(tk) + kb0 * TL::RB;
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *(f32x4*)(mine + 128 * r32 + 16 * ((2 * g + h) ^ (r32 & 7))) =
              f32x4{sc[0][4 * g] * u, sc[0][4 * g + 1] * u, sc[0][4 * g + 2] * u, sc[0][4 * g + 3] * u};
        float* const dst = A.scores + S.rows * (pair * A.score_ld + (t0 + it) * KT + kb0);
        for (int r = lane >> 3; r < (int)S.rows; r += 8)
          *(f32x4*)(dst + 32 * r + 4 * (lane & 7)) = *(const f32x4*)(mine + 128 * r + 16 * ((lane & 7) ^ (r & 7)));
      }
    }
    float mx = -kInf;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = fmaxf(mx, sc[n][e]);
    mx = half_max(mx) * f;
    // a new reference only where the maximum rose by more than 2^8: weights
    // stay below 2^8 and the accumulators are seldom rescaled
    if (__any(mx > m + 8.0f)) {
      const float mn = fmaxf(m, mx);
      const float a = mn == -kInf ? 1.0f : ex2(m - mn);
      m = mn;
      l *= a;
#pragma unroll
      for (int n = 0; n < NDB; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[n][e] *= a;
    }
    const float mu = m == -kInf ? 0.0f : m;  // a row with no live key yet: all weights 0
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        sc[n][e] = ex2(fmaf(sc[n][e], f, -mu));
        l += sc[n][e];
      }
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const V8 p = pack<T>(sc[n], s);
        if constexpr (WK > 1 && sizeof(T) == 2) {
          // few rows wait for memory, not for products: weights in two parts, so
          // that a token's result is off by its own rounding alone
          const V8 r = pack_rest<T>(sc[n], s, p);
#pragma unroll
          for (int x = 0; x < NDB; ++x) {
            const V8 f = TL::col_frag(tv, kb0 + 32 * n + 16 * s, 32 * x, lane);
            o[x] = mma(f, r, mma(f, p, o[x]));
          }
        } else {
#pragma unroll
          for (int x = 0; x < NDB; ++x) o[x] = mma(TL::col_frag(tv, kb0 + 32 * n + 16 * s, 32 * x, lane), p, o[x]);
        }
      }
  }
  l = half_sum(l);
  // rows behind their sequence (whose zero scores weigh nothing), and rows without
  // any key, which masked ones would make NaN where the row is no number
  const bool live_keys = keys.live();
  const bool has = live_row && live_keys;
  if (!has) {
    m = -kInf;
    l = 0.0f;
  }

  // the row's result, column group by column group: group index c4 of four
  // columns, value x (not divided by the sum)
  const bool part = A.opart != nullptr;
  if constexpr (WK > 1) {
    float* const so = sm.join;
    __syncthreads();
    if (h == 0) sml[wk * 32 + r32] = f32x2{m, l};
#pragma unroll
    for (int x = 0; x < NDB; ++x)
#pragma unroll
      for (int e = 0; e < 16; ++e) so[(wk * W + 32 * x + 8 * (e >> 2) + 4 * h + (e & 3)) * 32 + r32] = has ? o[x][e] : 0.0f;
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
    for (int it = 0; it < (W * 8 + NT - 1) / NT; ++it) {
      const int c = 4 * ((tid >> 5) + it * (NT / 32));
      if (c >= W) break;
      f32x4 x = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < WK; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = fmaf(f[w], so[(w * W + c + e) * 32 + (tid & 31)], x[e]);
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
        A.lse[((int64_t)b * S.hq + jh) * S.lq + ji] = log_sum(mm, ll);
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
        f32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = has ? o[n][4 * g + e] : 0.0f;
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
        A.lse[((int64_t)b * S.hq + qh) * S.lq + qi] = log_sum(m, l);
    }
  }
}

// Joins the splits of a row: 32 lanes per column group of four; GR groups of
// lanes take every GR-th split and are added in a fixed order, 8 / GR rows per
// workgroup. Few rows with many splits (decoding) take GR = 8: their loads are
// then all in flight at once instead of one after the other (26 -> 4 us for 33
// splits).
template <class T, int GR>
__device__ __forceinline__ void join_rows(const AttendArgs& A, int64_t blk) {
  __shared__ f32x4 so[GR > 1 ? 256 : 1];
  __shared__ f32x2 sml[GR > 1 ? 8 : 1];
  const Shape& S = A.S;
  const int64_t n = (int64_t)S.batch * S.hkv * S.rows;  // rows in all
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int64_t idx = blk * (8 / GR) + grp / GR;
  const bool live = idx < n;
  const int c = 4 * lane;
  // maximum over this group's splits, then over the groups
  const int g = grp % GR;
  float mm = -kInf;
  if (live)
    for (int s = g + GR * lane; s < A.nsplit; s += GR * 32) mm = fmaxf(mm, A.mlpart[s * n + idx][0]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) mm = fmaxf(mm, __shfl_xor(mm, x, 32));
  if constexpr (GR > 1) {
    if (lane == 0) sml[grp][0] = mm;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < GR; ++k) mm = fmaxf(mm, sml[grp - g + k][0]);
    __syncthreads();
  }
  const float mu = mm == -kInf ? 0.0f : mm;
  float ll = 0.0f;
  f32x4 x = {0, 0, 0, 0};
  if (live) {
    int s = g;
    for (; s + 3 * GR < A.nsplit; s += 4 * GR) {
      f32x2 p[4];
      f32x4 o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        p[k] = A.mlpart[(s + k * GR) * n + idx];
        o[k] = c < A.dvp ? *(const f32x4*)(A.opart + ((s + k * GR) * n + idx) * A.dvp + c) : f32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = ex2(p[k][0] - mu);
        ll = fmaf(f, p[k][1], ll);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = fmaf(f, o[k][e], x[e]);
      }
    }
    for (; s < A.nsplit; s += GR) {
      const f32x2 p = A.mlpart[s * n + idx];
      const f32x4 o = c < A.dvp ? *(const f32x4*)(A.opart + (s * n + idx) * A.dvp + c) : f32x4{0, 0, 0, 0};
      const float f = ex2(p[0] - mu);
      ll = fmaf(f, p[1], ll);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = fmaf(f, o[e], x[e]);
    }
  }
  if constexpr (GR > 1) {
    so[threadIdx.x] = x;
    if (lane == 0) sml[grp][1] = ll;
    __syncthreads();
    if (g != 0) return;
#pragma unroll
    for (int k = 1; k < GR; ++k) {
      const f32x4 y = so[threadIdx.x + 32 * k];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] += y[e];
      ll += sml[grp + k][1];
    }
  }
  if (!live) return;
  const int64_t pair = idx / S.rows, row = idx - pair * S.rows;
  const int b = (int)(pair / S.hkv), hk = (int)(pair - (int64_t)b * S.hkv);
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
  if (c == 0) A.lse[((int64_t)b * S.hq + qh) * S.lq + qi] = log_sum(mm, ll);
}

template <class T, int GR>
__global__ __launch_bounds__(256) void k_join(AttendArgs A) {
  join_rows<T, GR>(A, blockIdx.x);
}

// The join and, in the workgroups behind its `joins`, the gathered weight. These
// take a row's reference and sum from the splits themselves: 8 lanes a row.
template <class T, int GR>
__global__ __launch_bounds__(256) void k_join_weight(AttendArgs A, MassArgs M, int64_t joins) {
  if (blockIdx.x < joins) {
    join_rows<T, GR>(A, blockIdx.x);
    return;
  }
  weight_keys(M, blockIdx.x - joins, 0.0f, [&](f32x2* srow, int64_t pair, int b, int, int64_t nrows) {
    const Shape& S = A.S;
    const int r = threadIdx.x >> 3, ln = threadIdx.x & 7;
    const int64_t n = (int64_t)S.batch * S.hkv * S.rows, idx = pair * S.rows + r;
    const bool live = r < nrows;
    float mm = -kInf, ll = 0.0f;
    if (live)
      for (int s = ln; s < A.nsplit; s += 8) mm = fmaxf(mm, A.mlpart[s * n + idx][0]);
#pragma unroll
    for (int x = 4; x > 0; x >>= 1) mm = fmaxf(mm, __shfl_xor(mm, x, 8));
    const float mu = mm == -kInf ? 0.0f : mm;
    if (live)
      for (int s = ln; s < A.nsplit; s += 8) {
        const f32x2 p = A.mlpart[s * n + idx];
        ll = fmaf(ex2(p[0] - mu), p[1], ll);
      }
#pragma unroll
    for (int x = 4; x > 0; x >>= 1) ll += __shfl_xor(ll, x, 8);
    if (ln == 0) {
      const float w = live && M.weight ? M.weight[b * S.lq + r / S.group] : 1.0f;
      srow[r] = f32x2{mu, ll == 0.0f ? 0.0f : w / ll};
    }
  });
}

// many: 128 rows per workgroup, else all rows in one tile of 32
template <class T, int W>
void attend_launch(const AttendArgs& A, bool many, hipStream_t st) {
  const int64_t blocks = xcd_blocks((int64_t)A.S.batch * A.S.hkv, A.tiles * A.nsplit);
  constexpr int RB = row_width(W) * (int)sizeof(T);
  // many rows: two waves a SIMD (three for rows of 128 bytes); with fewer
  // registers a wave spills, and half tiles cost more in what each tile
  // repeats than they gain in occupancy (8192 x 16384 x 32 heads of 128: 2.2 ms
  // against 5.2 when both were measured)
  constexpr int OCC = RB == 128 ? 3 : (RB == 256 ? 2 : 1);
  if (many)
    hipLaunchKernelGGL((k_attend<T, W, 4, 1, 2, 2, OCC>), grid1(blocks, 256), dim3(256), 0, st, A);
  else
    hipLaunchKernelGGL((k_attend<T, W, 1, few_waves(RB), 1, few_depth(RB), RB == 128 ? 2 : 1>),
                       grid1(blocks, 64 * few_waves(RB)), dim3(64 * few_waves(RB)), 0, st, A);
  SK_LAUNCH_CHECK();
}

// M: the gathered weight from the scores (else null).
template <class T>
void join_splits(const AttendArgs& A, const MassArgs* M, hipStream_t st) {
  const int64_t rows = (int64_t)A.S.batch * A.S.hkv * A.S.rows;
  auto join = [&](auto gr) {
    constexpr int GR = decltype(gr)::value;
    const int64_t blocks = GR == 8 ? rows : (rows + 7) / 8;
    if (M)
      hipLaunchKernelGGL((k_join_weight<T, GR>), grid1(blocks + weight_blocks(*M), 256), dim3(256), 0, st, A, *M, blocks);
    else
      hipLaunchKernelGGL((k_join<T, GR>), grid1(blocks, 256), dim3(256), 0, st, A);
    SK_LAUNCH_CHECK();
  };
  if (A.nsplit >= 8)
    join(std::integral_constant<int, 8>{});
  else
    join(std::integral_constant<int, 1>{});
}

// Instantiated once per element type (attend_*.hip). M: the gathered weight from
// the scores, where the keys are split (else null).
template <class T>
void attend(const AttendArgs& A, bool many, const MassArgs* M, hipStream_t st) {
  by_width(A.S.d, A.S.dv, [&](auto w) { attend_launch<T, decltype(w)::value>(A, many, st); });
  if (A.opart) join_splits<T>(A, M, st);
}

}  // namespace attn
}  // namespace sk
