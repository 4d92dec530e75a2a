// Cross attention, backward. With P = exp(s - lse) recomputed tile by tile and
// D_r = dout_r . out_r:
//   dV = P^T dout     dS = P o (dout V^T - D)     dQ = scale dS K     dK = scale dS^T Q
// in two kernels without atomics, so results do not depend on the order of
// workgroups: k_grad_q holds rows and runs over keys, k_grad_kv holds keys
// and runs over the rows of every head that shares them (seven products in
// place of the five that a single kernel with an atomic dQ would need).
// Both take their tiles as the forward kernel does: scores with the held side
// across, the other side down, so that the recomputed weights feed the next
// product from their registers. When the held side does not fill the chip,
// the other side is split over workgroups into fp32 partial sums, which
// k_grad_join adds in a fixed order.
#pragma once

#include <type_traits>

#include "attention.h"

namespace sk {
namespace attn {

struct GradArgs {
  Shape S;
  int64_t os[3], dos[3], dqs[3], dks[3], dvs[3];
  const void* out;
  const void* dout;
  const float* lse;
  void* dq;
  void* dk;
  void* dv;
  f32x2* stat;       // [batch * hkv][rows_pad] from k_grad_q: minus lse (-inf: the row takes no part), D
  int64_t rows_pad;  // rows rounded up to 64
  float* part_q;  // [split][batch * hkv][rows][dp], nullable
  float* part_k;  // [split][batch * hkv][lk][dp], nullable
  float* part_v;  // [split][batch * hkv][lk][dvp], nullable
  int32_t dp, dvp;
  int32_t split_q, split_kv;
  int64_t tiles_q, tiles_kv;
  bool vec_q, vec_k, vec_v;  // dq, dk, dv may be written four elements at a time
  bool out_vec;              // out may be read 16 bytes at a time
};

// exp(score - lse) of a product x, its column term (if it has one) and minus the
// row's lse.
template <class T, bool TERM>
__device__ __forceinline__ float weight(const Shape& S, float x, float term, float minus) {
  if constexpr (sizeof(T) == 4)
    return ex2((fmaf(x, S.scale, fmaf(x, S.scale_lo, term)) + minus) * (float)kLog2e);
  else
    return ex2(fmaf(x, S.c, TERM ? term + minus : minus));
}

// Writes a transposed result (column: row `row` of the output, down: its
// elements) either as a partial or rounded to T.
template <class T, int NDB>
__device__ __forceinline__ void write_cols(const f32x16 (&x)[NDB], float f, float* prow, int dp, T* orow, int d,
                                           bool vec, int h) {
#pragma unroll
  for (int n = 0; n < NDB; ++n)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int c = 32 * n + 8 * g + 4 * h;
      const f32x4 v = {f * x[n][4 * g], f * x[n][4 * g + 1], f * x[n][4 * g + 2], f * x[n][4 * g + 3]};
      if (prow) {
        if (c < dp) *(f32x4*)(prow + c) = v;
      } else if (vec) {
        store4<T, true>(orow, c, d, v);
      } else {
        store4<T, false>(orow, c, d, v);
      }
    }
}

// dQ: 4 waves of 32 rows, tiles of KT keys in two LDS buffers (as k_attend). It
// also makes the rows' statistics for k_grad_kv, as it holds dout anyway: minus
// the lse (natural units for fp32, log2 units for the 16-bit types) and D (a
// kernel of its own took 7 of 110 us at 512 x 1000 x 16 heads x 8, bf16, and one
// of seven launches).
template <class T, int W>
__global__ __launch_bounds__(256, sizeof(T) * row_width(W) <= 256 ? 2 : 1) void k_grad_q(GradArgs A) {
  constexpr int DP = row_width(W);
  using TL = Tile<T, DP>;
  using V8 = typename Vec<T>::V8;
  constexpr int KT = sizeof(T) * DP <= 256 ? 64 : 32, NT = 256, NS = W / 16, NDB = W / 32;
  using KeyT = KeyTiles<T, DP, KT, NT, 2>;
  __shared__ typename KeyT::Shared sm;

  const Shape& S = A.S;
  const int64_t pairs = (int64_t)S.batch * S.hkv;
  const int64_t item = xcd_item(pairs, A.tiles_q * A.split_q);
  if (item < 0) return;
  int64_t pair = item / (A.tiles_q * A.split_q);
  const int64_t rest = item - pair * (A.tiles_q * A.split_q);
  const int64_t tile = rest / A.split_q;
  const int split = (int)(rest - tile * A.split_q);
  const int pos = (int)(pair / S.hkv), hk = (int)(pair - (int64_t)pos * S.hkv);
  const int b = batch_entry(S, pos);
  pair = (int64_t)b * S.hkv + hk;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r32 = lane & 31;

  const int64_t nkeys = live_keys(S, b), nrows = live_rows(S, b);
  const int64_t row0 = tile * 128, row = row0 + 32 * wave + r32;
  const bool live_row = row < nrows;
  const int64_t qi = row / S.group;
  const int qh = hk * S.group + (int)(row - qi * S.group);
  const int64_t ntiles = row0 < nrows ? (nkeys + KT - 1) / KT : 0;
  const int64_t per = (ntiles + A.split_q - 1) / A.split_q;
  const int64_t t0 = split * per, t1 = t0 + per < ntiles ? t0 + per : ntiles;

  KeyT keys(sm, S, b, hk, t0, t1, nkeys, sizeof(T) == 4 ? 1.0f : (float)kLog2e, wave, lane);
  keys.begin();

  V8 qf[NS], gf[NS];
  {
    const T* qrow = (const T*)S.q + b * S.qs[0] + qi * S.qs[1] + qh * S.qs[2];
    const T* grow = (const T*)A.dout + b * A.dos[0] + qi * A.dos[1] + qh * A.dos[2];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      qf[s] = global_frag<T>(qrow, live_row && t0 < t1, s, h, S.d);
      gf[s] = global_frag<T>(grow, live_row && t0 < t1, s, h, S.dv);
    }
  }
  f32x2 st = {-kInf, 0.0f};
  if (live_row && t0 < t1) {
    const T* orow = (const T*)A.out + b * A.os[0] + qi * A.os[1] + qh * A.os[2];
    const float e = A.lse[((int64_t)b * S.hq + qh) * S.lq + qi];
    float dot = 0.0f;
    if (A.out_vec) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const V8 x = global_frag<T>(orow, true, s, h, S.dv);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf((float)x[i], (float)gf[s][i], dot);
      }
    } else {
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (16 * s + 8 * h + i < S.dv) dot = fmaf((float)orow[16 * s + 8 * h + i], (float)gf[s][i], dot);
    }
    dot = half_sum(dot);  // both lanes of a row are here
    if (e != -kInf) st = f32x2{sizeof(T) == 4 ? -e : -e * (float)kLog2e, dot};
  }
  // for k_grad_kv; a tile without live rows or keys is not read there
  if (split == 0 && h == 0 && row < A.rows_pad) A.stat[pair * A.rows_pad + row] = st;
  loads_done();
  f32x16 dq[NDB];
#pragma unroll
  for (int n = 0; n < NDB; ++n) dq[n] = zero16();

  if constexpr (TL::RB == 256) one_ahead();
  for (int it = 0; it < keys.count; ++it) {
    keys.next(it);
    const char* const tk = keys.ktile(it);
    const char* const tv = keys.vtile(it);
    const float* const term = keys.term(it);
    const bool masked = keys.masked(it);
#pragma unroll
    for (int n = 0; n < KT / 32; ++n) {
      f32x16 p = zero16(), g = zero16();
      if constexpr (TL::RB == 128) {
        V8 a[NS][2];  // all on their way before the first product, as in k_attend
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          a[s][0] = TL::row_frag(tk, 32 * n + r32, s, h);
          a[s][1] = TL::row_frag(tv, 32 * n + r32, s, h);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          p = mma(a[s][0], qf[s], p);
          g = mma(a[s][1], gf[s], g);
        }
      } else {
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          p = mma(TL::row_frag(tk, 32 * n + r32, s, h), qf[s], p);
          g = mma(TL::row_frag(tv, 32 * n + r32, s, h), gf[s], g);
        }
      }
      auto weights = [&](auto terms) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4 ct = {0, 0, 0, 0};
          if constexpr (decltype(terms)::value) ct = *(const f32x4*)&term[32 * n + 8 * q + 4 * h];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 4 * q + e;
            p[i] = weight<T, decltype(terms)::value>(S, p[i], ct[e], st[0]) * (g[i] - st[1]);
          }
        }
      };
      if (masked)
        weights(std::true_type{});
      else
        weights(std::false_type{});
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const V8 ds = pack<T>(p, s);
#pragma unroll
        for (int x = 0; x < NDB; ++x) dq[x] = mma(TL::col_frag(tk, 32 * n + 16 * s, 32 * x, lane), ds, dq[x]);
      }
    }
  }
  if (row >= S.rows) return;
  // a row without keys has no gradient, whatever dout and q hold (0 dout is NaN
  // where dout is no number)
  if (st[0] == -kInf) {
#pragma unroll
    for (int n = 0; n < NDB; ++n) dq[n] = zero16();
  }
  float* prow = A.part_q ? A.part_q + (((int64_t)split * pairs + pair) * S.rows + row) * A.dp : nullptr;
  T* orow = (T*)A.dq + b * A.dqs[0] + qi * A.dqs[1] + qh * A.dqs[2];
  write_cols<T, NDB>(dq, S.scale, prow, A.dp, orow, S.d, A.vec_q, h);
}

// dK and dV of 128 keys. Waves work in pairs on the same 32 keys: the first
// computes S and the weights P and accumulates dV = P^T dout, the second computes
// dout V^T and dS and accumulates dK = dS^T Q one tile of rows later, from the P
// that its partner left in LDS (fp32, each lane's own registers). Either holds half of
// the operands and accumulators, so two waves fit a SIMD, whose matrix and vector
// work then overlap; one wave doing all needs more than 256 registers at 128
// columns and a SIMD to itself (4096 x 8192 x 32 heads, bf16: 3.4 ms against
// 2.4). Tiles of 32 rows in a ring: the second
// wave's, the first's, and those being loaded (a tile is computed on in less
// time than memory takes to answer).
template <class T, int W>
__global__ __launch_bounds__(512, 2) void k_grad_kv(GradArgs A) {
  constexpr int DP = row_width(W);
  using TL = Tile<T, DP>;
  using V8 = typename Vec<T>::V8;
  constexpr int RT = 32, NT = 512, NS = W / 16, NDB = W / 32;
  constexpr bool AHEAD = sizeof(T) * DP <= 256;  // registers for it
  constexpr int RING = sizeof(T) * DP <= 256 ? 4 : 3;  // tiles in LDS: fp32 of 128 columns leaves no room for more
  constexpr int kTileBytes = RT * TL::RB;
  __shared__ __attribute__((aligned(16))) char sm[RING][2][kTileBytes];  // q, dout
  __shared__ __attribute__((aligned(16))) f32x4 sp[2][4][4][64];      // P: [buffer][pair][registers][lane]
  __shared__ __attribute__((aligned(16))) f32x2 sstat[RING][RT];

  const Shape& S = A.S;
  const int64_t pairs = (int64_t)S.batch * S.hkv;
  const int64_t item = xcd_item(pairs, A.tiles_kv * A.split_kv);
  if (item < 0) return;
  int64_t pair = item / (A.tiles_kv * A.split_kv);
  const int64_t rest = item - pair * (A.tiles_kv * A.split_kv);
  const int64_t tile = rest / A.split_kv;
  const int split = (int)(rest - tile * A.split_kv);
  const int pos = (int)(pair / S.hkv), hk = (int)(pair - (int64_t)pos * S.hkv);
  const int b = batch_entry(S, pos);
  pair = (int64_t)b * S.hkv + hk;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r32 = lane & 31;
  const int wp = wave & 3;
  const bool first = wave < 4;  // of its pair (waves w and w + 4 run on the same SIMD)

  const int64_t nkeys = live_keys(S, b), nrows = live_rows(S, b);
  const int64_t key0 = tile * 128, key = key0 + 32 * wp + r32;
  const float* bias = S.bias ? S.bias + b * S.bs[0] + hk * S.bs[1] : nullptr;
  const float term = column_term(bias, key, nkeys, sizeof(T) == 4 ? 1.0f : (float)kLog2e);
  const int64_t ntiles = key0 < nkeys ? (nrows + RT - 1) / RT : 0;
  const int64_t per = (ntiles + A.split_kv - 1) / A.split_kv;
  const int64_t t0 = split * per, t1 = t0 + per < ntiles ? t0 + per : ntiles;
  const int count = t1 > t0 ? (int)(t1 - t0) : 0;

  RowTiles<T, DP, RT, NT> rq(S, S.q, S.qs, b, hk, S.d, t0, nrows, wave, lane),
      rg(S, A.dout, A.dos, b, hk, S.dv, t0, nrows, wave, lane);
  auto start = [&](int n) {
    if (n >= count) return;
    const int buf = n % RING;
    rq.start(S, sm[buf][0], wave, lane);
    rg.start(S, sm[buf][1], wave, lane);
    // 32 rows of statistics, 8 bytes each (rows_pad covers the tile)
    if (wave == 0) dma_load<4>(dma_rsrc(A.stat + pair * A.rows_pad + (t0 + n) * RT), lds_offset(sstat[buf]), 4 * lane);
  };
  V8 fr[NS];  // the keys' rows of k (first) or v (second)
  {
    const T* row = first ? (const T*)S.k + b * S.ks[0] + key * S.ks[1] + hk * S.ks[2]
                         : (const T*)S.v + b * S.vs[0] + key * S.vs[1] + hk * S.vs[2];
    const bool live = term != -kInf && count > 0;  // no rows: nothing to read them for
#pragma unroll
    for (int s = 0; s < NS; ++s) fr[s] = global_frag<T>(row, live, s, h, first ? S.d : S.dv);
  }
  loads_done();
#pragma unroll
  for (int n = 0; n < RING - 2; ++n) start(n);
  f32x16 acc[NDB];  // dV (first) or dK (second), transposed
#pragma unroll
  for (int n = 0; n < NDB; ++n) acc[n] = zero16();

  using Ld = Loader<T, DP, RT, NT>;
  // Makes tile `it` readable and the weights of tile it - 1, and starts a tile.
  // Both kinds of wave call it once for each it = 0 .. count.
  auto next = [&](int it) {
    // the loads of the FLY tiles after it may be on their way
    constexpr int FLY = RING - 3;
    static_assert(Ld::N == 1 || Ld::TOTAL % Ld::NW == 0, "a wave has all of a tile's loads or none");
    if (FLY > 0 && it + FLY < count && wave == 0)
      dma_wait<FLY * (2 * Ld::N + 1)>();
    else if (FLY > 0 && it + FLY < count && Ld::has(0, wave))
      dma_wait<FLY * 2 * Ld::N>();
    else
      dma_wait<0>();
    __syncthreads();
    start(it + RING - 2);
  };
  if (first) {
    // ahead of its partner, which needs its weights (forward and backward, 4096 x
    // 8192 x 32 heads x 2: 4834 -> 4796 us; the partner ahead 4885, each product's
    // instructions ahead 5008)
    __builtin_amdgcn_s_setprio(1);
    for (int it = 0; it < count; ++it) {
      next(it);
      const char* const tq = sm[it % RING][0];
      const char* const tg = sm[it % RING][1];
      const f32x2* const stat = sstat[it % RING];
      // all fragments on their way before the first product: left alone, the
      // compiler reads one or two ahead and each product waits for LDS
      V8 ra[NS], ca[2][NDB];
#pragma unroll
      for (int s = 0; s < NS; ++s) ra[s] = TL::row_frag(tq, r32, s, h);
      if constexpr (AHEAD) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int x = 0; x < NDB; ++x) ca[s][x] = TL::col_frag(tg, 16 * s, 32 * x, lane);
        __builtin_amdgcn_sched_barrier(0);
      }
      f32x16 p = zero16();
#pragma unroll
      for (int s = 0; s < NS; ++s) p = mma(ra[s], fr[s], p);
      auto weights = [&](auto biased) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const f32x4 w = *(const f32x4*)&stat[8 * (q >> 1) + 4 * h + 2 * (q & 1)];  // two rows: {-lse, D, -lse, D}
          p[2 * q] = weight<T, decltype(biased)::value>(S, p[2 * q], term, w[0]);
          p[2 * q + 1] = weight<T, decltype(biased)::value>(S, p[2 * q + 1], term, w[2]);
        }
      };
      // without a bias the column term is 0 for every live key; what a key
      // behind the sequence gathers is dropped below
      if (bias)
        weights(std::true_type{});
      else
        weights(std::false_type{});
#pragma unroll
      for (int q = 0; q < 4; ++q) sp[it & 1][wp][q][lane] = f32x4{p[4 * q], p[4 * q + 1], p[4 * q + 2], p[4 * q + 3]};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const V8 pw = pack<T>(p, s);
#pragma unroll
        for (int x = 0; x < NDB; ++x)
          acc[x] = mma(AHEAD ? ca[s][x] : TL::col_frag(tg, 16 * s, 32 * x, lane), pw, acc[x]);
      }
    }
    next(count);
  } else {
    next(0);
    for (int it = 0; it < count; ++it) {
      next(it + 1);
      const char* const tq = sm[it % RING][0];
      const char* const tg = sm[it % RING][1];
      const f32x2* const stat = sstat[it % RING];
      V8 ra[NS], ca[2][NDB];
#pragma unroll
      for (int s = 0; s < NS; ++s) ra[s] = TL::row_frag(tg, r32, s, h);
      if constexpr (AHEAD) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int x = 0; x < NDB; ++x) ca[s][x] = TL::col_frag(tq, 16 * s, 32 * x, lane);
        __builtin_amdgcn_sched_barrier(0);
      }
      f32x16 g = zero16();
#pragma unroll
      for (int s = 0; s < NS; ++s) g = mma(ra[s], fr[s], g);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 p = sp[it & 1][wp][q][lane];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const f32x4 w = *(const f32x4*)&stat[8 * q + 4 * h + 2 * e];
          g[4 * q + 2 * e] = p[2 * e] * (g[4 * q + 2 * e] - w[1]);
          g[4 * q + 2 * e + 1] = p[2 * e + 1] * (g[4 * q + 2 * e + 1] - w[3]);
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const V8 ds = pack<T>(g, s);
#pragma unroll
        for (int x = 0; x < NDB; ++x)
          acc[x] = mma(AHEAD ? ca[s][x] : TL::col_frag(tq, 16 * s, 32 * x, lane), ds, acc[x]);
      }
    }
  }
  if (key >= S.lk) return;
  if (term == -kInf) {
#pragma unroll
    for (int n = 0; n < NDB; ++n) acc[n] = zero16();
  }
  const int64_t pi = ((int64_t)split * pairs + pair) * S.lk + key;
  if (first) {
    T* row = (T*)A.dv + b * A.dvs[0] + key * A.dvs[1] + hk * A.dvs[2];
    write_cols<T, NDB>(acc, 1.0f, A.part_v ? A.part_v + pi * A.dvp : nullptr, A.dvp, row, S.dv, A.vec_v, h);
  } else {
    T* row = (T*)A.dk + b * A.dks[0] + key * A.dks[1] + hk * A.dks[2];
    write_cols<T, NDB>(acc, S.scale, A.part_k ? A.part_k + pi * A.dp : nullptr, A.dp, row, S.d, A.vec_k, h);
  }
}

// The same for 64 columns of 16 bits, where one wave holds both operands and
// both accumulators of its 32 keys in less than 256 registers: 4 waves, tiles of
// 64 rows in two LDS buffers, half the barriers and nothing passed between
// waves (512 x 1000 x 16 heads x 8, bf16: 48 us against 60).
template <class T, int W>
__global__ __launch_bounds__(256, 2) void k_grad_kv_one(GradArgs A) {
  constexpr int DP = row_width(W);
  using TL = Tile<T, DP>;
  using V8 = typename Vec<T>::V8;
  constexpr int RT = 64, NT = 256, NS = W / 16, NDB = W / 32;
  constexpr int kTileBytes = RT * TL::RB;
  __shared__ __attribute__((aligned(16))) char sm[2][2][kTileBytes];  // q, dout
  __shared__ __attribute__((aligned(16))) f32x2 sstat[2][RT];

  const Shape& S = A.S;
  const int64_t pairs = (int64_t)S.batch * S.hkv;
  const int64_t item = xcd_item(pairs, A.tiles_kv * A.split_kv);
  if (item < 0) return;
  int64_t pair = item / (A.tiles_kv * A.split_kv);
  const int64_t rest = item - pair * (A.tiles_kv * A.split_kv);
  const int64_t tile = rest / A.split_kv;
  const int split = (int)(rest - tile * A.split_kv);
  const int pos = (int)(pair / S.hkv), hk = (int)(pair - (int64_t)pos * S.hkv);
  const int b = batch_entry(S, pos);
  pair = (int64_t)b * S.hkv + hk;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r32 = lane & 31;

  const int64_t nkeys = live_keys(S, b), nrows = live_rows(S, b);
  const int64_t key0 = tile * 128, key = key0 + 32 * wave + r32;
  const float* bias = S.bias ? S.bias + b * S.bs[0] + hk * S.bs[1] : nullptr;
  const float term = column_term(bias, key, nkeys, (float)kLog2e);
  const int64_t ntiles = key0 < nkeys ? (nrows + RT - 1) / RT : 0;
  const int64_t per = (ntiles + A.split_kv - 1) / A.split_kv;
  const int64_t t0 = split * per, t1 = t0 + per < ntiles ? t0 + per : ntiles;
  const int count = t1 > t0 ? (int)(t1 - t0) : 0;

  RowTiles<T, DP, RT, NT> rq(S, S.q, S.qs, b, hk, S.d, t0, nrows, wave, lane),
      rg(S, A.dout, A.dos, b, hk, S.dv, t0, nrows, wave, lane);
  auto start = [&](int n) {
    if (n >= count) return;
    rq.start(S, sm[n & 1][0], wave, lane);
    rg.start(S, sm[n & 1][1], wave, lane);
    // 64 rows of statistics, 8 bytes each (rows_pad covers the tile)
    if (wave < 2)
      dma_load<4>(dma_rsrc(A.stat + pair * A.rows_pad + (t0 + n) * RT), lds_offset(sstat[n & 1]) + wave * 256,
                  wave * 256 + 4 * lane);
  };
  V8 kf[NS], vf[NS];
  {
    const T* krow = (const T*)S.k + b * S.ks[0] + key * S.ks[1] + hk * S.ks[2];
    const T* vrow = (const T*)S.v + b * S.vs[0] + key * S.vs[1] + hk * S.vs[2];
    const bool live = term != -kInf && count > 0;  // no rows: nothing to read them for
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      kf[s] = global_frag<T>(krow, live, s, h, S.d);
      vf[s] = global_frag<T>(vrow, live, s, h, S.dv);
    }
  }
  loads_done();
  start(0);
  f32x16 dk[NDB], dv[NDB];
#pragma unroll
  for (int n = 0; n < NDB; ++n) {
    dk[n] = zero16();
    dv[n] = zero16();
  }
  for (int it = 0; it < count; ++it) {
    dma_wait<0>();
    __syncthreads();
    start(it + 1);
    const char* const tq = sm[it & 1][0];
    const char* const tg = sm[it & 1][1];
    const f32x2* const stat = sstat[it & 1];
#pragma unroll
    for (int n = 0; n < RT / 32; ++n) {
      f32x16 p = zero16(), g = zero16();
      V8 a[NS][2];  // all on their way before the first product, as in k_attend
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        a[s][0] = TL::row_frag(tq, 32 * n + r32, s, h);
        a[s][1] = TL::row_frag(tg, 32 * n + r32, s, h);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        p = mma(a[s][0], kf[s], p);
        g = mma(a[s][1], vf[s], g);
      }
      auto weights = [&](auto biased) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const f32x4 w = *(const f32x4*)&stat[32 * n + 8 * (q >> 1) + 4 * h + 2 * (q & 1)];  // {-lse, D, -lse, D}
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = 2 * q + e;
            p[i] = weight<T, decltype(biased)::value>(S, p[i], term, w[2 * e]);
            g[i] = p[i] * (g[i] - w[2 * e + 1]);
          }
        }
      };
      if (bias)
        weights(std::true_type{});
      else
        weights(std::false_type{});  // as in k_grad_kv
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const V8 pw = pack<T>(p, s), ds = pack<T>(g, s);
#pragma unroll
        for (int x = 0; x < NDB; ++x) {
          dv[x] = mma(TL::col_frag(tg, 32 * n + 16 * s, 32 * x, lane), pw, dv[x]);
          dk[x] = mma(TL::col_frag(tq, 32 * n + 16 * s, 32 * x, lane), ds, dk[x]);
        }
      }
    }
  }
  if (key >= S.lk) return;
  if (term == -kInf) {
#pragma unroll
    for (int n = 0; n < NDB; ++n) {
      dk[n] = zero16();
      dv[n] = zero16();
    }
  }
  const int64_t pi = ((int64_t)split * pairs + pair) * S.lk + key;
  T* dkrow = (T*)A.dk + b * A.dks[0] + key * A.dks[1] + hk * A.dks[2];
  T* dvrow = (T*)A.dv + b * A.dvs[0] + key * A.dvs[1] + hk * A.dvs[2];
  write_cols<T, NDB>(dk, S.scale, A.part_k ? A.part_k + pi * A.dp : nullptr, A.dp, dkrow, S.d, A.vec_k, h);
  write_cols<T, NDB>(dv, 1.0f, A.part_v ? A.part_v + pi * A.dvp : nullptr, A.dvp, dvrow, S.dv, A.vec_v, h);
}

// Adds the partial sums of a gradient in split order: 32 lanes per row. Rows of
// dQ are packed (group > 1); rows of dK, dV are keys (group = 1).
struct GradJoin {
  const float* part;
  int64_t rows;
  int32_t nsplit, dp, group, d;
  void* out;
  int64_t s[3];
  bool vec;
};
struct GradJoins {
  GradJoin g[3];
  int64_t pairs;
  int32_t hkv;
};

template <class T>
__global__ __launch_bounds__(256) void k_grad_join(GradJoins all) {
  const GradJoin& J = all.g[blockIdx.y];
  const int64_t n = all.pairs * J.rows;
  const int64_t idx = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int c = 4 * (threadIdx.x & 31);
  if (idx >= n || c >= J.dp) return;
  const int64_t pair = idx / J.rows, row = idx - pair * J.rows;
  const int b = (int)(pair / all.hkv), hk = (int)(pair - (int64_t)b * all.hkv);
  f32x4 x = {0, 0, 0, 0};
  for (int s = 0; s < J.nsplit; ++s) {
    const f32x4 v = *(const f32x4*)(J.part + (s * n + idx) * J.dp + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] += v[e];
  }
  const int64_t qi = row / J.group;
  const int qh = hk * J.group + (int)(row - qi * J.group);
  T* orow = (T*)J.out + b * J.s[0] + qi * J.s[1] + qh * J.s[2];
  if (J.vec)
    store4<T, true>(orow, c, J.d, x);
  else
    store4<T, false>(orow, c, J.d, x);
}

template <class T, int W>
void grad_launch(const GradArgs& A, hipStream_t st) {
  const int64_t pairs = (int64_t)A.S.batch * A.S.hkv;
  if (A.S.rows > 0) {
    hipLaunchKernelGGL((k_grad_q<T, W>), grid1(xcd_blocks(pairs, A.tiles_q * A.split_q), 256), dim3(256), 0, st, A);
    SK_LAUNCH_CHECK();
  }
  if (A.S.lk > 0) {
    const int64_t items = xcd_blocks(pairs, A.tiles_kv * A.split_kv);
    if constexpr (row_width(W) * sizeof(T) == 128)
      hipLaunchKernelGGL((k_grad_kv_one<T, W>), grid1(items, 256), dim3(256), 0, st, A);
    else
      hipLaunchKernelGGL((k_grad_kv<T, W>), grid1(items, 512), dim3(512), 0, st, A);
    SK_LAUNCH_CHECK();
  }
}

// Instantiated once per element type (attend_grad_*.hip).
template <class T>
void attend_grad(const GradArgs& A, hipStream_t st) {
  const int64_t pairs = (int64_t)A.S.batch * A.S.hkv;
  by_width(A.S.d, A.S.dv, [&](auto w) { grad_launch<T, decltype(w)::value>(A, st); });
  GradJoins all{};
  all.pairs = pairs;
  all.hkv = A.S.hkv;
  unsigned n = 0;
  int64_t most = 0;
  auto join = [&](const float* part, int nsplit, int64_t rows, int32_t dp, int32_t group, void* out, const int64_t* s,
                  int32_t d, bool vec) {
    if (!part || rows == 0) return;
    all.g[n++] = GradJoin{part, rows, nsplit, dp, group, d, out, {s[0], s[1], s[2]}, vec};
    most = rows > most ? rows : most;
  };
  join(A.part_q, A.split_q, A.S.rows, A.dp, A.S.group, A.dq, A.dqs, A.S.d, A.vec_q);
  join(A.part_k, A.split_kv, A.S.lk, A.dp, 1, A.dk, A.dks, A.S.d, A.vec_k);
  join(A.part_v, A.split_kv, A.S.lk, A.dvp, 1, A.dv, A.dvs, A.S.dv, A.vec_v);
  if (n > 0) {
    dim3 grid = grid1((pairs * most + 7) / 8, 256);
    grid.y = n;
    hipLaunchKernelGGL((k_grad_join<T>), grid, dim3(256), 0, st, all);
    SK_LAUNCH_CHECK();
  }
}

}  // namespace attn
}  // namespace sk
