// The attention weight that each key gathers over the rows and heads that
// read it:  mass_out_j = mass_in_j + sum_r w_r exp(s_rj - lse_r).
//
// k_mass holds keys (a wave has 32 across) and runs over rows: one product and
// one exponential per score, the sum over rows in a lane's own registers.
// Rows are split over workgroups when the keys do not fill the chip; partial
// sums are added in split order by k_mass_join. No atomics.
//
// For a single tile of rows (decoding) the forward kernel leaves its scores in
// a workspace and weight_keys reads those: keys are then read once from memory,
// by the forward pass. Where that was split, it runs beside the join of the
// splits (attend.h), from the splits' references and sums: one launch less
// (24 -> 21 us for 5 x 4097 x 12 heads x 3).
#pragma once

#include <type_traits>

#include "attention.h"

namespace sk {
namespace attn {

struct MassArgs {
  Shape S;
  const float* lse;       // [batch][hq][lq]
  const float* weight;    // [batch][lq], nullable: 1
  const float* mass_in;   // [batch][hkv][lk], nullable: 0
  float* mass_out;        // [batch][hkv][lk], may be mass_in
  float* part;            // [split][batch * hkv][lk], nullable
  f32x2* stat;            // [batch * hkv][rows_pad]: minus lse (-inf: the row takes no part), weight
  int64_t rows_pad;       // rows rounded up to 64
  int32_t nsplit;
  int64_t tiles;
  const float* scores;    // of the forward kernel, nullable
  int64_t score_ld;
  bool exact;             // scores in natural units (fp32), else log2 units
  bool deal;              // weight_keys: 256 keys and four groups of rows a workgroup, else 1024 keys
};

// A row's log-sum-exp (+inf: the row takes no part) and weight. In log2 units
// unless `natural`; what the fp32 product lse log2e rounds off goes into the
// weight.
__device__ __forceinline__ f32x2 mass_row(const MassArgs& A, int b, int hk, int64_t row, int64_t nrows, bool natural) {
  const Shape& S = A.S;
  if (row >= nrows) return f32x2{kInf, 0.0f};
  const uint32_t qi = (uint32_t)row / (uint32_t)S.group;  // rows below 2^31
  const int qh = hk * S.group + (int)((uint32_t)row - qi * S.group);
  const float e = A.lse[((int64_t)b * S.hq + qh) * S.lq + qi];
  const float w = A.weight ? A.weight[b * S.lq + qi] : 1.0f;
  if (e == -kInf) return f32x2{kInf, w};
  if (natural) return f32x2{e, w};
  const float t = e * (float)kLog2e;
  const float lost = fmaf(e, (float)kLog2e, -t) + e * (float)(kLog2e - (double)(float)kLog2e);
  return f32x2{t, w * ex2(-lost)};
}

// The weight of block `blk`'s keys from the forward kernel's scores of the pair's
// rows (32 at most), four keys a thread: 1024 keys, or, where that leaves the chip
// empty, 256 with the rows dealt to four groups of 64 threads (16 x 8 x 32768
// keys, 4 rows: join and weight 21 us with 1024 keys, 30 with 256; 3 x 4 x 4097
// keys, 15 rows: 5.3 us with 256, with 1024 the weight alone took 6.2). rows(...)
// puts each row's reference (log2 units) and the factor of its weights into LDS.
// lo: what the fp32 log2e misses, where the references were made without that
// loss (else it cancels).
template <class F>
__device__ __forceinline__ void weight_keys(const MassArgs& A, int64_t blk, float lo, F&& rows) {
  __shared__ f32x2 srow[32];
  __shared__ f32x4 sx[3][64];
  const Shape& S = A.S;
  const bool deal = A.deal;
  const int64_t chunks = (S.lk + (deal ? 255 : 1023)) / (deal ? 256 : 1024);
  const int64_t pair = blk / chunks;
  const int b = (int)(pair / S.hkv), hk = (int)(pair - (int64_t)b * S.hkv);
  const int t = threadIdx.x & 63, g = threadIdx.x >> 6, step = deal ? 4 : 1;
  const int64_t j = (blk - pair * chunks) * (deal ? 256 : 1024) + 4 * (deal ? t : (int)threadIdx.x);
  const int64_t nkeys = live_keys(S, b), nrows = live_rows(S, b);
  rows(srow, pair, b, hk, nrows);
  __syncthreads();
  f32x4 x = {0, 0, 0, 0};
  const float f = A.exact ? (float)kLog2e : 1.0f;
  if (j < nkeys) {
    // the forward kernel wrote whole tiles of the live keys
    const float* sc = A.scores + S.rows * (pair * A.score_ld + (j & ~int64_t(31))) + (j & 31);
    for (int r = deal ? g : 0; r < (int)nrows; r += step) {
      const f32x4 v = *(const f32x4*)(sc + 32 * r);
      const f32x2 st = srow[r];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = fmaf(st[1], ex2(fmaf(v[e], f, lo > 0.0f ? fmaf(v[e], lo, -st[0]) : -st[0])), x[e]);
    }
  }
  if (deal) {
    if (g > 0) sx[g - 1][t] = x;
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const f32x4 y = sx[k][t];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] += y[e];
    }
  }
  // by the mask itself, as a masked key's weight is NaN under a row that is no number
  const float* bias = S.bias ? S.bias + b * S.bs[0] + hk * S.bs[1] : nullptr;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (j + e < S.lk) {
      const int64_t i = pair * S.lk + j + e;
      const bool live = column_term(bias, j + e, nkeys, 1.0f) != -kInf;
      A.mass_out[i] = (A.mass_in ? A.mass_in[i] : 0.0f) + (live ? x[e] : 0.0f);
    }
}
inline int64_t weight_blocks(const MassArgs& A) {
  return (int64_t)A.S.batch * A.S.hkv * ((A.S.lk + (A.deal ? 255 : 1023)) / (A.deal ? 256 : 1024));
}

// Bound by the vector work of a score (an exponential, two fma) beside its product:
// 2 x 2048 x 8191 keys, 16 heads of 128 on 4, bf16: 158 us, 870 TFLOP/s. Three
// waves a SIMD where the registers allow it without spilling (96 columns: two); the
// products of both 32-row blocks ahead of the first's weights spill: 164 us.
template <class T, int W>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? (W == 96 ? 2 : 3) : 1) void k_mass(MassArgs A) {
  constexpr int DP = row_width(W);
  using TL = Tile<T, DP>;
  using V8 = typename Vec<T>::V8;
  constexpr int RT = 64, NT = 256, NS = W / 16;
  constexpr bool kExact = sizeof(T) == 4;  // scores in natural units, rounded once
  constexpr int kTileBytes = RT * TL::RB;
  __shared__ __attribute__((aligned(16))) char sm[2 * kTileBytes];
  __shared__ __attribute__((aligned(16))) f32x2 sstat[2][RT];

  const Shape& S = A.S;
  const int64_t pairs = (int64_t)S.batch * S.hkv;
  const int64_t item = xcd_item(pairs, A.tiles * A.nsplit);
  if (item < 0) return;
  const int64_t pair = item / (A.tiles * A.nsplit);
  const int64_t rest = item - pair * (A.tiles * A.nsplit);
  const int64_t tile = rest / A.nsplit;
  const int split = (int)(rest - tile * A.nsplit);
  const int b = (int)(pair / S.hkv), hk = (int)(pair - (int64_t)b * S.hkv);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r32 = lane & 31;

  const int64_t nkeys = live_keys(S, b), nrows = live_rows(S, b);
  const int64_t key0 = tile * 128, key = key0 + 32 * wave + r32;
  const float* bias = S.bias ? S.bias + b * S.bs[0] + hk * S.bs[1] : nullptr;
  const float term = column_term(bias, key, nkeys, kExact ? 1.0f : (float)kLog2e);
  const int64_t ntiles = key0 < nkeys ? (nrows + RT - 1) / RT : 0;
  const int64_t per = (ntiles + A.nsplit - 1) / A.nsplit;
  const int64_t t0 = split * per, t1 = t0 + per < ntiles ? t0 + per : ntiles;

  RowTiles<T, DP, RT, NT> rows(S, S.q, S.qs, b, hk, S.d, t0, nrows, wave, lane);
  auto start = [&](int64_t t) {
    const int buf = (int)(t - t0) & 1;
    rows.start(S, sm + buf * kTileBytes, wave, lane);
    // 64 rows of statistics, 8 bytes each (rows_pad covers the tile)
    if (wave < 2)
      dma_load<4>(dma_rsrc(A.stat + pair * A.rows_pad + t * RT), lds_offset(sstat[buf]) + wave * 256, wave * 256 + 4 * lane);
  };
  V8 kf[NS];
  {
    const T* krow = (const T*)S.k + b * S.ks[0] + key * S.ks[1] + hk * S.ks[2];
#pragma unroll
    for (int s = 0; s < NS; ++s) kf[s] = global_frag<T>(krow, term != -kInf && t0 < t1, s, h, S.d);
  }
  loads_done();
  if (t0 < t1) start(t0);
  float sum = 0.0f;
  for (int64_t t = t0; t < t1; ++t) {
    const int buf = (int)(t - t0) & 1;
    dma_wait<0>();
    __syncthreads();
    if (t + 1 < t1) start(t + 1);
    const char* tq = sm + buf * kTileBytes;
    // without a bias the column term is 0 for every live key
    auto tile = [&](auto biased) {
#pragma unroll
      for (int n = 0; n < RT / 32; ++n) {
        f32x16 p = zero16();
#pragma unroll
        for (int s = 0; s < NS; ++s) p = mma(TL::row_frag(tq, 32 * n + r32, s, h), kf[s], p);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          // two rows: {-lse, weight, -lse, weight}
          const f32x4 w = *(const f32x4*)&sstat[buf][32 * n + 8 * (q >> 1) + 4 * h + 2 * (q & 1)];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = p[2 * q + e];
            float a;
            if constexpr (kExact)
              a = (fmaf(x, S.scale, fmaf(x, S.scale_lo, term)) + w[2 * e]) * (float)kLog2e;
            else
              a = fmaf(x, S.c, decltype(biased)::value ? term + w[2 * e] : w[2 * e]);
            sum = fmaf(w[2 * e + 1], ex2(a), sum);
          }
        }
      }
    };
    if (bias)
      tile(std::true_type{});
    else
      tile(std::false_type{});
  }
  sum = term == -kInf ? 0.0f : half_sum(sum);
  if (h != 0 || key >= S.lk) return;
  if (A.part)
    A.part[((int64_t)split * pairs + pair) * S.lk + key] = sum;
  else
    A.mass_out[pair * S.lk + key] = (A.mass_in ? A.mass_in[pair * S.lk + key] : 0.0f) + sum;
}

// Instantiated once per element type (attend_mass_*.hip).
template <class T>
void attend_mass(const MassArgs& A, hipStream_t st) {
  const dim3 grid = grid1(xcd_blocks((int64_t)A.S.batch * A.S.hkv, A.tiles * A.nsplit), 256);
  by_width(A.S.d, 1, [&](auto w) {
    hipLaunchKernelGGL((k_mass<T, decltype(w)::value>), grid, dim3(256), 0, st, A);
  });
  SK_LAUNCH_CHECK();
}

}  // namespace attn
}  // namespace sk
