// The attention weight that each key gathers over the rows and heads that
// read it:  mass_out_j = mass_in_j + sum_r w_r exp(s_rj - lse_r).
//
// k_mass holds keys (a wave has 32 across) and runs over rows: one product and
// one exponential per score, the sum over rows in a lane's own registers.
// Rows are split over workgroups when the keys do not fill the chip; partial
// sums are added in split order by k_mass_join. No atomics.
//
// For a single tile of rows (decoding) the forward kernel leaves its scores in
// a workspace and k_mass_scores reads those: keys are then read once from
// memory, by the forward pass.
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
  const float* scores;    // of the forward kernel (k_mass_scores)
  int64_t score_ld;
  bool exact;             // scores in natural units (fp32), else log2 units
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
