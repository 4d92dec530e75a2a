// Attention of new tokens over a paged cache: row i of an entry's n new tokens is at
// place p = keys - n + i of its sequence and sees key j <= p, and of these, with
// `recent`, only j > p - recent or j < first.
//
// The tiles, the softmax and the split of the keys are those of k_attend (attend.h),
// with the differences below. (Their code stands here as functions; k_attend keeps its
// own in line: called as functions they cost it 1 to 3% in fp32, 20000 x 24001 at 50
// columns 996 -> 1009 to 1033 us.)
//
// Pages. A wave loads a tile's rows in groups of 8, which lie in one page because page
// sizes are multiples of 8: a group's address goes into the scalar base of its loads,
// so a lane's offsets are the same in every tile and a cache may be of any size. The
// addresses of 64 groups, of the next 16 tiles or 32, are made side by side in the
// lanes of a vector register and read from there lane by lane. (Made one by one in
// scalar registers for each tile they took the longer part of a tile's time with few
// rows, 16 x 32768 keys x 8 heads 326 -> 276 us side by side; tile by tile, ahead of its
// loads, they cost the chunk of 2048 over 16384 keys x 32 heads 574 -> 548 us.)
//
// Few rows: a wave loads the keys that it computes on itself, k and v in turn, and the
// waves of a workgroup meet only at the end.
//
// Masks are of the pair, but only in tiles at the rows' own places and at the
// window's edge; tiles that no row of the workgroup sees are not loaded, and waves
// leave out those that none of their rows sees. A hidden key's score becomes
// -infinity, its weight 0; a value there that is no number must not reach the row
// through 0 x infinity, so the workgroup first looks through such a tile for any (a
// share each, 2 operations per 4 bytes, and a barrier). If there is one, those values
// are added, key by key, to the rows that see them, and 0 takes their places.
//
// Order. The rows at the end of a chunk see the most keys: their tiles come first.
#pragma once

#include "attend.h"
#include "pages.h"

namespace sk {
namespace attn {

// Rows of a workgroup: 128, or 32 with the keys of a step dealt to its waves; these alone
// on a compute unit with all keys.
enum class PagedForm { kMany, kFew, kAlone };

struct PagedArgs {
  AttendArgs A;  // S.k, S.v: the cache; S.ks, S.vs: page, slot, head; S.klen: P.lengths
  Paging P;
  int32_t first, recent;  // recent 0: all keys
  int32_t rows, tiles, per;  // rows and row tiles of a pair, tiles times splits
  Divide by_group, by_heads, by_per, by_split;
  bool qvec;              // q may be read 16 bytes a lane
  bool pair_up;           // long and short row tiles together
};

// The tiles of KT keys that a workgroup runs over: `ns` from the sequence's start on,
// then those from tile t_lo on; of all these, `count` from the n0-th on. A wave loads
// RW consecutive rows of a tile.
//
// Many rows: two buffers, k and v in each; tile n + 1 is started while all waves
// compute on tile n. Few rows (PLACES > 0): a wave's rows are those that it computes on,
// so waves do not wait for each other, and k and v take turns in a ring of PLACES places
// of the wave's own: k of tile n is half 2 n of the run, v half 2 n + 1, and while one
// is computed on, those behind it are in flight.
template <class T, int DP, int KT, int NT, int PLACES>
struct PageTiles {
  static constexpr bool OWN = PLACES > 0;
  using TL = Tile<T, DP>;
  static constexpr int NW = NT / 64, RW = KT / NW;
  static constexpr int kTileBytes = KT * TL::RB, kOwnBytes = RW * TL::RB;
  static constexpr int RPI = 64 / TL::CPR;               // rows of an instruction
  static constexpr int IPO = 8 / RPI;                    // instructions for 8 rows, which lie in one page
  static constexpr int N = RW / RPI;                     // instructions of a wave for k, and for v
  static constexpr int KIND = N < 2 * IPO ? N : 2 * IPO;  // the chunks' permutation repeats after 16 rows
  static constexpr int GROUPS = RW / 8;                  // of 8 rows, of a wave
  static constexpr int BATCH = 64 / GROUPS;              // tiles whose groups fill a wave's lanes
  static_assert(KT % NW == 0 && RW % 16 == 0 && IPO >= 1 && BATCH * GROUPS == 64 && BATCH > 2, "whole groups of 8 rows");
  struct Shared {
    __attribute__((aligned(16))) char tiles[(OWN ? PLACES : 4) * kTileBytes];
    uint64_t fine[2][NW];  // `fine` of each wave, of this batch of tiles and the next
    int odd;  // the last tile, counted from 1, that was found to hold values that are no numbers
  };
  Shared& sm;
  const Paging& P;
  const char* k;
  const char* v;
  int64_t kpage, vpage;  // bytes
  uint32_t kslot, vslot;
  const int32_t* table;
  uint32_t koff[KIND], voff[KIND];  // byte offset of this lane's chunk from its 8 rows' start
  uint64_t kat, vat;  // lane i: address of the wave's group i % GROUPS of the batch's tile i / GROUPS
  uint64_t ok;        // bit i: it lies in the cache
  uint64_t fine;      // bit i: it does, or is behind the keys
  int nkeys, n0, count, ns, t_lo, wave, lane;

  __device__ __forceinline__ PageTiles(Shared& sm_, const PagedArgs& A, int b, int hk, int nkeys_, int ns_, int t_lo_, int n0_,
                                       int count_, int wave_, int lane_)
      : sm(sm_), P(A.P), k((const char*)A.A.S.k + (int64_t)hk * A.A.S.ks[2] * sizeof(T)),
        v((const char*)A.A.S.v + (int64_t)hk * A.A.S.vs[2] * sizeof(T)), kpage(A.A.S.ks[0] * sizeof(T)),
        vpage(A.A.S.vs[0] * sizeof(T)), kslot((uint32_t)(A.A.S.ks[1] * sizeof(T))), vslot((uint32_t)(A.A.S.vs[1] * sizeof(T))),
        table(A.P.table + b * A.P.stride), nkeys(nkeys_), n0(n0_), count(count_), ns(ns_), t_lo(t_lo_), wave(wave_), lane(lane_) {
#pragma unroll
    for (int i = 0; i < KIND; ++i) {
      const int r = i * RPI + lane / TL::CPR, c = (lane % TL::CPR) ^ TL::swz(r);
      koff[i] = c * TL::EPC < A.A.S.d ? r % 8 * kslot + 16 * c : kOutside;
      voff[i] = c * TL::EPC < A.A.S.dv ? r % 8 * vslot + 16 * c : kOutside;
    }
  }
  // first key of tile n
  __device__ __forceinline__ int key(int n) const {
    const int x = n0 + n;
    return (int)((uint32_t)(x < ns ? x : x - ns + t_lo) * KT);
  }
  // Addresses for the batch of tiles that begins with tile n.
  __device__ __forceinline__ void locate(int n) {
    const int t = n + lane / GROUPS;
    const uint32_t j = (uint32_t)key(t) + wave * RW + 8 * (lane % GROUPS);  // behind the last tile it may pass 2^31
    const bool live = t < count && j < (uint32_t)nkeys;
    uint32_t slot = 0;
    int32_t at = 0;
    if (live) {
      const uint32_t page = P.page(j);
      slot = j - page * (uint32_t)P.size;
      at = table[page];
    }
    const bool in = live && (uint32_t)at < (uint32_t)P.pages;
    at = in ? at : 0;
    kat = (uint64_t)k + (uint64_t)at * (uint64_t)kpage + (uint64_t)slot * kslot;
    vat = (uint64_t)v + (uint64_t)at * (uint64_t)vpage + (uint64_t)slot * vslot;
    ok = __ballot(in);
    fine = __ballot(in || !live);
    if constexpr (!OWN)
      if (lane == 0) sm.fine[n / BATCH % 2][wave] = fine;
  }
  // A scalar register that a vector instruction has written may be read by a memory
  // instruction five wait states later; the compiler does not see the loads in assembly.
  __device__ __forceinline__ static __amdgpu_buffer_rsrc_t rsrc_of(uint64_t at, int i) {
    uint32_t a = __builtin_amdgcn_readlane((uint32_t)at, i), b = __builtin_amdgcn_readlane((uint32_t)(at >> 32), i);
    asm volatile("s_nop 4" : "+s"(a), "+s"(b));
    return __builtin_amdgcn_make_buffer_rsrc((void*)((uint64_t)b << 32 | a), 0, (int)kOutside, 0x00027000);
  }
  // Starts the wave's rows of k or v of tile n, whose batch is located, to the wave's part at `to`.
  __device__ __forceinline__ void load(int n, uint64_t base, const uint32_t (&off)[KIND], const char* to) const {
    const int at = n % BATCH * GROUPS;
    const int mine = nkeys - __builtin_amdgcn_readfirstlane(key(n)) - wave * RW;  // keys from this wave's first row on
    const uint32_t lds = lds_offset(to);
    constexpr uint64_t kAll = (uint64_t(1) << GROUPS) - 1;
    auto all = [&](auto&& live) {
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const __amdgpu_buffer_rsrc_t r = rsrc_of(base, at + g);
#pragma unroll
        for (int s = 0; s < IPO; ++s) {
          const int i = g * IPO + s;
          dma_load<16, OWN>(r, lds + i * 1024, live(g, i * RPI + lane / TL::CPR) ? off[i % KIND] : kOutside);
        }
      }
    };
    if (mine >= RW && (ok >> at & kAll) == kAll)
      all([](int, int) { return true; });
    else
      all([&](int g, int r) { return (ok >> (at + g) & 1) != 0 && r < mine; });
  }
  __device__ __forceinline__ char* place(int half) const { return sm.tiles + (PLACES * wave + half % (OWN ? PLACES : 1)) * kOwnBytes; }
  // Where k and v of tile n lie: with OWN the wave's rows of it.
  __device__ __forceinline__ const char* ktile(int n) const {
    return OWN ? place(2 * n) : sm.tiles + n % 2 * 2 * kTileBytes;
  }
  __device__ __forceinline__ char* vtile(int n) const {
    return OWN ? place(2 * n + 1) : sm.tiles + (n % 2 * 2 + 1) * kTileBytes;
  }
  __device__ __forceinline__ void start_k(int n) {
    if (n >= count) return;
    if (n % BATCH == 0) locate(n);
    load(n, kat, koff, ktile(n) + (OWN ? 0 : wave * kOwnBytes));
  }
  __device__ __forceinline__ void start_v(int n) {
    if (n < count) load(n, vat, voff, vtile(n) + (OWN ? 0 : wave * kOwnBytes));
  }
  __device__ __forceinline__ void begin() {
    if (wave == 0) sm.odd = 0;  // read behind the first tile's barrier
    start_k(0);
    start_v(0);
#pragma unroll
    for (int half = 2; half < PLACES; ++half) start(half);
  }
  // Few rows: starts a half of the run.
  __device__ __forceinline__ void start(int half) {
    if (half & 1)
      start_v(half >> 1);
    else
      start_k(half >> 1);
  }
  // Waits for the wave's reads of LDS, before a load goes to where they were.
  __device__ __forceinline__ static void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

  // Many rows: makes tile n readable and starts the next one. Returns whether the
  // batch has pages outside the cache, asked at its first tile.
  __device__ __forceinline__ bool next(int n, bool bad) {
    dma_wait<0>();
    __syncthreads();
    if (n % BATCH == 0) {
      uint64_t all = ~uint64_t(0);
#pragma unroll
      for (int w = 0; w < NW; ++w) all &= sm.fine[n / BATCH % 2][w];
      bad = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)all & (uint32_t)(all >> 32)) != ~0u;
    }
    start_k(n + 1);
    start_v(n + 1);
    return bad;
  }
  // Few rows: waits for a half; those behind it, of which PLACES - 1 are started, stay in flight.
  __device__ __forceinline__ void wait(int half) const {
    const int behind = 2 * count - 1 - half;
    if (PLACES > 2 && behind >= 2)
      dma_wait<2 * N>();
    else if (behind >= 1)
      dma_wait<N>();
    else
      dma_wait<0>();
  }
  // Of a batch that has bad pages: are the 8 keys from row r of tile n on in the cache
  // (or behind the keys)? With OWN r is the wave's own and `own` its `fine`.
  __device__ __forceinline__ bool in_cache(int n, int r, uint64_t own) const {
    const int bit = n % BATCH * GROUPS + r % RW / 8;
    if constexpr (OWN) return (own >> bit & 1) != 0;
    return (sm.fine[n / BATCH % 2][r / RW] >> bit & 1) != 0;
  }
};

// Few rows: waves of a workgroup, one for each SIMD; by the bytes of a row, workgroups
// of a compute unit that the keys are split for, and places of a wave's ring. With 32
// keys a place, two places leave room for four waves of the widest rows and a second
// workgroup of 256-byte ones; three keep more in flight for rows of 128 bytes, which are
// done with sooner. Against k and v of whole tiles in two buffers (two waves of the
// widest rows): 8 x 16384 keys x 8 heads of 128 fp32 387 -> 205 us, of 64 134 -> 106,
// 64 x 2048 x 8 of 128 bf16 78 -> 71, 16 x 32768 x 8 265 -> 262 (three places 264), of 64
// 163 -> 157 (two places 163). Splits for a second workgroup of 256-byte rows: 26.0 for
// 27.1 us and 0.4 less for the least calls, 20.8 for 17.9 of 64 columns, 265 for 262.
// A workgroup that has a compute unit and all keys of its rows to itself takes twice the
// waves where LDS holds their rings: 32 pairs of 64 columns bf16 over 500 keys 8.7 us
// (four waves 9.9), over 1000 11.3 (14.3), of 128 14.2 (16.7).
constexpr int kPagedWaves = 4;
constexpr int alone_waves(int64_t bytes) { return bytes <= 256 ? 2 * kPagedWaves : kPagedWaves; }
constexpr int paged_groups(int64_t bytes) { return bytes <= 128 ? 2 : 1; }
constexpr int paged_places(int64_t bytes) { return bytes <= 128 ? 3 : 2; }

// sc = the products of keys kb0 .. of the tile (down) with the lane's row of q (across).
template <class T, int DP, bool AHEAD, int NB, int NS>
__device__ __forceinline__ void score_tile(const char* tk, int kb0, int lane, const typename Vec<T>::V8 (&qf)[NS], int d,
                                           f32x16 (&sc)[NB]) {
  using TL = Tile<T, DP>;
  using V8 = typename Vec<T>::V8;
  const int h = lane >> 5, r32 = lane & 31;
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
      for (int n = 0; n < NB; ++n)
        sc[n] = s + 2 < NS ? mma(TL::row_frag(tk, kb0 + 32 * n + r32, s, h), qf[s], sc[n])
                           : mma_first(TL::row_frag(tk, kb0 + 32 * n + r32, s, h), qf[s], sc[n], d - 16 * s);
  }
}

// fp16 holds weights below 2^-14 in steps of 2^-24, and none below 2^-25: thousands of
// them that together matter would be lost. Its reference lies 2^7 below the maximum,
// so that they begin at 2^-21 and 2^-32 of it (the largest weight, 2^15, is within
// fp16); a power of two moves nothing else. bf16 has fp32's range.
template <class T>
constexpr float kLift = std::is_same<T, _Float16>::value ? 7.0f : 0.0f;

// One tile's scores of a row become weights 2^(f sc - m); m, the sum l and the
// result o follow the running reference.
template <class T, int NB, int NDB>
__device__ __forceinline__ void soften(f32x16 (&sc)[NB], float f, float& m, float& l, f32x16 (&o)[NDB]) {
  float mx = -kInf;
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int e = 0; e < 16; ++e) mx = fmaxf(mx, sc[n][e]);
  mx = half_max(mx) * f;
  // a new reference only where the maximum rose by more than 2^8: weights stay
  // below 2^8 (2^15 with kLift) and the accumulators are seldom rescaled. Each row by
  // its own maximum: the others of the wave keep their reference, and so their
  // roundings, whatever this row's keys, which they may not see, hold
  const bool rose = mx - m > 8.0f + kLift<T>;  // (an exact difference where it is that small)
  if (__any(rose)) {
    const float mn = rose ? mx - kLift<T> : m;
    const float a = rose ? ex2(m - mn) : 1.0f;
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
}

// o += weights times the values of keys kb0 .. of the tile. With few rows, which wait for
// memory, not for products, weights of 16-bit types go in two parts, so that a token's
// result is off by its own rounding alone. With MANY a weight is rounded once, to the
// type: half a step each (2^-9 to 2^-8 of it in bf16), which over a row adds about as much
// as the result's own rounding (bf16 0.0022 relative to 64 bits in place of 0.0017). A
// second part costs a third: 2048 rows over 16384 keys x 32 heads of 128 567 -> 753 us,
// prompts of 8192 x 32 heads of 64 under a window 115 -> 151, 4 x 512 over 4096 158 -> 204.
template <class T, int DP, bool MANY, int NB, int NDB>
__device__ __forceinline__ void add_values(const char* tv, int kb0, int lane, const f32x16 (&sc)[NB], f32x16 (&o)[NDB]) {
  using V8 = typename Vec<T>::V8;
  using TL = Tile<T, DP>;
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const V8 p = pack<T>(sc[n], s);
      if constexpr (!MANY && sizeof(T) == 2) {
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

// Writes the rows of a workgroup: o (not divided by the sum), reference m and
// sum l of this lane's row, or zeros without `has`; as a partial result where the
// keys are split. With few rows the waves' parts of the keys are joined through
// so [WK][W][32] and sml [WK][32] first.
template <class T, int W, int WQ, int WK>
__device__ __forceinline__ void finish_rows(const PagedArgs& G, float* so, f32x2* sml, const f32x16 (&o)[W / 32], float m,
                                            float l, bool has, int split, int b, int hk, int row0) {
  constexpr bool MANY = WQ > 1;
  constexpr int NDB = W / 32, NT = 64 * WQ * WK;
  const AttendArgs& A = G.A;
  const Shape& S = A.S;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r32 = lane & 31;
  const int wq = wave % WQ, wk = wave / WQ;
  // partial results of this split and pair start at this row
  const int64_t part0 = ((int64_t)split * (S.batch * S.hkv) + b * S.hkv + hk) * G.rows;
  // the row's result, column group by column group: group index c4 of four
  // columns, value x (not divided by the sum)
  const bool part = A.opart != nullptr;
  if constexpr (!MANY) {
    __syncthreads();
    if (h == 0) sml[wk * 32 + r32] = f32x2{m, l};
#pragma unroll
    for (int x = 0; x < NDB; ++x)
#pragma unroll
      for (int e = 0; e < 16; ++e) so[(wk * W + 32 * x + 8 * (e >> 2) + 4 * h + (e & 3)) * 32 + r32] = has ? o[x][e] : 0.0f;
    __syncthreads();
    // thread: row tid % 32, column groups tid / 32, + NT / 32, ...
    const int jrow = row0 + (tid & 31);
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
    if (jrow >= G.rows) return;
    const int ji = (int)G.by_group((uint32_t)jrow), jh = hk * S.group + jrow - ji * S.group;
    // a NaN sum is kept; only an empty row is 0
    const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
    T* orow = (T*)A.out + b * A.os[0] + ji * A.os[1] + jh * A.os[2];
    float* prow = part ? A.opart + (part0 + jrow) * A.dvp : nullptr;
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
        A.mlpart[part0 + jrow] = f32x2{mm, ll};
      else
        A.lse[((int64_t)b * S.hq + jh) * S.lq + ji] = log_sum(mm, ll);
    }
  } else {
    const int row = row0 + 32 * wq + r32;
    if (row >= G.rows) return;
    const int qi = (int)G.by_group((uint32_t)row), qh = hk * S.group + row - qi * S.group;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    T* orow = (T*)A.out + b * A.os[0] + qi * A.os[1] + qh * A.os[2];
    const int64_t prow_i = part0 + row;
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

// Is any value of BYTES bytes no number? By NT threads, a share each; the answer of
// this one's.
template <class T, int BYTES, int NT>
__device__ __forceinline__ bool no_numbers(const char* tv, int thread) {
  const char* p = tv + 16 * thread;
  constexpr int N = BYTES / 16 / NT;
  static_assert(N * NT * 16 == BYTES, "whole shares");
  if constexpr (sizeof(T) == 4) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const u32x4 x = *(const u32x4*)(p + 16 * NT * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, x[e] & 0x7fffffffu);
    }
    return top >= 0x7f800000u;
  } else {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    constexpr unsigned short inf = std::is_same<T, __bf16>::value ? 0x7f80 : 0x7c00;
    u16x2 top = {0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const u32x4 x = *(const u32x4*)(p + 16 * NT * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, x[e] & 0x7fff7fffu));
    }
    return (top[0] >= inf) | (top[1] >= inf);
  }
}
// Puts 0 in their places.
template <class T, int BYTES, int NT>
__device__ __forceinline__ void clear_no_numbers(char* tv, int thread) {
  typedef typename Vec<T>::V4 V4;
#pragma unroll 1
  for (int i = thread; i < BYTES / (int)sizeof(V4); i += NT) {
    V4 x = ((V4*)tv)[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = fabsf((float)x[e]) < kInf ? x[e] : (T)0.0f;
    ((V4*)tv)[i] = x;
  }
}

// Adds the values of keys kb0 .. that are no numbers to the rows that see them; seen(i)
// tells whether the lane's row sees key kb0 + i + 4 h (h: the lane's half).
template <class T, int DP, int KEYS, int NDB, class F>
__device__ __forceinline__ void add_no_numbers(const char* tv, int kb0, int lane, f32x16 (&o)[NDB], F&& seen) {
  using TL = Tile<T, DP>;
  typedef typename Vec<T>::V4 V4;
  const int h = lane >> 5;
#pragma unroll 1
  for (int i = 0; i < KEYS; ++i) {
    if (!seen(i - 4 * h)) continue;
#pragma unroll
    for (int x = 0; x < NDB; ++x)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = 32 * x + 8 * g + 4 * h;
        const V4 y = *(const V4*)(tv + TL::at(kb0 + i, c / TL::EPC) + c % TL::EPC * (int)sizeof(T));
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[x][4 * g + e] += fabsf((float)y[e]) < kInf ? 0.0f : (float)y[e];
        __builtin_amdgcn_sched_barrier(0);  // one at a time: few registers
      }
  }
}

template <class T, int W, int WQ, int WK, int NB, int OCC>
__global__ __launch_bounds__(64 * WQ * WK, OCC) void k_attend_paged(PagedArgs G) {
  constexpr int DP = row_width(W);
  constexpr bool MANY = WQ > 1;
  using TL = Tile<T, DP>;
  using V8 = typename Vec<T>::V8;
  constexpr int NT = 64 * WQ * WK;
  constexpr int KT = 32 * NB * WK;  // keys per tile
  constexpr int KW = 32 * NB;       // of them a wave's own
  constexpr int NS = W / 16, NDB = W / 32;
  constexpr bool kExact = sizeof(T) == 4;  // scores in natural units, as in k_attend
  constexpr bool AHEAD = MANY && TL::RB == 128;
  static_assert(WQ > 1 || (WQ == 1 && NB == 1), "few rows: one tile of 32, a wave's own 32 keys");
  constexpr int kPlaces = MANY ? 0 : paged_places(TL::RB);
  using KeyT = PageTiles<T, DP, KT, NT, kPlaces>;
  constexpr int kJoinBytes = !MANY ? WK * 32 * W * 4 : 0;
  union Memory {
    typename KeyT::Shared keys;
    float join[kJoinBytes / 4 + 1];
  };
  __shared__ Memory sm;
  __shared__ f32x2 sml[MANY ? 1 : WK * 32];

  const AttendArgs& A = G.A;
  const Shape& S = A.S;
  // workgroup -> (pair, row tile, split), as xcd_item deals them
  const int pairs = S.batch * S.hkv;
  int place, rest;
  {
    const int x = blockIdx.x & 7, i = blockIdx.x >> 3;
    if (xcd_by_pair(pairs)) {
      const int p = (int)G.by_per((uint32_t)i);
      place = 8 * p + x;
      rest = i - p * G.per;
    } else {
      const int run = (pairs * G.per + 7) >> 3, item = x * run + i;
      if (i >= run) return;
      place = (int)G.by_per((uint32_t)item);
      rest = item - place * G.per;
    }
    if (place >= pairs) return;
  }
  int tile = (int)G.by_split((uint32_t)rest);
  const int split = rest - tile * A.nsplit;
  // the last rows see the most keys: they come first; where all workgroups run at a
  // time, the second half of a pair's comes in the other order, so that a compute unit
  // gets a long one and a short one (prompts of 2048 x 32 heads 68.6 -> 63.8 us, of 4096 x 16
  // 114.6 -> 106; the chunk of 2048 over 16384 keys 542 -> 537)
  if (G.pair_up && tile >= (G.tiles + 1) / 2) tile = G.tiles - 1 - (tile - (G.tiles + 1) / 2);
  tile = G.tiles - 1 - tile;
  const int pos = (int)G.by_heads((uint32_t)place), hk = place - pos * S.hkv;
  const int b = batch_entry(S, pos);

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r32 = lane & 31;
  const int wq = wave % WQ, wk = wave / WQ;

  const int nkeys = __builtin_amdgcn_readfirstlane(paged_keys(G.P, b));
  int nq = (int)S.lq;  // live queries
  if (S.qlen) {
    const int n = __builtin_amdgcn_readfirstlane(S.qlen[b]);
    nq = n < 0 ? 0 : (n < nq ? n : nq);
  }
  const int nrows = nq * S.group;
  const int row0 = tile * (32 * WQ), row = row0 + 32 * wq + r32;
  const bool live_row = row < nrows;
  const int qi = (int)G.by_group((uint32_t)row), qh = hk * S.group + row - qi * S.group;

  // keys that row r (a live one) may see end at end_of(r), and its window starts at
  // from_of(that)
  const int base = nkeys - nq;  // place of the entry's first row
  auto end_of = [&](int r) {
    const int x = base + (int)G.by_group((uint32_t)r) + 1;
    return x < 0 ? 0 : x;
  };
  auto from_of = [&](int end) {
    const int x = end - G.recent;
    return G.recent == 0 || x < 0 ? 0 : x;
  };
  // (a tile's end may pass 2^31: bounds are compared with its first key)
  int ns = 0, t_lo = 0, total = 0;
  const int last = row0 + 32 * WQ < nrows ? row0 + 32 * WQ - 1 : nrows - 1;
  if (row0 < nrows) {
    const int end = end_of(last), t_end = end / KT + (end % KT != 0);
    t_lo = from_of(end_of(row0)) / KT;
    const int f = G.first < end ? G.first : end, n = f > 0 ? (f - 1) / KT + 1 : 0;
    ns = n < t_lo ? n : t_lo;
    total = ns + t_end - t_lo;
  }
  const int per = (int)G.by_split((uint32_t)(total + A.nsplit - 1));
  const int n0 = split * per, count = total - n0 < per ? total - n0 : per;

  KeyT keys(sm.keys, G, b, hk, nkeys, ns, t_lo, n0, count > 0 ? count : 0, wave, lane);
  keys.begin();

  V8 qf[NS];
  {
    const T* qrow = (const T*)S.q + b * S.qs[0] + qi * S.qs[1] + qh * S.qs[2];
    const bool need = live_row && keys.count > 0;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if (G.qvec) {
        qf[s] = global_frag<T>(qrow, need, s, h, S.d);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) qf[s][e] = need && 16 * s + 8 * h + e < S.d ? qrow[16 * s + 8 * h + e] : (T)0.0f;
      }
    }
  }
  loads_done();
  f32x16 o[NDB];
#pragma unroll
  for (int n = 0; n < NDB; ++n) o[n] = zero16();
  float m = -kInf, l = 0.0f;

  // this lane's row sees keys below `end`, and of these from `from` on or below G.first;
  // over the wave's live rows these bounds run from e_lo to e_hi and f_lo to f_hi
  // (over the workgroup's: b_lo and b_hi)
  const int end = end_of(row), from = from_of(end);
  const int w0 = row0 + 32 * wq, w1 = w0 + 31 < nrows ? w0 + 31 : nrows - 1;
  const int e_lo = end_of(w0), e_hi = w0 < nrows ? end_of(w1) : 0, f_lo = from_of(e_lo), f_hi = from_of(e_hi);

  const int b_lo = end_of(row0), b_hi = from_of(end_of(last));

  uint64_t fine = 0;  // keys.fine of the batch that is computed on
  bool bad = false;   // the batch has pages outside the cache
  for (int it = 0; it < keys.count; ++it) {
    const int kb0 = KW * wk;  // this wave's keys of the tile
    const int j0 = __builtin_amdgcn_readfirstlane(keys.key(it) + kb0);
    if constexpr (MANY) {
      bad = keys.next(it, bad);
    } else {
      if (it % KeyT::BATCH == 0) {
        fine = keys.fine;
        bad = fine != ~uint64_t(0);
      }
      keys.wait(2 * it);
    }
    const char* const tk = keys.ktile(it);
    char* const tv = keys.vtile(it);
    // does every row that computes on these values see every key? If not, are there any
    // that are no numbers? With many rows the workgroup looks together.
    bool odd = false;
    if constexpr (MANY) {
      if (j0 > b_lo - KT || (j0 < b_hi && j0 > G.first - KT)) {
        if (no_numbers<T, KeyT::kTileBytes, NT>(tv, tid)) sm.keys.odd = it + 1;
        __syncthreads();
        odd = __builtin_amdgcn_readfirstlane(sm.keys.odd) == it + 1;
      }
    }
    auto clear = [&] {
      if constexpr (MANY) {
        __syncthreads();
        clear_no_numbers<T, KeyT::kTileBytes, NT>(tv, tid);
        __syncthreads();
      } else {
        clear_no_numbers<T, KeyT::kOwnBytes, 64>(tv, lane);
      }
    };
    if (j0 >= e_hi || (j0 <= f_lo - KW && j0 >= G.first)) {  // no row of this wave sees any
      if constexpr (MANY) {
        if (odd) clear();
      } else {
        keys.start(2 * it + kPlaces);
        keys.wait(2 * it + 1);
        keys.start(2 * it + 1 + kPlaces);
      }
      continue;
    }
    f32x16 sc[NB];
    score_tile<T, DP, AHEAD, NB, NS>(tk, 0, lane, qf, S.d, sc);
    // the products of a tile stay together, and so do its vector instructions: two
    // waves of a SIMD then take turns of themselves (without, and with one of two
    // workgroups ahead by priority as k_attend has it: 2048 rows over 16384 keys of 128
    // 526 us for 509, 4 x 512 over 4096 129 for 115, 2048 x 4096 fp32 of 64 143 for 138;
    // 4096 of 96 under a window 53 for 54.6). With three waves it costs 1%.
    if constexpr (MANY && OCC < 3) __builtin_amdgcn_sched_barrier(0);
    if constexpr (!MANY) {
      keys.reads_done();
      keys.start(2 * it + kPlaces);
    }
    const float f = kExact ? (float)kLog2e : S.c;  // to log2 units
    if constexpr (kExact) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) sc[n][e] = fmaf(sc[n][e], S.scale, sc[n][e] * S.scale_lo);
    }
    const bool all = j0 <= e_lo - KW && (j0 >= f_hi || j0 <= G.first - KW);  // every row sees every key
    // does the row see key i + 4 h of this wave's own? Without branches: a select each.
    const int f0 = from - j0 - 4 * h, g0 = (G.first < end ? G.first : end) - j0 - 4 * h;
    const uint32_t span = (uint32_t)(end - from);
    auto seen = [&](int i) { return ((uint32_t)i - (uint32_t)f0 < span) | (i < g0); };
    if (__builtin_expect(!all, 0)) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) sc[n][e] = seen(32 * n + 8 * (e >> 2) + (e & 3)) ? sc[n][e] : -kInf;
    }
    if (__builtin_expect(bad, 0)) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const bool in = keys.in_cache(it, kb0 + 32 * n + 8 * g, fine);
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][4 * g + e] = in ? sc[n][4 * g + e] : -kInf;
        }
    }
    soften<T, NB, NDB>(sc, f, m, l, o);
    if constexpr (!MANY) {
      keys.wait(2 * it + 1);
      if (__builtin_expect(!all, 0)) odd = __any(no_numbers<T, KeyT::kOwnBytes, 64>(tv, lane));
    }
    if (__builtin_expect(odd, 0)) {
      add_no_numbers<T, DP, KW>(tv, 0, lane, o, seen);
      clear();
    }
    add_values<T, DP, MANY, NB, NDB>(tv, 0, lane, sc, o);
    if constexpr (!MANY) {
      keys.reads_done();
      keys.start(2 * it + 1 + kPlaces);
    }
  }
  l = half_sum(l);
  if (!live_row) {
    m = -kInf;
    l = 0.0f;
  }
  finish_rows<T, W, WQ, WK>(G, sm.join, sml, o, m, l, live_row, split, b, hk, row0);
}

template <class T, int W>
void attend_paged_launch(const PagedArgs& G, PagedForm form, hipStream_t st) {
  const int64_t blocks = xcd_blocks((int64_t)G.A.S.batch * G.A.S.hkv, G.A.tiles * G.A.nsplit);
  constexpr int RB = row_width(W) * (int)sizeof(T);
  constexpr int OCC = RB == 128 ? 3 : (RB == 256 ? 2 : 1);
  constexpr int FEW = kPagedWaves, ALONE = alone_waves(RB);
  if (form == PagedForm::kMany) {
    hipLaunchKernelGGL((k_attend_paged<T, W, 4, 1, 2, OCC>), grid1(blocks, 256), dim3(256), 0, st, G);
  } else if (ALONE == FEW || form == PagedForm::kFew) {
    hipLaunchKernelGGL((k_attend_paged<T, W, 1, FEW, 1, (paged_groups(RB) * FEW + 3) / 4>), grid1(blocks, 64 * FEW), dim3(64 * FEW),
                       0, st, G);
  } else {
    hipLaunchKernelGGL((k_attend_paged<T, W, 1, ALONE, 1, ALONE / 4>), grid1(blocks, 64 * ALONE), dim3(64 * ALONE), 0, st, G);
  }
  SK_LAUNCH_CHECK();
}

// Instantiated once per element type (attend_paged_*.hip).
template <class T>
void attend_paged(const PagedArgs& G, PagedForm form, hipStream_t st) {
  const AttendArgs& A = G.A;
  by_width(A.S.d, A.S.dv, [&](auto w) { attend_paged_launch<T, decltype(w)::value>(G, form, st); });
  if (A.opart) join_splits<T>(A, nullptr, st);
}

}  // namespace attn
}  // namespace sk
