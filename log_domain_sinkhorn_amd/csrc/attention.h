// Attention between two sets of different length: the tile machinery shared
// by the forward, gradient and gathered-weight kernels.
//
// Rows. The query heads that share a key head are packed: for one (batch
// entry, key head) pair the rows are r = i * G + g (i: query, g: head within
// the group of G), M = Lq * G of them, so every tile of keys serves the whole
// group. Scores are kept in log2 units: t = c q.k + log2e bias, c = scale log2e.
//
// Matrix tiles. All products run on 32 x 32 MFMA tiles with K = 16 steps
// (16-bit types: v_mfma_f32_32x32x16; fp32: eight v_mfma_f32_32x32x2, a lane's
// eight elements taken one per instruction). Lane l = 32 h + r holds
//   A operand: row r,    k = 8 h + e (e < 8)
//   B operand: column r, k = 8 h + e
//   result:    column r, rows 8 (e / 4) + 4 h + e % 4 (e < 16).
// The order of k within a step is free as long as A and B agree. A result
// (say a transposed tile of weights, keys down and queries across) is therefore
// used as the next product's B operand straight from its registers: registers
// 8 s .. 8 s + 7 are step s with k = 16 s + 4 h + {0..3} and 16 s + 8 + 4 h +
// {0..3}; the A operand is read from LDS in that order (col_frag).
#pragma once

#include <type_traits>

#include "internal.h"

namespace sk {
namespace attn {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kMaxD = 128;         // largest head width
// Head widths are computed on in units of 32 (W: 32, 64, 96 or 128 columns) and
// held in LDS in rows of DP = 64 or 128.
constexpr int row_width(int w) { return w <= 64 ? 64 : 128; }
inline int head_width(int32_t d, int32_t dv) { return ((d > dv ? d : dv) + 31) / 32 * 32; }
// f(std::integral_constant<int, W>) for the width of d and dv
template <class F>
void by_width(int32_t d, int32_t dv, F&& f) {
  switch (head_width(d, dv)) {
    case 32: f(std::integral_constant<int, 32>{}); break;
    case 64: f(std::integral_constant<int, 64>{}); break;
    case 96: f(std::integral_constant<int, 96>{}); break;
    default: f(std::integral_constant<int, 128>{}); break;
  }
}
constexpr float kMasked = -1e30f;  // a bias at or below this masks the key
constexpr float kInf = __builtin_inff();

template <class T>
struct Vec;
template <>
struct Vec<__bf16> {
  typedef bf16x4 V4;
  typedef bf16x8 V8;
};
template <>
struct Vec<_Float16> {
  typedef f16x4 V4;
  typedef f16x8 V8;
};
template <>
struct Vec<float> {
  typedef f32x4 V4;
  typedef f32x8 V8;
};

__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(f16x8 a, f16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(f32x8 a, f32x8 b, f32x16 c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
  return c;
}

// The same where only the first `left` of a lane's k matter (the rest is zero): a
// wave of fp32 spends 64 cycles on each k, so the zeros behind a width that is
// no multiple of 16 are left out (50 columns: 26 instructions in place of 32).
template <class V>
__device__ __forceinline__ f32x16 mma_first(V a, V b, f32x16 c, int left) {
  if constexpr (sizeof(a[0]) == 4) {
    if (left >= 8) return mma(a, b, c);
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < left) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
    return c;
  } else {
    return mma(a, b, c);
  }
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int e = 0; e < 16; ++e) z[e] = 0.0f;
  return z;
}

// Maximum / sum of a lane's value and that of the lane 32 away.
__device__ __forceinline__ float half_max(float x) {
  auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float lg2(float x) { return __builtin_amdgcn_logf(x); }

// Natural log-sum-exp from a log2 reference and the sum of 2^(t - reference).
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.0f ? -kInf : fmaf(m, (float)kLn2, lg2(l) * (float)kLn2);
}

// Eight registers of a result as a B operand (rounded to T: the weights are
// rounded once, to nearest, before the product that consumes them).
template <class T>
__device__ __forceinline__ typename Vec<T>::V8 pack(const f32x16& x, int s) {
  typename Vec<T>::V8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (T)x[8 * s + e];
  return v;
}

// What that rounding left of them, rounded in its turn: both parts together
// hold a weight to 2^-16 (bf16) or 2^-22 (fp16) of it.
template <class T>
__device__ __forceinline__ typename Vec<T>::V8 pack_rest(const f32x16& x, int s, typename Vec<T>::V8 first) {
  typename Vec<T>::V8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (T)(x[8 * s + e] - (float)first[e]);
  return v;
}

// ---------------------------------------------------------------- LDS tiles
// A tile of rows of DP elements, row-major in 16-byte chunks; chunk c of row r
// sits at c ^ swz(r). swz takes 16 consecutive rows to 16 different chunks
// (8 for 128-byte rows, where two rows span the 64 banks), so the 16-byte
// reads of row_frag spread over all banks, and rows that differ in their low
// two bits to different groups of four chunks, which does the same for the
// transposed 8-byte reads of col_frag.
template <class T, int DP>
struct Tile {
  static constexpr int RB = DP * (int)sizeof(T);     // bytes per row
  static constexpr int CPR = RB / 16;                // chunks per row
  static constexpr int EPC = 16 / (int)sizeof(T);    // elements per chunk

  __device__ __forceinline__ static int swz(int r) {
    if constexpr (CPR == 4) return (r >> 2) & 3;
    if constexpr (CPR == 8) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    return ((r & 3) << 2) | ((r >> 2) & 3);
  }
  __device__ __forceinline__ static int at(int r, int c) { return r * RB + ((c ^ swz(r)) << 4); }

  // A (or B) operand: row `row` of the tile, k = 16 s + 8 h + e
  __device__ __forceinline__ static typename Vec<T>::V8 row_frag(const char* t, int row, int s, int h) {
    if constexpr (sizeof(T) == 2) {
      return *(const typename Vec<T>::V8*)(t + at(row, 2 * s + h));
    } else {
      const f32x4 a = *(const f32x4*)(t + at(row, 4 * s + 2 * h));
      const f32x4 b = *(const f32x4*)(t + at(row, 4 * s + 2 * h + 1));
      return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
  }

  // A operand of the transposed tile: row m0 + r (an element index), k =
  // rows k0 + 4 h + {0..3} and k0 + 8 + 4 h + {0..3} of the tile
  __device__ __forceinline__ static typename Vec<T>::V8 col_frag(const char* t, int k0, int m0, int lane) {
    if constexpr (sizeof(T) == 2) {
      // ds_read_b64_tr_b16: of every 16 lanes, lane i gives the address of four
      // elements of row i / 4 and receives element i of the four rows
      const int g = lane >> 4, i = lane & 15;
      const int row = k0 + 4 * (g >> 1) + (i >> 2);
      const int c = (m0 >> 3) + 2 * (g & 1) + ((i & 3) >> 1);
      const char* p0 = t + at(row, c) + 8 * (i & 1);
      const char* p1 = t + at(row + 8, c) + 8 * (i & 1);
      typedef __attribute__((address_space(3))) s16x4 lds4;
      union {
        s16x4 s[2];
        typename Vec<T>::V8 v;
      } u;
      u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p0);
      u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p1);
      return u.v;
    } else {
      const int h = lane >> 5, m = m0 + (lane & 31);
      f32x8 v;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int row = k0 + 4 * h + (e & 3) + 8 * (e >> 2);
        v[e] = *(const float*)(t + at(row, m >> 2) + 4 * (m & 3));
      }
      return v;
    }
  }
};

// Chunk c of a row of d elements in memory (16-byte aligned, whole chunks),
// zero behind d.
template <class T>
__device__ __forceinline__ u32x4 load_chunk(const T* row, int c, int d) {
  constexpr int EPC = 16 / (int)sizeof(T);
  if (c * EPC >= d) return u32x4{0, 0, 0, 0};
  return *(const u32x4*)(row + c * EPC);
}

// Operand fragment straight from memory: k = 16 s + 8 h + e of the row, zero
// behind d or when the row is not live.
template <class T>
__device__ __forceinline__ typename Vec<T>::V8 global_frag(const T* row, bool live, int s, int h, int d) {
  constexpr int N = sizeof(T) / 2;  // chunks per fragment
  union {
    u32x4 u[N];
    typename Vec<T>::V8 v;
  } x;
#pragma unroll
  for (int n = 0; n < N; ++n) x.u[n] = live ? load_chunk<T>(row, (2 * s + h) * N + n, d) : u32x4{0, 0, 0, 0};
  return x.v;
}

// Tiles go straight from memory to LDS (buffer loads with an LDS destination:
// no registers, no LDS writes by the waves), 16 bytes a lane. A wave's
// instruction fills 1 KB of LDS in lane order, so the swizzle is applied to
// the chunk a lane fetches. Rows that take no part, and chunks behind a row's
// width, get an offset behind the buffer's end, for which the load puts zero. A
// tile spans less than 2^31 bytes (the host copies operands for which it
// would not).
constexpr uint32_t kOutside = 0x80000000u;

// Written as assembly because the compiler waits for a load to LDS before any
// LDS read that may alias it, so also before reads of the other buffer;
// dma_wait() comes before the barrier behind which the data is read. The loads
// have no destination register. CH: bytes a lane, 16 or 4. ONCE: the data is read
// once (a non-temporal load, which leaves the caches to others).
template <int CH, bool ONCE = false>
__device__ __forceinline__ void dma_load(__amdgpu_buffer_rsrc_t rsrc, uint32_t lds, uint32_t off) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  if constexpr (CH == 16 && ONCE)
    asm volatile(
        "s_mov_b32 m0, %0\n"
        "s_nop 0\n"
        "buffer_load_dwordx4 %1, %2, 0 offen nt lds"
        :
        : "s"(lds), "v"(off), "s"(rsrc)
        : "memory", "m0");
  else if constexpr (CH == 16)
    asm volatile(
        "s_mov_b32 m0, %0\n"
        "s_nop 0\n"
        "buffer_load_dwordx4 %1, %2, 0 offen lds"
        :
        : "s"(lds), "v"(off), "s"(rsrc)
        : "memory", "m0");
  else
    asm volatile(
        "s_mov_b32 m0, %0\n"
        "s_nop 0\n"
        "buffer_load_dword %1, %2, 0 offen lds"
        :
        : "s"(lds), "v"(off), "s"(rsrc)
        : "memory", "m0");
}
// base: the same for all lanes (the reads make that known to the compiler)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t dma_rsrc(const void* base) {
  const uint64_t p = (uint64_t)base;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)p), hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)((uint64_t)hi << 32 | lo), 0, (int)kOutside, 0x00027000);
}
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}
// Waits until at most N of the wave's memory operations are outstanding (they
// complete in order, so all but the last N have).
template <int N>
__device__ __forceinline__ void dma_wait() {
  static_assert(N >= 0 && N < 64, "vmcnt has six bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Waits for all outstanding loads in a way that the compiler knows of. Behind
// the loads of operands that stay in registers and before the first load to LDS:
// the compiler would otherwise put its own wait for them into the loop over
// tiles, and there wait for the tiles being loaded as well.
__device__ __forceinline__ void loads_done() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt 0

// Loader of ROWS rows by the workgroup's NT threads: instructions of 1 KB, the
// waves in turn. `wave` must be uniform.
template <class T, int DP, int ROWS, int NT, bool ONCE = false>
struct Loader {
  using TL = Tile<T, DP>;
  static constexpr int TOTAL = ROWS * TL::CPR / 64;        // instructions
  static constexpr int NW = NT / 64;                       // waves
  static constexpr int N = (TOTAL + NW - 1) / NW;          // instructions of a wave at most
  static constexpr int RPI = 64 / TL::CPR;                 // rows per instruction
  static_assert(TOTAL * 64 == ROWS * TL::CPR && RPI >= 1, "whole instructions");
  uint32_t off[N];  // byte offset of this lane's chunk from the tile's start

  // tile row of this lane's chunk n
  __device__ __forceinline__ static int row(int n, int wave, int lane) { return (n * NW + wave) * RPI + lane / TL::CPR; }
  __device__ __forceinline__ static bool has(int n, int wave) { return TOTAL % NW == 0 || n * NW + wave < TOTAL; }

  // at(r): byte offset of row r of the tile
  template <class F>
  __device__ __forceinline__ void place(F&& at, int d, int wave, int lane) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int r = row(n, wave, lane);
      const int c = (lane % TL::CPR) ^ TL::swz(r);
      off[n] = c * TL::EPC < d ? at(r) + 16 * c : kOutside;
    }
  }
  // live(r): row r takes part
  template <class F>
  __device__ __forceinline__ void start(const T* base, char* t, F&& live, int wave, int lane) const {
    const __amdgpu_buffer_rsrc_t rsrc = dma_rsrc(base);
    const uint32_t lds = lds_offset(t) + wave * 1024;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (has(n, wave)) dma_load<16, ONCE>(rsrc, lds + n * NW * 1024, live(row(n, wave, lane)) ? off[n] : kOutside);
  }
};

// ---------------------------------------------------------------- arguments
// One attention call as the kernels see it (strides in elements: batch, row,
// head; the innermost dimension has stride 1).
struct Shape {
  int32_t batch, hq, hkv, group;
  int32_t d, dv;
  uint32_t group_mul;    // ceil(2^32 / group): x / group = (x group_mul) >> 32 while x group < 2^32; 0 for 1
  int64_t lq, lk, rows;  // rows = lq * group
  int64_t qs[3], ks[3], vs[3];
  const void* q;
  const void* k;
  const void* v;
  const float* bias;  // nullable; bias + b * bs[0] + hkv * bs[1] + j
  int64_t bs[2];
  const int32_t* qlen;  // nullable
  const int32_t* klen;  // nullable
  float scale, scale_lo;  // of the scores: the fp32 value and what it misses
  float c;                // scale * log2(e)
};

__device__ __forceinline__ int64_t live_keys(const Shape& S, int b) {
  if (!S.klen) return S.lk;
  const int64_t n = S.klen[b];
  return n < 0 ? 0 : (n > S.lk ? S.lk : n);
}
__device__ __forceinline__ int64_t live_rows(const Shape& S, int b) {
  if (!S.qlen) return S.rows;
  const int64_t n = S.qlen[b];
  return (n < 0 ? 0 : (n > S.lq ? S.lq : n)) * S.group;
}

// The batch entry that the workgroups at place `pos` of the batch work on. With
// lengths of its own for each entry: the longer half first, longest at the front,
// then the shorter half from its shortest up, so that of two workgroups that share
// a compute unit one is short where the other is long (512 x 2000 x 16 heads x 8,
// lengths from 1125 to 2000 in random order: 44.7 -> 40.9 us; from longest to
// shortest 42.2, long and short in turn 44.6).
__device__ __forceinline__ int batch_entry(const Shape& S, int pos) {
  if (!S.klen || S.batch < 2 || S.batch > 64) return pos;
  const int lane = threadIdx.x & 63;
  const int mine = lane < S.batch ? S.klen[lane] : -1;
  int rank = 0;
  for (int b = 0; b < S.batch; ++b) {
    const int other = __builtin_amdgcn_readlane(mine, b);
    rank += other > mine || (other == mine && b < lane);
  }
  const int half = (S.batch + 1) / 2;
  const int want = pos < half ? pos : S.batch - 1 - (pos - half);
  return (int)__builtin_ctzll(__ballot(lane < S.batch && rank == want));
}

// With two waves a SIMD, of two workgroups: one of them issues ahead of the
// other, so that the matrix work of one meets the vector work of the other (8192 x
// 16384 x 32 heads of 128, bf16: 2075 -> 2055 us; with three waves, at 64 columns,
// it costs 5%).
__device__ __forceinline__ void one_ahead() {
  if ((blockIdx.x >> 8) & 1) __builtin_amdgcn_s_setprio(1);
}

// Rows of the packed (query, head) side: byte offset of row r of a tile that
// starts at head `rem` of its first query.
__device__ __forceinline__ uint32_t packed_row(const Shape& S, int r, int rem, uint32_t row_bytes, uint32_t head_bytes) {
  const uint32_t x = (uint32_t)(r + rem);
  if (S.group == 1) return x * row_bytes;
  const uint32_t i = __umulhi(x, S.group_mul);
  return i * row_bytes + (x - i * (uint32_t)S.group) * head_bytes;
}

// Column term of key j: its bias times `unit`, -inf for a masked key.
__device__ __forceinline__ float column_term(const float* bias, int64_t j, int64_t count, float unit) {
  if (j >= count) return -kInf;
  if (!bias) return 0.0f;
  const float x = bias[j];
  return x <= kMasked ? -kInf : x * unit;
}

// Tiles of RT packed rows of q (or dout), by loads to LDS, one after the other
// from tile t0 on. Where the group divides RT a lane's offsets are the same in
// every tile.
template <class T, int DP, int RT, int NT>
struct RowTiles {
  Loader<T, DP, RT, NT> ld;
  const T* base;
  int64_t row_stride, left;  // left: live rows from the next tile's first on
  uint32_t row_bytes, head_bytes;
  int d, rem, step, step_rem;  // rem: the next tile's first head; a tile is `step` queries and `step_rem` heads long

  __device__ __forceinline__ RowTiles(const Shape& S, const void* p, const int64_t* s, int b, int hk, int d_, int64_t t0,
                                      int64_t nrows, int wave, int lane)
      : row_stride(s[1]), left(nrows - t0 * RT), row_bytes((uint32_t)(s[1] * sizeof(T))),
        head_bytes((uint32_t)(s[2] * sizeof(T))), d(d_), step(RT / S.group), step_rem(RT % S.group) {
    const int64_t qi = t0 * RT / S.group;
    rem = (int)(t0 * RT - qi * S.group);
    base = (const T*)p + b * s[0] + (int64_t)hk * S.group * s[2] + qi * row_stride;
    ld.place([&](int r) { return packed_row(S, r, 0, row_bytes, head_bytes); }, d, wave, lane);
  }
  // starts the next tile
  __device__ __forceinline__ void start(const Shape& S, char* tile, int wave, int lane) {
    if (step_rem != 0)
      ld.place([&](int r) { return packed_row(S, r, rem, row_bytes, head_bytes); }, d, wave, lane);
    if (left >= RT)
      ld.start(base, tile, [](int) { return true; }, wave, lane);
    else
      ld.start(base, tile, [&](int r) { return r < left; }, wave, lane);
    left -= RT;
    base += step * row_stride;
    rem += step_rem;
    if (rem >= S.group) {
      rem -= S.group;
      base += row_stride;
    }
  }
};

// The tiles of KT keys that a workgroup runs over, the n-th (n = 0 .. count - 1) from
// tile t0 on, in a ring of D buffers (k, then v, in each): tile n + D - 1 is
// started while tile n is computed on. Biases arrive D - 1 tiles before that,
// in a ring of their own: when a tile is started they decide which of its rows
// are loaded and become its column terms (times `unit`; -inf: masked).
// SOME: live() is asked for behind the last tile.
template <class T, int DP, int KT, int NT, int D, bool ONCE = false, bool SOME = false>
struct KeyTiles {
  using Ld = Loader<T, DP, KT, NT, ONCE>;
  static constexpr int kTileBytes = KT * Tile<T, DP>::RB;
  static constexpr int kOps = 2 * Ld::N;  // loads of a wave per tile
  static_assert(D == 2 || Ld::TOTAL % Ld::NW == 0, "counted loads: the same of every wave");
  struct Shared {
    __attribute__((aligned(16))) char tiles[D][2][kTileBytes];
    __attribute__((aligned(16))) float term[D][KT], raw[D][KT];
    int some;  // with a bias: has a key that takes part been seen? (in LDS: a register for it makes fp32 of 128 columns spill)
  };
  Ld lk, lv;
  Shared& sm;
  const T* k;
  const T* v;
  int64_t ks, vs;
  const float* bias;
  int64_t t0, nkeys;
  int count, wave, lane;
  float unit;

  __device__ __forceinline__ KeyTiles(Shared& sm_, const Shape& S, int b, int hk, int64_t first, int64_t last,
                                      int64_t nkeys_, float unit_, int wave_, int lane_)
      : sm(sm_), k((const T*)S.k + b * S.ks[0] + hk * S.ks[2]), v((const T*)S.v + b * S.vs[0] + hk * S.vs[2]),
        ks(S.ks[1]), vs(S.vs[1]), bias(S.bias ? S.bias + b * S.bs[0] + hk * S.bs[1] : nullptr), t0(first),
        nkeys(nkeys_), count(last > first ? (int)(last - first) : 0), wave(wave_), lane(lane_), unit(unit_) {
    const uint32_t kp = (uint32_t)(ks * sizeof(T)), vp = (uint32_t)(vs * sizeof(T));
    lk.place([&](int r) { return r * kp; }, S.d, wave, lane);
    lv.place([&](int r) { return r * vp; }, S.dv, wave, lane);
  }
  __device__ __forceinline__ void fetch(int n) const {
    const int j = wave * 64 + lane;
    if (!bias || n >= count || j >= KT) return;  // a lane that loads also writes: none behind the tile
    const int64_t first = (t0 + n) * KT;
    dma_load<4>(dma_rsrc(bias + first), lds_offset(sm.raw[n % D]) + wave * 256, first + j < nkeys ? 4 * j : kOutside);
  }
  __device__ __forceinline__ void start(int n) const {
    if (n >= count) return;
    const int buf = n % D, tid = wave * 64 + lane;
    const float* raw = sm.raw[buf];
    const int64_t first = (t0 + n) * KT, left = nkeys - first;  // live keys from the tile's first on
    if (tid < KT) {
      float term = 0.0f;
      if (bias) {
        const float x = raw[tid];
        term = x <= kMasked ? -kInf : x * unit;
      }
      if (tid >= left) term = -kInf;
      sm.term[buf][tid] = term;
      if (SOME && bias && term != -kInf) sm.some = 1;
    }
    auto both = [&](auto&& live) {
      lk.start(k + first * ks, sm.tiles[buf][0], live, wave, lane);
      lv.start(v + first * vs, sm.tiles[buf][1], live, wave, lane);
    };
    if (bias)
      both([&](int r) { return r < left && !(raw[r] <= kMasked); });
    else if (left < KT)
      both([&](int r) { return r < left; });
    else
      both([](int) { return true; });
  }
  // before the first tile
  __device__ __forceinline__ void begin() const {
    if (bias) {
      if (SOME && wave == 0) sm.some = 0;
#pragma unroll
      for (int n = 0; n < 2 * (D - 1) && n < D; ++n) fetch(n);
      dma_wait<0>();
      __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < D - 1; ++n) {
      start(n);
    }
    if (bias && D > 2) {
      // the rest of the biases that the first tiles' starts will want
      __syncthreads();
#pragma unroll
      for (int n = D; n < 2 * (D - 1); ++n) fetch(n);
      dma_wait<0>();
    }
  }
  // Makes tile n readable and starts the one D - 1 further on. The loads of the
  // tiles after n stay in flight, and of what else the wave has issued since
  // the loads of tile n at least `stores` operations (0 or STORES), so that
  // waiting for loads does not mean waiting for the caller's stores; any more
  // than that only make the wait longer.
  template <int STORES = 0>
  __device__ __forceinline__ void next(int n, bool stores = false) const {
    const int ahead = count - 1 - n;
    if constexpr (D == 2)
      dma_wait<0>();
    else if (ahead >= D - 2 && stores)
      dma_wait<(D - 2) * kOps + STORES>();
    else if (ahead >= D - 2)
      dma_wait<(D - 2) * kOps>();
    else if (D > 3 && ahead == 1)
      dma_wait<kOps>();
    else
      dma_wait<0>();
    __syncthreads();
    fetch(n + 2 * (D - 1));
    start(n + D - 1);
  }
  __device__ __forceinline__ const char* ktile(int n) const { return sm.tiles[n % D][0]; }
  __device__ __forceinline__ const char* vtile(int n) const { return sm.tiles[n % D][1]; }
  __device__ __forceinline__ const float* term(int n) const { return sm.term[n % D]; }
  // behind the last tile, by all threads of the workgroup: does any of its keys take part?
  __device__ __forceinline__ bool live() const {
    static_assert(SOME, "kept where it is asked for");
    if (!bias) return count > 0;
    __syncthreads();
    return sm.some != 0;
  }
  // does tile n have masked columns? (without a bias only where the live keys end)
  __device__ __forceinline__ bool masked(int n) const { return bias != nullptr || (t0 + n + 1) * KT > nkeys; }
};

// Workgroup index -> work item (pair * per + one of the pair's `per`), or -1.
// Workgroups go to the 8 XCDs in turn, and those that read the same keys should
// share one's L2. With pairs in multiples of 8 (or many) an XCD takes every
// eighth pair, so that the heads of a short sequence do not all fall to one XCD
// (against one contiguous run of the items, sequences of half to whole length: 512
// x 2000 x 16 heads x 8 48 -> 45 us, one token a sequence x 32768 x 8 heads x 16
// 357 -> 332); otherwise it takes such a run, which also deals out fewer pairs.
__host__ __device__ inline bool xcd_by_pair(int64_t pairs) { return pairs % 8 == 0 || pairs >= 64; }
__device__ __forceinline__ int64_t xcd_item(int64_t pairs, int64_t per) {
  const int64_t x = blockIdx.x & 7, i = blockIdx.x >> 3;
  if (xcd_by_pair(pairs)) {
    const int64_t p = i / per, pair = 8 * p + x;
    return pair < pairs ? pair * per + (i - p * per) : -1;
  }
  const int64_t item = x * ((pairs * per + 7) >> 3) + i;
  return i < ((pairs * per + 7) >> 3) && item < pairs * per ? item : -1;
}
inline int64_t xcd_blocks(int64_t pairs, int64_t per) {
  return xcd_by_pair(pairs) ? 8 * ((pairs + 7) / 8) * per : ((pairs * per + 7) >> 3) << 3;
}

// Four consecutive elements of a row in memory from fp32; VEC: aligned and d
// a multiple of four.
template <class T, bool VEC>
__device__ __forceinline__ void store4(T* row, int c, int d, f32x4 x) {
  if constexpr (VEC) {
    if (c < d) {
      typename Vec<T>::V4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = (T)x[e];
      *(typename Vec<T>::V4*)(row + c) = v;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < d) row[c + e] = (T)x[e];
  }
}

// ---------------------------------------------------------------- host side
// May the rows of a matrix be read (or written) in units of `bytes`?
inline bool rows_aligned(const void* p, const int64_t* stride, int64_t width, int64_t size, int64_t bytes) {
  const int64_t q = bytes / size;
  return ((uintptr_t)p % bytes) == 0 && stride[0] % q == 0 && stride[1] % q == 0 && stride[2] % q == 0 &&
         width % q == 0;
}

// Have two arrays of n and m bytes no byte in common? (a null one has none)
inline bool apart(const void* a, int64_t n, const void* b, int64_t m) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x == 0 || y == 0 || x + (uintptr_t)n <= y || y + (uintptr_t)m <= x;
}

}  // namespace attn
}  // namespace sk
