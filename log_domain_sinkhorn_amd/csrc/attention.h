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

// Chunk c of a row of d elements in memory, zero behind d. AL: rows and the
// base are 16-byte aligned and d is a multiple of the chunk.
template <class T, bool AL>
__device__ __forceinline__ u32x4 load_chunk(const T* row, int c, int d) {
  constexpr int EPC = 16 / (int)sizeof(T);
  if constexpr (AL) {
    if (c * EPC >= d) return u32x4{0, 0, 0, 0};
    return *(const u32x4*)(row + c * EPC);
  } else {
    union {
      T e[EPC];
      u32x4 u;
    } x;
    x.u = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < EPC; ++e)
      if (c * EPC + e < d) x.e[e] = row[c * EPC + e];
    return x.u;
  }
}

// Operand fragment straight from memory: k = 16 s + 8 h + e of the row, zero
// behind d or when the row is not live.
template <class T, bool AL>
__device__ __forceinline__ typename Vec<T>::V8 global_frag(const T* row, bool live, int s, int h, int d) {
  constexpr int N = sizeof(T) / 2;  // chunks per fragment
  union {
    u32x4 u[N];
    typename Vec<T>::V8 v;
  } x;
#pragma unroll
  for (int n = 0; n < N; ++n)
    x.u[n] = live ? load_chunk<T, AL>(row, (2 * s + h) * N + n, d) : u32x4{0, 0, 0, 0};
  return x.v;
}

// Rows [j0, j0 + ROWS) of a matrix, staged by the workgroup's NT threads
// through registers into a Tile: issue the loads of the next tile, compute,
// then put them down. Rows at or behind `count` become zero.
template <class T, int DP, int ROWS, int NT, bool AL>
struct Stage {
  using TL = Tile<T, DP>;
  static constexpr int N = ROWS * TL::CPR / NT;  // chunks per thread
  static constexpr int STEP = NT / TL::CPR;      // rows between a thread's chunks
  static_assert(N * NT == ROWS * TL::CPR && N >= 1, "tile and workgroup sizes");
  u32x4 x[N];

  __device__ __forceinline__ void load(const T* base, int64_t stride, int64_t j0, int64_t count, int d, int tid) {
    const int c = tid % TL::CPR, r0 = tid / TL::CPR;
    const T* p = base + (j0 + r0) * stride;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      x[n] = j0 + r0 + n * STEP < count ? load_chunk<T, AL>(p, c, d) : u32x4{0, 0, 0, 0};
      p += STEP * stride;
    }
  }
  __device__ __forceinline__ void put(char* t, int tid) const {
    const int c = tid % TL::CPR, r0 = tid / TL::CPR;
#pragma unroll
    for (int n = 0; n < N; ++n) *(u32x4*)(t + TL::at(r0 + n * STEP, c)) = x[n];
  }
  // the same with the rows whose column term in LDS is -inf cleared
  __device__ __forceinline__ void put_masked(char* t, const float* term, int tid) const {
    const int c = tid % TL::CPR, r0 = tid / TL::CPR;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int r = r0 + n * STEP;
      *(u32x4*)(t + TL::at(r, c)) = term[r] == -kInf ? u32x4{0, 0, 0, 0} : x[n];
    }
  }
};

// The same straight from memory to LDS (buffer loads with an LDS destination:
// no registers, no LDS writes by the waves), CH = 16 or 4 bytes a lane: 16 for
// rows that are 16-byte aligned and a whole number of 16-byte chunks long, 4 for
// any multiple of four bytes. A wave's instruction fills 64 CH bytes of LDS in
// lane order, so the swizzle is applied to the address a lane fetches. Rows
// that are not live, and what lies behind a row's width, get an offset behind
// the buffer's end, for which the load puts zero. A tile may span at most
// 2^31 bytes.
constexpr uint32_t kOutside = 0x80000000u;

// Written as assembly because the compiler waits for a load to LDS before any
// LDS read that may alias it, so also before reads of the other buffer;
// dma_wait() comes before the barrier behind which the data is read. The loads
// have no destination register.
template <int CH>
__device__ __forceinline__ void dma_load(__amdgpu_buffer_rsrc_t rsrc, uint32_t lds, uint32_t off) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  if constexpr (CH == 16)
    asm volatile(
        "s_mov_b32 m0, %0\n"
        "s_nop 0\n"
        "buffer_load_dwordx4 %1, %2, 0 offen lds"
        :
        : "s"(lds), "v"(off), "s"(rsrc)
        : "memory");
  else
    asm volatile(
        "s_mov_b32 m0, %0\n"
        "s_nop 0\n"
        "buffer_load_dword %1, %2, 0 offen lds"
        :
        : "s"(lds), "v"(off), "s"(rsrc)
        : "memory");
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

// Loader of the rows of a tile by the workgroup's NT threads: start(t, ...)
// begins, land() finishes (staged loads only), dma_wait() and a barrier make
// the tile readable. `wave` must be uniform.
template <class T, int DP, int ROWS, int NT, int CH>
struct Loader {
  using TL = Tile<T, DP>;
  static constexpr int UPR = TL::RB / CH;              // units per row
  static constexpr int N = ROWS * UPR / NT;            // units per thread
  static constexpr int RPI = UPR > 64 ? 1 : 64 / UPR;  // rows per instruction of a wave
  static constexpr int IPR = UPR > 64 ? UPR / 64 : 1;  // instructions per row
  static constexpr int NR = N / IPR;                   // different rows of a lane
  static_assert(N * NT == ROWS * UPR && N >= IPR && N % IPR == 0, "tile and workgroup sizes");

  uint32_t off[CH == 16 ? N : 1];  // byte offset of this lane's unit from the tile's start
  uint32_t pitch;                  // bytes between rows

  // tile row of this lane's units n * IPR ...
  __device__ __forceinline__ static int row(int n, int wave, int lane) {
    return (wave * NR + n) * RPI + (UPR >= 64 ? 0 : lane / UPR);
  }
  __device__ __forceinline__ void init(int64_t stride, int d, int wave, int lane) {
    pitch = (uint32_t)(stride * (int64_t)sizeof(T));
    if constexpr (CH == 16) {
      static_assert(IPR == 1, "16-byte units: at most 64 a row");
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int r = row(n, wave, lane);
        const int c = (lane % UPR) ^ TL::swz(r);
        off[n] = c * TL::EPC < d ? r * pitch + 16 * c : kOutside;
      }
    }
  }
  // live(r): row r of the tile takes part
  template <class F>
  __device__ __forceinline__ void start(const T* base, char* t, F&& live, int d, int wave, int lane) {
    const __amdgpu_buffer_rsrc_t rsrc = dma_rsrc(base);
    const uint32_t lds = lds_offset(t) + wave * (N * 64 * CH);
    // keeps the many offsets and masks of 4-byte units from being computed
    // ahead of the loop over tiles and held in registers
    uint32_t step = pitch;
    if constexpr (CH == 4) asm volatile("" : "+s"(step), "+s"(d));
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      if constexpr (CH == 16) {
        dma_load<16>(rsrc, lds + n * 1024, live(row(n, wave, lane)) ? off[n] : kOutside);
      } else {
        const int r = row(n, wave, lane);
        const bool on = live(r);
#pragma unroll
        for (int i = 0; i < IPR; ++i) {
          const int u = UPR > 64 ? lane + 64 * i : lane % UPR;     // 4-byte unit of the LDS row
          const int w = (((u >> 2) ^ TL::swz(r)) << 2) + (u & 3);  // and of the row in memory
          const bool in = on && w * 4 < d * (int)sizeof(T);
          dma_load<4>(rsrc, lds + (n * IPR + i) * 256, in ? r * step + 4 * w : kOutside);
        }
      }
    }
  }
  __device__ __forceinline__ void land(char*, int, int) const {}
};

// Rows at odd addresses (CH = 2): element by element through registers, in
// the same places.
template <class T, int DP, int ROWS, int NT>
struct Loader<T, DP, ROWS, NT, 2> {
  using TL = Tile<T, DP>;
  static constexpr int N = ROWS * TL::CPR / NT, NR = N, RPI = 64 / TL::CPR;
  static_assert(N * NT == ROWS * TL::CPR && N >= 1, "tile and workgroup sizes");
  u32x4 x[N];
  int64_t pitch;

  __device__ __forceinline__ static int row(int n, int wave, int lane) { return (wave * N + n) * RPI + lane / TL::CPR; }
  __device__ __forceinline__ void init(int64_t stride, int, int, int) { pitch = stride; }
  template <class F>
  __device__ __forceinline__ void start(const T* base, char*, F&& live, int d, int wave, int lane) {
#pragma unroll
    for (int n = 0; n < N; ++n)
      x[n] = live(row(n, wave, lane)) ? load_chunk<T, false>(base + row(n, wave, lane) * pitch, lane % TL::CPR, d)
                                      : u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void land(char* t, int wave, int lane) const {
#pragma unroll
    for (int n = 0; n < N; ++n) *(u32x4*)(t + TL::at(row(n, wave, lane), lane % TL::CPR)) = x[n];
  }
};

__device__ __forceinline__ void dma_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// ---------------------------------------------------------------- arguments
// One attention call as the kernels see it (strides in elements: batch, row,
// head; the innermost dimension has stride 1).
struct Shape {
  int32_t batch, hq, hkv, group;
  int32_t d, dv;
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

// Column term of key j in log2 units: -inf for a masked key.
__device__ __forceinline__ float column_term(const float* bias, int64_t j, int64_t count) {
  if (j >= count) return -kInf;
  if (!bias) return 0.0f;
  const float x = bias[j];
  return x <= kMasked ? -kInf : x * (float)kLog2e;
}

// Workgroup index -> work item, such that each XCD (workgroups go to the 8
// XCDs in turn) takes one contiguous run of items and neighbouring items,
// which read the same keys, share its L2. Items at or behind `total`: none.
__device__ __forceinline__ int64_t xcd_item(int64_t total) {
  const int64_t per = (total + 7) >> 3;
  return (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
}
inline int64_t xcd_blocks(int64_t total) { return ((total + 7) >> 3) << 3; }

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



}  // namespace attn
}  // namespace sk
