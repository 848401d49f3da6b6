// Device pieces of the attention kernels: fragments of the 32 x 32 matrix
// products, tiles in LDS that are read by rows and by columns, the packed
// sequences' bounds, and the line of relative position biases.  Header-only,
// internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hlq_rows.h"

namespace hlq {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634074f;
constexpr float kLn2 = 0.69314718055994530942f;

// A fragment: 8 values a lane of a 32 x 16 operand of D = A B + C.  Lane l
// holds row (A) or column (B) l & 31 and, of the 16 values along the sum, those
// of its half l >> 5.  Which of them is which element is free as long as A and B
// agree.  The result has column l & 31 and rows acc_row(r, half) in register r.
template <int DT>
struct FragOf {
  typedef f32x8 type;
};
template <>
struct FragOf<1> {
  typedef bf16x8 type;
};
template <int DT>
using Frag = typename FragOf<DT>::type;

__device__ __forceinline__ constexpr int acc_row(int r) { return 8 * (r >> 2) + (r & 3); }

// bf16: one instruction; fp32: eight of two values along the sum each (no
// rounding of the operands).
__device__ __forceinline__ f32x16 mma(const bf16x8& a, const bf16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(const f32x8& a, const f32x8& b, f32x16 c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
  return c;
}

template <int DT>
__device__ __forceinline__ Frag<DT> zero_frag() {
  Frag<DT> f;
  __builtin_memset(&f, 0, sizeof f);
  return f;
}

// Registers 8 c .. 8 c + 7 of a result as the fragment of a following product
// that sums over its rows: rows 16 c + 8 (e >> 2) + 4 half + (e & 3), which is
// the order col_frag reads in.  In bf16 this rounds probabilities and score
// gradients to nearest even (2^-8 of each at most): the matrix instructions take
// bf16 only with bf16.  In o the error averages out (0.0017 of it in all, 0.0016 of
// that o's own rounding), in the gradients of k and v it is as large as their own
// rounding (0.0023 in all); see acc_rest for that of q.
template <int DT>
__device__ __forceinline__ Frag<DT> acc_frag(const f32x16& s, int c) {
  Frag<DT> f;
  if constexpr (DT == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = s[8 * c + e];
  } else {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack_bf16(s[8 * c + 2 * e], s[8 * c + 2 * e + 1]);
    __builtin_memcpy(&f, &w, 16);
  }
  return f;
}

// What acc_frag(s, c) = f has rounded off, as a fragment of its own: the product with
// it makes up for the rounding.  With D_i from the o that is not rounded a row's score
// gradients sum to zero, and what keys have in common cancels in the gradient of q, but not
// in their rounding errors.  For the formula, which takes o as it is stored, this product
// halves the error of g_q (ViT-B 0.0034 in all, with it 0.0017, that of rounding g_q).  For
// the gradient itself it does little in bf16: there the rounding of o moves D_i, the sums
// are not zero, and g_q is 0.0061 off (0.0068 without; keys of 24 in common 0.05).  It costs
// 3 of 48 us there, 58 of 343 on 8192 ragged tokens with heads of 128.
__device__ __forceinline__ bf16x8 acc_rest(const f32x16& s, int c, const bf16x8& f) {
  u32x4 w;
  __builtin_memcpy(&w, &f, 16);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = pack_bf16(s[8 * c + 2 * e] - __uint_as_float(w[e] << 16),
                     s[8 * c + 2 * e + 1] - __uint_as_float(w[e] & 0xFFFF0000u));
  bf16x8 r;
  __builtin_memcpy(&r, &w, 16);
  return r;
}

// Where hidden pairs have probability zero, an infinity or NaN in the other operand
// would reach the columns that do not see it (0 * NaN).  Blocks of which some
// columns see a part are looked through for such values first.  If there are any,
// the product goes without them, and a column that sees one becomes NaN as a whole.

// The high bits of the halves (bf16) or words (fp32) whose value is not finite.
template <int DT>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  if constexpr (DT == 1) return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
  else return ((w & 0x7F800000u) + 0x00800000u) & 0x80000000u;
}
template <int DT>
__device__ __forceinline__ uint32_t not_finite(const Frag<DT>& f) {
  uint32_t w[sizeof f / 4], bad = 0;
  __builtin_memcpy(w, &f, sizeof f);
#pragma unroll
  for (unsigned i = 0; i < sizeof f / 4; ++i) bad |= not_finite<DT>(w[i]);
  return bad;
}
// f with those values set to zero if `clean`, the same in all lanes.
template <int DT>
__device__ __forceinline__ Frag<DT> only_finite(const Frag<DT>& f, bool clean) {
  if (!clean) return f;
  uint32_t w[sizeof f / 4];
  __builtin_memcpy(w, &f, sizeof f);
#pragma unroll
  for (unsigned i = 0; i < sizeof f / 4; ++i) {
    const uint32_t t = not_finite<DT>(w[i]);
    w[i] &= DT == 1 ? ~((t - (t >> 15)) | t) : t ? 0u : ~0u;
  }
  Frag<DT> r;
  __builtin_memcpy(&r, w, sizeof f);
  return r;
}

// ------------------------------------------------------------ tiles in LDS

// Rows of DP elements in 16-byte chunks, chunk c of row r at c ^ mix(r).  The 64
// banks give 256 bytes a cycle: 16 lanes of a read by rows (one chunk of 16
// consecutive rows), 32 of a transposing read (four chunks of four rows), 64 of a
// read of single words (eight chunks of two rows, four apart).  The mix puts each of
// these into banks of its own; it is linear over exclusive or.  (No conflicts are
// counted; with a mix for 32 banks they were as many cycles as the reads.)
template <int DT, int DP>
struct Tile {
  static constexpr int CE = DT == 0 ? 4 : 8;          // elements a chunk
  static constexpr int CHUNKS = DP / CE;              // of a row
  static constexpr int PITCH = CHUNKS <= 8 ? 8 : CHUNKS <= 16 ? 16 : 32;
  static constexpr int ROW_BYTES = PITCH * 16;
  static constexpr int MIXED = PITCH == 8 ? 7 : 15;   // chunk bits that take part
  typedef __attribute__((address_space(3))) const char L;

  __device__ static __forceinline__ constexpr int mix(int r) {
    if (PITCH == 8) return ((r & 2) << 1) | ((r >> 2) & 3);  // two rows fill the banks
    if (DT == 0) return ((r & 4) << 1) | ((r & 3) << 1) | ((r >> 3) & 1);
    return ((r & 3) << 2) | ((r >> 2) & 3);
  }
  __device__ static __forceinline__ int at(int r, int c) { return (r * PITCH + (c ^ mix(r))) * 16; }

  // A lane's place in a tile read by rows (row lane & 31, the first of its half's
  // chunks) and by columns (see col_frag): what at() gives without the constant
  // parts of row and chunk, which are put in by an exclusive or where they meet the
  // mix and by addition above.
  __device__ static __forceinline__ uint32_t row_lane() {
    const int lane = threadIdx.x & 63, half = lane >> 5;
    return at(lane & 31, DT == 1 ? half : 2 * half);
  }
  __device__ static __forceinline__ uint32_t col_lane() {
    const int lane = threadIdx.x & 63, half = lane >> 5;
    if constexpr (DT == 1) {
      const int col = (lane & 16) + 4 * (lane & 3);
      return at(4 * half + ((lane & 15) >> 2), col >> 3) + (col & 4) * 2;
    } else {
      return at(4 * half, (lane & 31) >> 2) + (lane & 3) * 4;
    }
  }
  // row: a multiple of 32, and low rows of the 16 that share no bit with the lane's
  __device__ static __forceinline__ L* place(uint32_t lane, int row, int low, int chunk) {
    return (L*)(uintptr_t)((lane ^ (((chunk & MIXED) ^ mix(low)) * 16)) + (chunk & ~MIXED) * 16 +
                           (row + low) * ROW_BYTES);
  }

  // Rows r .. r + 31 (one a lane), elements 16 c + 8 half .. + 7.  tile: row_lane()
  // plus the tile's place in LDS.
  __device__ static __forceinline__ Frag<DT> row_frag(uint32_t tile, int r, int c) {
    Frag<DT> f;
    if constexpr (DT == 1) {
      f = *(__attribute__((address_space(3))) const bf16x8*)place(tile, r, 0, 2 * c);
    } else {
      typedef __attribute__((address_space(3))) const f32x4 V;
      const f32x4 a = *(V*)place(tile, r, 0, 4 * c), b = *(V*)place(tile, r, 0, 4 * c + 1);
      f = (f32x8){a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
    return f;
  }

  // Columns 32 d .. 32 d + 31 (one a lane), rows r + 8 (e >> 2) + 4 half + (e & 3)
  // (r a multiple of 16): the operand whose sum runs over rows.  bf16: two transposing
  // reads, in which lane j of 16 points at row j / 4, columns 4 (j % 4) of a 4 x 16
  // block and gets column j.  tile: col_lane() plus the tile's place.
  __device__ static __forceinline__ Frag<DT> col_frag(uint32_t tile, int r, int d) {
    Frag<DT> f;
    if constexpr (DT == 1) {
      typedef __attribute__((address_space(3))) s16x4 V;
      s16x4 v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((V*)place(tile, r, 8 * i, 4 * d));
      __builtin_memcpy(&f, v, 16);
    } else {
      typedef __attribute__((address_space(3))) const float V;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f[e] = *(V*)place(tile, r, 8 * (e >> 2) + (e & 3), 8 * d);
    }
    return f;
  }
};

// Elements d .. of a row of n as a chunk of 16 bytes; past the row: zero.
// VEC: rows start at 16-byte boundaries and hold whole chunks.
template <int DT, bool VEC>
__device__ __forceinline__ u32x4 row_chunk(const void* row, int d, int n) {
  typedef typename Piece<DT>::Elem E;
  if constexpr (VEC) {
    if (d < n) return *reinterpret_cast<const u32x4*>(static_cast<const E*>(row) + d);
    return (u32x4){0u, 0u, 0u, 0u};
  }
  return load_piece<DT>(row, d, n - d);
}

template <int DT, bool VEC>
__device__ __forceinline__ Frag<DT> global_frag(const void* row, int d, int n) {
  Frag<DT> f;
  u32x4 w[DT == 0 ? 2 : 1];
  w[0] = row_chunk<DT, VEC>(row, d, n);
  if constexpr (DT == 0) w[1] = row_chunk<DT, VEC>(row, d + 4, n);
  __builtin_memcpy(&f, w, sizeof f);
  return f;
}

// Four values of elements d .. d + 3 of an output row of n.
template <int DT>
__device__ __forceinline__ void store4(void* row, int d, int n, bool vec, float a, float b, float c,
                                       float e) {
  typedef typename Piece<DT>::Elem E;
  E* p = static_cast<E*>(row) + d;
  if (d >= n) return;
  if constexpr (DT == 0) {
    if (vec) {
      *reinterpret_cast<float4*>(p) = make_float4(a, b, c, e);
      return;
    }
    const float v[4] = {a, b, c, e};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (d + i < n) p[i] = v[i];
  } else {
    const uint32_t lo = pack_bf16(a, b), hi = pack_bf16(c, e);
    if (vec) {
      *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
      return;
    }
    const uint32_t w[2] = {lo, hi};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (d + i < n) p[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
  }
}

// Bit i: row r + i of a tile holds a value that is not finite.  The same in every lane.
template <int DT, int DP>
__device__ __forceinline__ uint32_t rows_not_finite(uint32_t tile, int r) {
  uint32_t bad = 0;
#pragma unroll
  for (int c = 0; c < DP / 16; ++c) bad |= not_finite<DT>(Tile<DT, DP>::row_frag(tile, r, c));
  const uint64_t lanes = __ballot(bad != 0);
  return (uint32_t)lanes | (uint32_t)(lanes >> 32);
}
// Bits low .. high - 1 of 32.
__device__ __forceinline__ uint32_t bit_range(int low, int high) {
  const uint32_t below = high >= 32 ? ~0u : high <= 0 ? 0u : (1u << high) - 1u;
  return low >= 32 ? 0u : low <= 0 ? below : below & ~((1u << low) - 1u);
}

// A tile's way from global memory into LDS, by 256 threads: straight, without
// registers, where rows are whole 16-byte chunks (VEC; 8192 ragged tokens' backward 2853
// us through registers, 1203 so).  A load writes 16 bytes of
// each lane of a wave behind one another, so the mix of a row's chunks is made by the
// lanes' addresses; chunks that do not exist come from a page of zeros.  A thread has
// the same chunk of every RS-th row; its bytes from the tile's first row on are
// 32-bit offsets (token strides are limited for that).
__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0, 0, 0, 0};

// v, which the compiler takes for unknown: what is made of it is not kept in
// registers from before the loop.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The loads are written out: the compiler would wait for all of them before the
// first transposing read of any tile, also of those that are there.  All of a tile at
// once: spread over the products before they were as slow (8192 tokens 586 and 584 us,
// the backward pass 800 and 827).  They have no
// result in a register; feed_wait() is what waits for them.
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(lds), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds(const char* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :: "s"(lds), "v"(p) : "memory", "m0");
}
// Every load into LDS of this thread has arrived, and, after the barrier, the group's.
__device__ __forceinline__ void feed_wait() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

template <int DT, int DP, int ROWS, bool VEC>
struct Feed {
  typedef Tile<DT, DP> T;
  static constexpr int RS = 256 / T::PITCH, N = ROWS / RS;
  static_assert(RS % 8 == 0 && ROWS % RS == 0, "whole turns of a thread");
  uint32_t off, step;

  __device__ static __forceinline__ int row() { return threadIdx.x / T::PITCH; }
  // The thread's chunk at turn i: where rows step by 8 every other one has another mix.
  __device__ static __forceinline__ int chunk(int i) {
    return (int)(threadIdx.x % T::PITCH) ^ T::mix(row()) ^ (RS == 8 && (i & 1) ? T::mix(8) : 0);
  }
  // Strides in bytes; pack heads of a token make neighbouring rows (pack divides RS).
  __device__ __forceinline__ void init(uint32_t token, uint32_t head, int pack) {
    step = RS / pack * token;
    off = (uint32_t)(row() / pack) * token + (uint32_t)(row() % pack) * head + chunk(0) * 16;
  }
  // base: the tile's first row; n: how many rows there are from it on; lds: the tile's
  // place.  For the others of the group the tile is there after feed_wait().
  __device__ __forceinline__ void issue(const char* base, int n, int D, uint32_t lds) const {
    const int flip = RS == 8 ? (chunk(1) - chunk(0)) * 16 : 0;
    if constexpr (VEC) {
      const uint32_t mine = lds + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
      if (n >= ROWS && D == DP && T::PITCH == T::CHUNKS) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          load_to_lds(base + (size_t)(i * step), off + (i & 1 ? flip : 0), mine + i * 4096);
        return;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int r = opaque(row()) + i * RS;
        const char* p = base + (size_t)(off + (i & 1 ? flip : 0) + i * step);
        load_to_lds(r < n && chunk(i) * T::CE < D ? p : (const char*)kZeros, mine + i * 4096);
      }
      return;
    }
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
      const int c = chunk(i);
      u32x4 v = {0u, 0u, 0u, 0u};
      if (row() + i * RS < n && c * T::CE < D)
        v = load_piece<DT>(base + (size_t)(off + (i & 1 ? flip : 0) + i * step), 0, D - c * T::CE);
      *(__attribute__((address_space(3))) u32x4*)(uintptr_t)(lds + (i * 256 + threadIdx.x) * 16) = v;
    }
  }
};

// The kernel's argument (its only one) to be read where it is needed: the compiler
// loads what it knows to be constant at the start, and has no registers to keep it
// in until the end.
template <typename A>
__device__ __forceinline__ const __attribute__((address_space(4))) A* again() {
  typedef const __attribute__((address_space(4))) A C;
  uint64_t p = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return (C*)p;
}

// ------------------------------------------------------------ sequences

// First token and length of sequence s, within [0, T].
__device__ __forceinline__ void sequence(const int64_t* start, int64_t s, int64_t T, int& first,
                                         int& n) {
  int64_t a = 0, b = T;
  if (start) {
    a = start[s];
    b = start[s + 1];
    a = a < 0 ? 0 : a > T ? T : a;
    b = b < 0 ? 0 : b > T ? T : b;
  }
  first = (int)a;
  n = b > a ? (int)(b - a) : 0;
}

// Unit and tile of a work item (see AttnShape); false for the items that fill the
// last round of the XCDs.  A workgroup's XCD is its number modulo 8.
__device__ __forceinline__ bool item_of(const AttnShape& g, unsigned item, unsigned& unit,
                                        unsigned& tile) {
  const unsigned n = g.tiles * g.splits;
  unsigned i = item, units = g.units;
  if (g.by_xcd) {
    i = item / 8;
    units = (g.units + 7) / 8;
  }
  if (g.by_tile) {
    tile = i / units;
    unit = i % units;
  } else {
    unit = i / n;
    tile = i % n;
  }
  if (g.by_xcd) unit = unit * 8 + item % 8;
  return unit < g.units;
}

// ------------------------------------------------------------ position bias

// The biases of one head, times log2(e), over the distances -(reach + 64) ..
// reach + 64: a 32 x 32 block of scores that is not beyond reach as a whole
// reads its line without limits.
constexpr int BIAS_MARGIN = 64;
__device__ __forceinline__ int bias_line_size(const AttnBias& b) {
  return 2 * (b.reach + BIAS_MARGIN) + 1;
}

// Bucket of a distance d = key position - query position; first: the first distance
// of each bucket of a side, in LDS.
__device__ __forceinline__ int bias_bucket(const AttnBias& b, const int16_t* first, int d) {
  const int n = b.bidirectional ? (d < 0 ? -d : d) : (d < 0 ? -d : 0);
  int low = 0, high = b.side;  // first[low] <= n < first[high]
  while (high - low > 1) {
    const int mid = (low + high) / 2;
    if (n >= first[mid]) low = mid;
    else high = mid;
  }
  return low + (b.bidirectional && d > 0 ? b.side : 0);
}

// Call by all threads; ends with first in place (BIAS_FIRST entries) but the line
// needing a barrier.
constexpr int BIAS_FIRST = 128;
__device__ __forceinline__ void load_bias_first(const AttnBias& b, int16_t* first) {
  for (int i = threadIdx.x; i < b.side; i += blockDim.x)
    first[i] = (int16_t)(i < b.exact ? i : b.first[i]);
  __syncthreads();
}
__device__ __forceinline__ void load_bias_line(const AttnBias& b, const int16_t* first, int head,
                                               int heads, float* line) {
  const int n = bias_line_size(b);
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int64_t at = (int64_t)bias_bucket(b, first, i - b.reach - BIAS_MARGIN) * heads + head;
    line[i] = kLog2e * (b.dtype == 0 ? static_cast<const float*>(b.table)[at]
                                     : bf16_lo(static_cast<const uint16_t*>(b.table)[at]));
  }
}

// The line's distances of bucket k: from .. to, none if from > to.
__device__ __forceinline__ void bucket_range(const AttnBias& b, const int16_t* first, int k, int& from,
                                             int& to) {
  const int j = k >= b.side ? k - b.side : k, end = b.reach + BIAS_MARGIN;
  const int near = first[j], far = j + 1 < b.side ? first[j + 1] - 1 : end;
  if (k >= b.side) {
    from = near > 1 ? near : 1;
    to = far;
  } else {
    from = -far;
    to = j == 0 && !b.bidirectional ? end : -near;
  }
}

// Sums along the diagonals of a wave's 32 x 32 block (rows of the accumulator at acc_row
// + 4 half, columns lanes): element (i, l) is written to place i of line i - l + 31, so
// that a line's 32 places, of which those without an element stay zero, are one lane's.
// 16 writes and 8 reads; adding to LDS with the unit's own fp32 additions takes 193
// cycles an instruction, 16 times as long, and the order of the additions is not ours.
// A line's pitch, in whole 16-byte pieces; its writes meet four to a bank, 5% of the
// kernel's time at most.
constexpr int SKEW = 36;
constexpr int SKEW_SIZE = 63 * SKEW;
__device__ __forceinline__ float diagonal_sum(float* skew, const f32x16& v) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
  float* const at = skew + (31 - (lane & 31)) * SKEW + 4 * half * (SKEW + 1);
#pragma unroll
  for (int r = 0; r < 16; ++r) at[acc_row(r) * (SKEW + 1)] = v[r];
  __builtin_amdgcn_wave_barrier();
  const f32x4* const mine = reinterpret_cast<const f32x4*>(skew + min(lane, 62) * SKEW);
  f32x4 sum = mine[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) sum += mine[i];
  __builtin_amdgcn_wave_barrier();
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

}  // namespace hlq
