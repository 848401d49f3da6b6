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
// gradients to nearest even (2^-9 of each at most): the matrix instructions take
// no other type, and the sums of a row average it out.
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

// Nonzero if one of the fragment's values is not finite (all exponent bits set).
__device__ __forceinline__ uint32_t not_finite(const bf16x8& f) {
  u32x4 w;
  __builtin_memcpy(&w, &f, 16);
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= ((w[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
  return bad;
}
__device__ __forceinline__ uint32_t not_finite(const f32x8& f) {
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    bad |= ((__float_as_uint(f[i]) & 0x7F800000u) + 0x00800000u) & 0x80000000u;
  return bad;
}

// acc += A B where the probabilities B of hidden pairs are zero but A may hold
// infinities or NaN in rows that some columns do not see (0 * NaN would reach
// them).  sees(i): whether this lane's column sees place i (0 .. 15) of the sum.
// Finite operands, the usual case, cost the test alone; else one product for
// each of the 16 places, kept by the columns that see it.
template <int DT, typename F>
__device__ __forceinline__ f32x16 mma_seen(const Frag<DT>& a, const Frag<DT>& b, f32x16 acc,
                                           F sees) {
  if (__builtin_expect(!__any(not_finite(a) != 0), 1)) return mma(a, b, acc);
  const int half = (threadIdx.x >> 5) & 1;
  for (int i = 0; i < 16; ++i) {
    const int h = (i >> 2) & 1, e = 4 * (i >> 3) + (i & 3);
    Frag<DT> one = zero_frag<DT>();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j == e && half == h) one[j] = a[j];
    const f32x16 next = mma(one, b, acc);
    const bool s = sees(i);
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = s ? next[r] : acc[r];
  }
  return acc;
}

// ------------------------------------------------------------ tiles in LDS

// Rows of DP elements in 16-byte chunks.  Chunk c of row r lies at c ^ mix(r):
// eight consecutive rows put one chunk into eight different bank groups (reads
// by rows), and four consecutive rows two neighbouring chunks (reads by columns).
template <int DT, int DP>
struct Tile {
  static constexpr int CE = DT == 0 ? 4 : 8;          // elements a chunk
  static constexpr int CHUNKS = DP / CE;              // of a row
  static constexpr int PITCH = CHUNKS <= 8 ? 8 : CHUNKS <= 16 ? 16 : 32;
  static constexpr int ROW_BYTES = PITCH * 16;

  __device__ static __forceinline__ int mix(int r) { return ((r & 3) << 1) | ((r >> 2) & 1); }
  __device__ static __forceinline__ int at(int r, int c) { return (r * PITCH + (c ^ mix(r))) * 16; }

  // Row r, elements d .. d + 7 (d a multiple of 8).
  __device__ static __forceinline__ Frag<DT> row_frag(const char* lds, int r, int d) {
    Frag<DT> f;
    if constexpr (DT == 1) {
      f = *reinterpret_cast<const bf16x8*>(lds + at(r, d / 8));
    } else {
      const float4 a = *reinterpret_cast<const float4*>(lds + at(r, d / 4));
      const float4 b = *reinterpret_cast<const float4*>(lds + at(r, d / 4 + 1));
      f = (f32x8){a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    }
    return f;
  }

  // Column d + (lane & 31), rows r + 8 (e >> 2) + 4 half + (e & 3): the operand
  // whose sum runs over rows.  bf16: two transposing reads, in which lane j of 16
  // points at row j / 4, columns 4 (j % 4) of a 4 x 16 block and gets column j.
  __device__ static __forceinline__ Frag<DT> col_frag(const char* lds, int r, int d) {
    const int lane = threadIdx.x & 63, half = lane >> 5;
    Frag<DT> f;
    if constexpr (DT == 1) {
      const int row = r + 4 * half + ((lane & 15) >> 2);
      const int col = d + (lane & 16) + 4 * (lane & 3);
      const int sub = (col & 4) * 2;
      typedef __attribute__((address_space(3))) s16x4 L;
      s16x4 v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (L*)(lds + at(row + 8 * i, col >> 3) + sub));
      __builtin_memcpy(&f, v, 16);
    } else {
      const int col = d + (lane & 31);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int row = r + 8 * (e >> 2) + 4 * half + (e & 3);
        f[e] = *reinterpret_cast<const float*>(lds + at(row, col >> 2) + (col & 3) * 4);
      }
    }
    return f;
  }
};

// Elements d .. of a row of n as a chunk of 16 bytes; past the row: zero.
// vec: rows start at 16-byte boundaries and hold whole chunks.
template <int DT>
__device__ __forceinline__ u32x4 row_chunk(const void* row, int d, int n, bool vec) {
  typedef typename Piece<DT>::Elem E;
  const E* p = static_cast<const E*>(row) + d;
  if (vec) {
    if (d < n) return *reinterpret_cast<const u32x4*>(p);
    return (u32x4){0u, 0u, 0u, 0u};
  }
  return load_piece<DT>(row, d, n - d);
}

template <int DT>
__device__ __forceinline__ Frag<DT> global_frag(const void* row, int d, int n, bool vec) {
  Frag<DT> f;
  u32x4 w[DT == 0 ? 2 : 1];
  w[0] = row_chunk<DT>(row, d, n, vec);
  if constexpr (DT == 0) w[1] = row_chunk<DT>(row, d + 4, n, vec);
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

// A tile's global loads, a chunk a time per thread of 256, held until the LDS
// is free.  row(r) is row r's address, null past the end (read as zeros).
template <int DT, int DP, int ROWS>
struct Stage {
  typedef Tile<DT, DP> T;
  static constexpr int N = (ROWS * T::CHUNKS + 255) / 256;
  u32x4 v[N];

  template <typename F>
  __device__ __forceinline__ void load(F row, int D, bool vec) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * 256 + threadIdx.x, r = at / T::CHUNKS, c = at % T::CHUNKS;
      v[i] = (u32x4){0u, 0u, 0u, 0u};
      if (at < ROWS * T::CHUNKS) {
        const void* p = row(r);
        if (p) v[i] = row_chunk<DT>(p, c * T::CE, D, vec);
      }
    }
  }
  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * 256 + threadIdx.x, r = at / T::CHUNKS, c = at % T::CHUNKS;
      if (at < ROWS * T::CHUNKS) *reinterpret_cast<u32x4*>(lds + T::at(r, c)) = v[i];
    }
  }
};

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

// Work items are numbered so that an XCD (workgroups go to the eight in turn)
// takes neighbouring ones, which share keys and values in its L2.
__device__ __forceinline__ int64_t first_item(unsigned groups) {
  const unsigned b = blockIdx.x, per = groups / 8;
  return groups % 8 ? b : (int64_t)(b % 8) * per + b / 8;
}

// ------------------------------------------------------------ position bias

// Bucket of a distance d = key position - query position.
__device__ __forceinline__ int bias_bucket(const AttnBias& b, int d) {
  int n = b.bidirectional ? (d < 0 ? -d : d) : (d < 0 ? -d : 0);
  if (n >= b.exact) {
    int k = b.exact;
    for (int i = b.exact + 1; i < b.side; ++i) k += n >= b.first[i];
    n = k;
  }
  return n + (b.bidirectional && d > 0 ? b.side : 0);
}

// The biases of one head, times log2(e), over the distances -(reach + 64) ..
// reach + 64: a 32 x 32 block of scores that is not beyond reach as a whole
// reads its line without limits.
constexpr int BIAS_MARGIN = 64;
__device__ __forceinline__ int bias_line_size(const AttnBias& b) {
  return 2 * (b.reach + BIAS_MARGIN) + 1;
}
__device__ __forceinline__ float bias_value(const AttnBias& b, int bucket, int head, int heads) {
  const int64_t at = (int64_t)bucket * heads + head;
  return b.dtype == 0 ? static_cast<const float*>(b.table)[at]
                      : bf16_lo(static_cast<const uint16_t*>(b.table)[at]);
}
__device__ __forceinline__ void load_bias_line(const AttnBias& b, int head, int heads, float* line) {
  const int n = bias_line_size(b);
  for (int i = threadIdx.x; i < n; i += blockDim.x)
    line[i] = bias_value(b, bias_bucket(b, i - b.reach - BIAS_MARGIN), head, heads) * kLog2e;
}

}  // namespace hlq
