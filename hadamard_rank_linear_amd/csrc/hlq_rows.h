// Device helpers of the row-wise kernels (layer norm, logits, gradient
// clipping): 16-byte pieces of rows that start at any element, and wave and
// workgroup reductions.  Header-only, internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "hlq_device.h"

namespace hlq {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 Loose __attribute__((aligned(2)));  // 16 bytes at any element

// A piece: 16 bytes of a row, 4 fp32 or 8 bf16 elements (dtype DT: 0 or 1).
template <int DT>
struct Piece {
  static constexpr int N = DT == 0 ? 4 : 8;
  typedef typename std::conditional<DT == 0, float, uint16_t>::type Elem;
};

// Piece at element e, of which the row holds n (n >= N: all of it, one
// 16-byte load; the row may start at any element: gfx950 takes element-aligned
// 16-byte accesses, at one more cache line per wave).  Elements past the row
// read as zero and are not touched.
template <int DT>
__device__ __forceinline__ u32x4 load_piece(const void* base, int64_t e, int64_t n) {
  typedef typename Piece<DT>::Elem E;
  const E* p = static_cast<const E*>(base) + e;
  u32x4 r = {0u, 0u, 0u, 0u};
  if (n >= Piece<DT>::N) {
    __builtin_memcpy(&r, p, 16);
  } else {
#pragma unroll
    for (int k = 0; k < Piece<DT>::N; ++k)
      if (k < n) {
        if constexpr (DT == 0) r[k] = __float_as_uint(p[k]);
        else r[k / 2] |= (uint32_t)p[k] << (16 * (k & 1));
      }
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void store_piece(void* base, int64_t e, int64_t n, u32x4 r) {
  typedef typename Piece<DT>::Elem E;
  E* p = static_cast<E*>(base) + e;
  if (n >= Piece<DT>::N) {
    __builtin_memcpy(p, &r, 16);
  } else {
#pragma unroll
    for (int k = 0; k < Piece<DT>::N; ++k)
      if (k < n) {
        if constexpr (DT == 0) p[k] = __uint_as_float(r[k]);
        else p[k] = (uint16_t)(r[k / 2] >> (16 * (k & 1)));
      }
  }
}

// Element k of a piece in fp32 (exact).
template <int DT>
__device__ __forceinline__ float piece_at(const u32x4& r, int k) {
  if constexpr (DT == 0) return __uint_as_float(r[k]);
  else return (k & 1) ? bf16_hi(r[k / 2]) : bf16_lo(r[k / 2]);
}

// Two fp32 values, each rounded to nearest even, as a pair of bf16.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 p = __builtin_convertvector((f2){lo, hi}, b2);
  uint32_t u;
  __builtin_memcpy(&u, &p, 4);
  return u;
}

// fp32 values to a piece, each rounded to nearest even when DT is bf16 (the
// one rounding of an output; v_cvt_pk_bf16_f32).
template <int DT>
__device__ __forceinline__ u32x4 make_piece(const float (&v)[Piece<DT>::N]) {
  u32x4 r;
  if constexpr (DT == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = __float_as_uint(v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
  }
  return r;
}

// N consecutive parameters (weight or bias) from element c of C in fp32;
// past the end: zero.
template <int N>
__device__ __forceinline__ void load_params(const void* base, int dt, int64_t c, int64_t C,
                                            float (&v)[N]) {
  const int64_t n = C - c;
  if (dt == 0) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const u32x4 r = load_piece<0>(base, c + j, n - j);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[j + k] = __uint_as_float(r[k]);
    }
  } else if constexpr (N == 8) {
    const u32x4 r = load_piece<1>(base, c, n);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = piece_at<1>(r, k);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + c;
    if (n >= 4) {
      uint32_t r[2];
      __builtin_memcpy(r, p, 8);
      v[0] = bf16_lo(r[0]); v[1] = bf16_hi(r[0]);
      v[2] = bf16_lo(r[1]); v[3] = bf16_hi(r[1]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = k < n ? bf16_lo(p[k]) : 0.f;
    }
  }
}

// ------------------------------------------------------------ reductions
// The 32-bit values of a lane and of the lane at distance M (one of them p, the
// other q): DPP for M up to 8, a swap of registers' halves for 16 and 32.
template <int M>
__device__ __forceinline__ void lanes_meet(uint32_t v, uint32_t& p, uint32_t& q) {
  p = v;
  if constexpr (M == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    p = r[0];
    q = r[1];
  } else if constexpr (M == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    p = r[0];
    q = r[1];
  } else if constexpr (M == 8) {  // rotation of 16 by 8
    q = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, true);
  } else if constexpr (M == 4) {  // shift of 16 left by 4 for quads 0 and 2, right for 1 and 3
    const int up = __builtin_amdgcn_update_dpp(0, (int)v, 0x104, 0xF, 0x5, false);
    q = (uint32_t)__builtin_amdgcn_update_dpp(up, (int)v, 0x114, 0xF, 0xA, false);
  } else {
    q = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, M == 2 ? 0x4E : 0xB1, 0xF, 0xF, true);
  }
}

// One stage of a butterfly: f (symmetric) of a lane's value and of the one at
// distance M.
template <int M, typename V, typename F>
__device__ __forceinline__ V lanes_stage(V v, F f) {
  constexpr int WORDS = sizeof(V) / 4;
  uint32_t w[WORDS], p[WORDS], q[WORDS];
  __builtin_memcpy(w, &v, sizeof v);
#pragma unroll
  for (int i = 0; i < WORDS; ++i) lanes_meet<M>(w[i], p[i], q[i]);
  V a, b;
  __builtin_memcpy(&a, p, sizeof v);
  __builtin_memcpy(&b, q, sizeof v);
  return f(a, b);
}

// Butterfly over groups of W neighbouring lanes (W a power of two up to 64);
// every lane gets its group's result, the same bits.  All lanes of a group are
// active.  No LDS instructions: a stage is a few cycles, through ds_bpermute
// about a hundred.
template <int W, typename V, typename F>
__device__ __forceinline__ V lanes_join(V v, F f) {
  if constexpr (W >= 64) v = lanes_stage<32>(v, f);
  if constexpr (W >= 32) v = lanes_stage<16>(v, f);
  if constexpr (W >= 16) v = lanes_stage<8>(v, f);
  if constexpr (W >= 8) v = lanes_stage<4>(v, f);
  if constexpr (W >= 4) v = lanes_stage<2>(v, f);
  if constexpr (W >= 2) v = lanes_stage<1>(v, f);
  return v;
}
template <int W, typename V>
__device__ __forceinline__ V lanes_sum(V v) {
  return lanes_join<W>(v, [](V p, V q) { return p + q; });
}
// Sum over the lanes of a wave that are L apart (8, 16 or 32); every lane gets
// its sum.
template <int L, typename V>
__device__ __forceinline__ V lanes_sum_across(V v) {
  const auto add = [](V p, V q) { return p + q; };
  if constexpr (L <= 8) v = lanes_stage<8>(v, add);
  if constexpr (L <= 16) v = lanes_stage<16>(v, add);
  if constexpr (L <= 32) v = lanes_stage<32>(v, add);
  return v;
}
template <int W = 64>
__device__ __forceinline__ float lanes_max(float v) {
  return lanes_join<W>(v, [](float p, float q) { return fmaxf(p, q); });
}

// Over a workgroup of W threads (a multiple of 64, up to 1024).  sm holds
// W / 64 values and may be used again after the next barrier.
template <int W, typename V>
__device__ __forceinline__ V group_sum(V v, V* sm) {
  v = lanes_sum<64>(v);
  if constexpr (W > 64) {
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
    __syncthreads();
    v = sm[threadIdx.x & (W / 64 - 1)];
    v = lanes_sum<W / 64>(v);
  }
  return v;
}

// One workgroup per row up to 2^20 workgroups (a launch holds fewer than 2^32
// threads); kernels step through the rows by the grid.
static inline dim3 rows_grid(int64_t T) { return dim3((unsigned)(T < (1 << 20) ? T : 1 << 20)); }

// Launches a kernel and returns the launch's own status.  From the array of
// argument addresses it takes the host 2.8 us, the <<<>>> form and
// hipGetLastError 3.3, where the small calls' kernels run for 3 to 6.
template <typename... P>
static inline hipError_t launch(void (*kernel)(P...), dim3 grid, int threads, hipStream_t s,
                                const typename std::decay<P>::type&... args) {
  void* at[] = {const_cast<void*>(static_cast<const void*>(&args))...};
  const hipError_t e =
      hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), at, 0, s);
  if (e != hipSuccess) (void)hipGetLastError();  // reported here, not by the next call
  return e;
}

}  // namespace hlq
