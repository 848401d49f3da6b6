// gfx950 (CDNA4) kernels of gradient clipping by the global norm.
//
//   norm = sqrt(sum v^2) or max |v|,   out = v * min(1, max_norm / (norm + 1e-6))
// Two launches over a list of tensors passed by value in the kernel arguments
// (nothing to copy, and a captured graph keeps the list): every workgroup
// writes one partial of the norm, then every workgroup of the scaling pass
// folds the partials itself, in the same order, and scales its part of the
// list.  Memory-bound: two reads and a write of every element (one read from
// cache for lists that fit it).  Squares are exact and summed in fp64, so
// neither a large nor a small norm overflows or vanishes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hlq_internal.h"
#include "hlq_rows.h"

namespace hlq {

// A chunk is CLIP_BYTES of a tensor, CLIP_PIECES 16-byte pieces per thread, all
// loaded before the first is used.  Workgroup b takes chunks b, b + grid, ...:
// the chip reads one stretch of memory at a time.
constexpr int CLIP_THREADS = CLIP_BYTES / 16 / CLIP_PIECES;

struct ClipChunk {
  const char* grad;
  char* out;
  uint32_t bytes;  // of the tensor from here on, CLIP_BYTES at most
  bool bf16;
};

// The tensors' first chunks, one per lane (every wave holds all of them), so
// that a chunk's tensor is found by comparing once and counting lanes: a search
// through the arguments costs a scalar load's latency per step (13.8 us
// instead of 10.1 for 146 small tensors, stepping from the first).
struct ClipIndex {
  uint32_t first[(CLIP_LIST + 63) / 64];
  __device__ __forceinline__ explicit ClipIndex(const ClipList& l) {
#pragma unroll
    for (int j = 0; j < (CLIP_LIST + 63) / 64; ++j) {
      const int i = (threadIdx.x & 63) + 64 * j;
      first[j] = i < l.count ? l.first[i] : 0xFFFFFFFFu;
    }
  }
  __device__ __forceinline__ ClipChunk chunk(const ClipList& l, uint32_t c) const {
    int i = -1;
#pragma unroll
    for (int j = 0; j < (CLIP_LIST + 63) / 64; ++j) i += __popcll(__ballot(first[j] <= c));
    const uint32_t size = l.size[i] & 0x7FFFFFFFu;
    const bool bf16 = l.size[i] >> 31;
    const uint64_t at = (uint64_t)(c - l.first[i]) * CLIP_BYTES;
    const uint64_t left = (uint64_t)size * (bf16 ? 2 : 4) - at;
    return ClipChunk{static_cast<const char*>(l.grad[i]) + at, static_cast<char*>(l.out[i]) + at,
                     (uint32_t)(left < CLIP_BYTES ? left : CLIP_BYTES), bf16};
  }
};

// What a thread holds of a chunk: piece j at byte (thread + j * threads) * 16.
// A piece past the chunk is zero; one across its end is read ending there and
// shifted into place (a chunk below 16 bytes: by elements).
template <bool ST>
__device__ __forceinline__ void clip_load(const ClipChunk& k, u32x4 (&r)[CLIP_PIECES]) {
#pragma unroll
  for (int j = 0; j < CLIP_PIECES; ++j) {
    const uint32_t at = (threadIdx.x + j * CLIP_THREADS) * 16;
    r[j] = (u32x4){0u, 0u, 0u, 0u};
    if (at >= k.bytes) continue;
    if (k.bytes < 16) {
      r[j] = k.bf16 ? load_piece<1>(k.grad, 0, k.bytes / 2) : load_piece<0>(k.grad, 0, k.bytes / 4);
      continue;
    }
    const uint32_t skip = at + 16 > k.bytes ? at + 16 - k.bytes : 0u;
    const Loose* p = reinterpret_cast<const Loose*>(k.grad + (at - skip));
    u32x4 v;
    if constexpr (ST) v = __builtin_nontemporal_load(p);
    else v = *p;
    if (skip) {
      if (skip & 2)
        v = (u32x4){(v[0] >> 16) | (v[1] << 16), (v[1] >> 16) | (v[2] << 16),
                    (v[2] >> 16) | (v[3] << 16), v[3] >> 16};
      if (skip & 4) v = (u32x4){v[1], v[2], v[3], 0u};
      if (skip & 8) v = (u32x4){v[2], v[3], 0u, 0u};
    }
    r[j] = v;
  }
}

template <int DT>
__device__ __forceinline__ void clip_take(const u32x4& r, int kind, double& sq, uint32_t& top) {
#pragma unroll
  for (int k = 0; k < Piece<DT>::N; ++k) {
    const float v = piece_at<DT>(r, k);
    if (kind == 0) sq = __builtin_fma((double)v, (double)v, sq);
    else top = max(top, __float_as_uint(v) & 0x7FFFFFFFu);  // bits order as |v|, NaN on top
  }
}

__device__ __forceinline__ uint32_t group_umax(uint32_t v, uint32_t* sm) {
  v = lanes_join<64>(v, [](uint32_t p, uint32_t q) { return max(p, q); });
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
  __syncthreads();
  v = sm[0];
#pragma unroll
  for (int w = 1; w < CLIP_THREADS / 64; ++w) v = max(v, sm[w]);
  return v;
}

template <bool ST>
__global__ __launch_bounds__(CLIP_THREADS) void k_clip_norm(ClipList l, int kind, double* part) {
  __shared__ double sm[CLIP_THREADS / 64];
  __shared__ uint32_t smu[CLIP_THREADS / 64];
  double sq = 0.0;
  uint32_t top = 0u;
  const ClipIndex index(l);
  for (uint32_t c = blockIdx.x; c < l.chunks; c += gridDim.x) {
    const ClipChunk k = index.chunk(l, c);
    u32x4 r[CLIP_PIECES];
    clip_load<ST>(k, r);
    if (k.bf16) {
#pragma unroll
      for (int j = 0; j < CLIP_PIECES; ++j) clip_take<1>(r[j], kind, sq, top);
    } else {
#pragma unroll
      for (int j = 0; j < CLIP_PIECES; ++j) clip_take<0>(r[j], kind, sq, top);
    }
  }
  double v;
  if (kind == 0) v = group_sum<CLIP_THREADS>(sq, sm);
  else v = (double)__uint_as_float(group_umax(top, smu));
  if (threadIdx.x == 0) part[blockIdx.x] = v;
}

template <int DT, bool ST>
__device__ __forceinline__ void clip_store(const ClipChunk& k, uint32_t at, const u32x4& r,
                                           float coef, int shift) {
  constexpr int N = Piece<DT>::N;
  if (at >= k.bytes) return;
  float v[N];
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = __builtin_ldexpf(piece_at<DT>(r, e) * coef, shift);
  const u32x4 o = make_piece<DT>(v);
  if (at + 16 <= k.bytes) {
    Loose* p = reinterpret_cast<Loose*>(k.out + at);
    if constexpr (ST) __builtin_nontemporal_store(o, p);
    else *p = o;
  } else {
    store_piece<DT>(k.out + at, 0, ((int)k.bytes - (int)at) / (DT == 0 ? 4 : 2), o);
  }
}

template <bool ST>
__global__ __launch_bounds__(CLIP_THREADS) void k_clip_scale(ClipList l, int kind,
                                                             const double* part, int64_t parts,
                                                             double max_norm, double* norm) {
  __shared__ double sm[CLIP_THREADS / 64];
  __shared__ uint32_t smu[CLIP_THREADS / 64];
  double v;
  if (kind == 0) {
    double s = 0.0;
#pragma unroll 4
    for (int64_t p = threadIdx.x; p < parts; p += CLIP_THREADS) s += part[p];
    v = sqrt(group_sum<CLIP_THREADS>(s, sm));
  } else {
    uint32_t top = 0u;
    for (int64_t p = threadIdx.x; p < parts; p += CLIP_THREADS)
      top = max(top, __float_as_uint((float)part[p]));
    v = (double)__uint_as_float(group_umax(top, smu));
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm) *norm = v;
  // The factor as coef 2^shift: where norms are so far above max_norm that fp32
  // would hold it with few bits or none, though the outputs are ordinary numbers,
  // its exponent is applied to the product (one more operation per element, hidden
  // behind the memory).
  double f = max_norm / (v + 1e-6);
  int shift = 0;
  if (f < 0x1p-100) f = frexp(f, &shift);
  const float coef = (float)(f >= 1.0 ? 1.0 : f);  // a NaN stays
  if (l.in_place && coef == 1.0f && shift == 0) return;
  const ClipIndex index(l);
  for (uint32_t c = blockIdx.x; c < l.chunks; c += gridDim.x) {
    const ClipChunk k = index.chunk(l, c);
    u32x4 r[CLIP_PIECES];
    clip_load<ST>(k, r);
#pragma unroll
    for (int j = 0; j < CLIP_PIECES; ++j) {
      const uint32_t at = (threadIdx.x + j * CLIP_THREADS) * 16;
      if (k.bf16) clip_store<1, ST>(k, at, r[j], coef, shift);
      else clip_store<0, ST>(k, at, r[j], coef, shift);
    }
  }
}

hipError_t launch_clip_norm(const ClipList& l, int kind, double* part, unsigned groups,
                            bool stream, hipStream_t s) {
  return launch(stream ? k_clip_norm<true> : k_clip_norm<false>, dim3(groups), CLIP_THREADS, s, l,
                kind, part);
}

hipError_t launch_clip_scale(const ClipList& l, int kind, const double* part, int64_t parts,
                             double max_norm, double* norm, unsigned groups, bool stream,
                             hipStream_t s) {
  return launch(stream ? k_clip_scale<true> : k_clip_scale<false>, dim3(groups), CLIP_THREADS, s,
                l, kind, part, parts, max_norm, norm);
}

}  // namespace hlq
