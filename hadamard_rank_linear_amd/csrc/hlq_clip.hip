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

constexpr int CLIP_THREADS = 256;

// The tensor that holds chunk `c` of the list.
__device__ __forceinline__ int clip_find(const ClipList& l, uint32_t c) {
  int lo = 0, hi = l.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.first[mid] <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double clip_take(float v, double acc) {
  const double d = (double)v;
  return __builtin_fma(d, d, acc);
}

template <int DT>
__device__ __forceinline__ void clip_norm_chunk(const void* g, int64_t e0, int64_t n, int kind,
                                                double& sq, uint32_t& top) {
  constexpr int N = Piece<DT>::N;
  for (int64_t e = threadIdx.x * N; e < n; e += CLIP_THREADS * N) {
    const u32x4 r = load_piece<DT>(g, e0 + e, n - e);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float v = piece_at<DT>(r, k);
      if (kind == 0) sq = clip_take(v, sq);
      else top = max(top, __float_as_uint(v) & 0x7FFFFFFFu);  // bits order as |v|, NaN on top
    }
  }
}

__device__ __forceinline__ uint32_t group_umax(uint32_t v, uint32_t* sm) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
  __syncthreads();
  return max(max(sm[0], sm[1]), max(sm[2], sm[3]));
}

// Each workgroup takes a contiguous range of the list's chunks.
__global__ __launch_bounds__(CLIP_THREADS) void k_clip_norm(ClipList l, int kind, double* part) {
  __shared__ double sm[4];
  __shared__ uint32_t smu[4];
  const uint32_t c0 = (uint32_t)((uint64_t)l.chunks * blockIdx.x / gridDim.x);
  const uint32_t c1 = (uint32_t)((uint64_t)l.chunks * (blockIdx.x + 1) / gridDim.x);
  double sq = 0.0;
  uint32_t top = 0u;
  int i = clip_find(l, c0);
  for (uint32_t c = c0; c < c1; ++c) {
    while (i + 1 < l.count && l.first[i + 1] <= c) ++i;
    const uint32_t size = l.size[i] & 0x7FFFFFFFu;
    const int64_t e0 = (int64_t)(c - l.first[i]) * CLIP_CHUNK;
    const int64_t n = min((int64_t)CLIP_CHUNK, (int64_t)size - e0);
    if (l.size[i] >> 31) clip_norm_chunk<1>(l.grad[i], e0, n, kind, sq, top);
    else clip_norm_chunk<0>(l.grad[i], e0, n, kind, sq, top);
  }
  double v;
  if (kind == 0) v = group_sum<CLIP_THREADS>(sq, sm);
  else v = (double)__uint_as_float(group_umax(top, smu));
  if (threadIdx.x == 0) part[blockIdx.x] = v;
}

template <int DT>
__device__ __forceinline__ void clip_scale_chunk(const void* g, void* o, int64_t e0, int64_t n,
                                                 float coef) {
  constexpr int N = Piece<DT>::N;
  for (int64_t e = threadIdx.x * N; e < n; e += CLIP_THREADS * N) {
    const u32x4 r = load_piece<DT>(g, e0 + e, n - e);
    float v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = piece_at<DT>(r, k) * coef;
    store_piece<DT>(o, e0 + e, n - e, make_piece<DT>(v));
  }
}

__global__ __launch_bounds__(CLIP_THREADS) void k_clip_scale(ClipList l, int kind,
                                                             const double* part, int64_t parts,
                                                             double max_norm, double* norm) {
  __shared__ double sm[4];
  __shared__ uint32_t smu[4];
  double v;
  if (kind == 0) {
    double s = 0.0;
    for (int64_t p = threadIdx.x; p < parts; p += CLIP_THREADS) s += part[p];
    v = sqrt(group_sum<CLIP_THREADS>(s, sm));
  } else {
    uint32_t top = 0u;
    for (int64_t p = threadIdx.x; p < parts; p += CLIP_THREADS)
      top = max(top, __float_as_uint((float)part[p]));
    v = (double)__uint_as_float(group_umax(top, smu));
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm) *norm = v;
  const double f = max_norm / (v + 1e-6);
  const float coef = (float)(f >= 1.0 ? 1.0 : f);  // a NaN stays
  if (l.in_place && coef == 1.0f) return;
  const uint32_t c0 = (uint32_t)((uint64_t)l.chunks * blockIdx.x / gridDim.x);
  const uint32_t c1 = (uint32_t)((uint64_t)l.chunks * (blockIdx.x + 1) / gridDim.x);
  int i = clip_find(l, c0);
  for (uint32_t c = c0; c < c1; ++c) {
    while (i + 1 < l.count && l.first[i + 1] <= c) ++i;
    const uint32_t size = l.size[i] & 0x7FFFFFFFu;
    const int64_t e0 = (int64_t)(c - l.first[i]) * CLIP_CHUNK;
    const int64_t n = min((int64_t)CLIP_CHUNK, (int64_t)size - e0);
    if (l.size[i] >> 31) clip_scale_chunk<1>(l.grad[i], l.out[i], e0, n, coef);
    else clip_scale_chunk<0>(l.grad[i], l.out[i], e0, n, coef);
  }
}

hipError_t launch_clip_norm(const ClipList& l, int kind, double* part, unsigned groups,
                            hipStream_t s) {
  hipLaunchKernelGGL(k_clip_norm, dim3(groups), dim3(CLIP_THREADS), 0, s, l, kind, part);
  return hipGetLastError();
}

hipError_t launch_clip_scale(const ClipList& l, int kind, const double* part, int64_t parts,
                             double max_norm, double* norm, unsigned groups, hipStream_t s) {
  hipLaunchKernelGGL(k_clip_scale, dim3(groups), dim3(CLIP_THREADS), 0, s, l, kind, part, parts,
                     max_norm, norm);
  return hipGetLastError();
}

}  // namespace hlq
