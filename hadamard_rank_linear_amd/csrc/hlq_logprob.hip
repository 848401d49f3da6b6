// gfx950 (CDNA4) kernels over rows of logits: log probability of a target,
// the gradient it sends back, the policy loss fused with both, and the policy
// and preference losses on log probabilities.
//
// Per row, with m = max x, e_v = exp(scale (x_v - m)) and s = sum e_v:
//   logprob = scale (x_t - m) - log s,   g_x = g scale ([v = t] - e_v / s)
// m and s come from one pass: a thread keeps the maximum of what it has seen
// and the sum relative to it, rescaling the sum when the maximum grows.  The
// difference x - m is formed before it is scaled, so logits of the type's
// lowest value (masks) neither overflow nor meet inf - inf.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hlq_internal.h"
#include "hlq_rows.h"

namespace hlq {

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// What the exponentials are taken relative to: the maximum, or 0 while only
// -inf has been seen (their exponentials are then 0, not exp(-inf + inf)).
__device__ __forceinline__ float ref_of(float m) { return m == -__builtin_huge_valf() ? 0.f : m; }

// The running maximum m and sum s of a thread over P pieces.
template <int DT, int P>
__device__ __forceinline__ void accumulate(const u32x4 (&r)[P], float c, float& m, float& s) {
  constexpr int N = Piece<DT>::N;
  float top = m;
#pragma unroll
  for (int j = 0; j < P; ++j)
#pragma unroll
    for (int k = 0; k < N; ++k) top = fmaxf(top, piece_at<DT>(r[j], k));
  const float ref = ref_of(top);
  float t = s * exp2_hw((m - ref) * c);
#pragma unroll
  for (int j = 0; j < P; ++j)
#pragma unroll
    for (int k = 0; k < N; ++k) t += exp2_hw((piece_at<DT>(r[j], k) - ref) * c);
  m = top;
  s = t;
}

// A piece whose elements past the row are -inf.
template <int DT>
__device__ __forceinline__ u32x4 load_logits(const void* base, int64_t e, int64_t n) {
  constexpr int N = Piece<DT>::N;
  u32x4 r = load_piece<DT>(base, e, n);
  if (n < N) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k >= n) {
        if constexpr (DT == 0) r[k] = 0xFF800000u;
        else r[k / 2] = (k & 1) ? (r[k / 2] & 0xFFFFu) | 0xFF800000u : 0xFF80u;
      }
  }
  return r;
}

// Maximum and sum of a row over a workgroup of W threads (every thread gets
// both).  sm: 2 * W / 64 values.
template <int DT, int W>
__device__ __forceinline__ void row_stats(const void* x, int64_t base, int64_t V, float c, float* sm,
                                          float& m, float& s) {
  constexpr int N = Piece<DT>::N, P = 4;
  m = -__builtin_huge_valf();
  s = 0.f;
  int64_t v = threadIdx.x * N;
  for (; v + (P - 1) * W * N + N <= V; v += P * W * N) {
    u32x4 r[P];
#pragma unroll
    for (int j = 0; j < P; ++j) r[j] = load_piece<DT>(x, base + v + j * W * N, N);
    accumulate<DT, P>(r, c, m, s);
  }
  for (; v < V; v += W * N) {
    u32x4 r[1] = {load_logits<DT>(x, base + v, V - v)};
    accumulate<DT, 1>(r, c, m, s);
  }
  const float top = group_max<W>(m, sm);
  s = group_sum<W>(s * exp2_hw((m - ref_of(top)) * c), sm + W / 64);
  m = top;
}

__device__ __forceinline__ double logprob_of(float xt, float m, float s, double scale) {
  if (s == 0.f) return -__builtin_huge_val();  // nothing but -inf
  return ((double)xt - (double)m) * scale - log((double)s);
}

// Gradient of a row: f ([v = t] - e_v / s) with f = g * scale; f / s is
// rounded once, then each product once, then the output.
template <int DT, int W>
__device__ __forceinline__ void row_gradient(const void* x, int64_t base, void* g_x, int64_t g_base,
                                             int64_t V, int64_t t, float c, float f, float m,
                                             float s) {
  constexpr int N = Piece<DT>::N;
  if (f == 0.f || s == 0.f) {
    const u32x4 z = {0u, 0u, 0u, 0u};
    for (int64_t v = threadIdx.x * N; v < V; v += W * N) store_piece<DT>(g_x, g_base + v, V - v, z);
    return;
  }
  const float k_s = -f / s;
  for (int64_t v = threadIdx.x * N; v < V; v += W * N) {
    const u32x4 r = load_piece<DT>(x, base + v, V - v);
    float o[N];
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] = k_s * exp2_hw((piece_at<DT>(r, k) - m) * c);
    if (t >= v && t < v + N) {
#pragma unroll
      for (int k = 0; k < N; ++k) o[k] += t - v == k ? f : 0.f;
    }
    store_piece<DT>(g_x, g_base + v, V - v, make_piece<DT>(o));
  }
}

template <int DT, int W>
__global__ __launch_bounds__(W) void k_logprob(LogitArgs a) {
  __shared__ float sm[2 * W / 64];
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const int64_t t = a.targets[row];
    float m = 0.f, s = 1.f, lp = 0.f;
    if (t >= 0 && t < a.V) {
      row_stats<DT, W>(a.logits, row * a.ld, a.V, a.c, sm, m, s);
      if (threadIdx.x == 0)
        lp = (float)logprob_of(load1<DT>(a.logits, row * a.ld + t), m, s, a.scale);
    }
    if (threadIdx.x == 0) {
      a.logprob[row] = lp;
      a.stats[2 * row] = m;
      a.stats[2 * row + 1] = s;
    }
    __syncthreads();  // sm is used again
  }
}

template <int DT, int W>
__global__ __launch_bounds__(W) void k_logprob_grad(LogitArgs a) {
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const int64_t t = a.targets[row];
    const bool live = t >= 0 && t < a.V;
    const float f = live ? a.g_logprob[row] * (float)a.scale : 0.f;
    row_gradient<DT, W>(a.logits, row * a.ld, a.g_x, row * a.g_ld, a.V, t, a.c, f,
                        a.stats[2 * row], a.stats[2 * row + 1]);
  }
}

// ------------------------------------------------------------ policy loss
// The terms of one token, in fp64 from the log probability: w times the loss,
// the KL estimate and whether the clamped ratio counted; returns the gradient.
__device__ __forceinline__ double policy_token(const PolicyArgs& p, int64_t i, double lp,
                                               double (&term)[3]) {
  const double w = p.weight ? (double)p.weight[i] : 1.0, A = (double)p.advantage[i];
  const double r = exp(lp - (double)p.old_logprob[i]);
  const double lo = 1.0 - p.clip_low, hi = 1.0 + p.clip_high;
  const double bounded = r < lo ? lo : (r > hi ? hi : r);
  const double free_ = r * A, clipped = bounded * A;
  const bool cut = clipped < free_;
  double kl = 0.0, g = cut ? 0.0 : -free_;
  if (p.ref_logprob) {
    const double d = (double)p.ref_logprob[i] - lp;
    kl = expm1(d) - d;
    g -= p.kl_coef * expm1(d);
  }
  term[0] = w * (p.kl_coef * kl - (cut ? clipped : free_));
  term[1] = w * kl;
  term[2] = cut ? w : 0.0;
  return w * g;
}

__device__ __forceinline__ bool policy_counts(const PolicyArgs& p, int64_t i) {
  return !p.weight || p.weight[i] != 0.f;
}

template <int DT, int W>
__global__ __launch_bounds__(W) void k_policy_logits(LogitArgs a, PolicyArgs p) {
  __shared__ float sm[2 * W / 64], sg;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const int64_t t = a.targets[row];
    const bool live = t >= 0 && t < a.V && policy_counts(p, row);
    float m = 0.f, s = 1.f;
    if (live) row_stats<DT, W>(a.logits, row * a.ld, a.V, a.c, sm, m, s);
    if (threadIdx.x == 0) {
      double term[3] = {0.0, 0.0, 0.0}, lp = 0.0, g = 0.0;
      if (live) {
        lp = logprob_of(load1<DT>(a.logits, row * a.ld + t), m, s, a.scale);
        g = policy_token(p, row, lp, term);
      }
      a.logprob[row] = (float)lp;
#pragma unroll
      for (int k = 0; k < 3; ++k) p.terms[3 * row + k] = term[k];
      sg = (float)g * (float)a.scale;
    }
    __syncthreads();
    row_gradient<DT, W>(a.logits, row * a.ld, a.g_x, row * a.g_ld, a.V, t, a.c, sg, m, s);
    __syncthreads();  // sm and sg are used again
  }
}

__global__ __launch_bounds__(256) void k_policy(PolicyArgs p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.T) return;
  double term[3] = {0.0, 0.0, 0.0}, g = 0.0;
  if (policy_counts(p, i)) g = policy_token(p, i, (double)p.logprob[i], term);
  p.g_logprob[i] = (float)g;
#pragma unroll
  for (int k = 0; k < 3; ++k) p.terms[3 * i + k] = term[k];
}

// sums[k] = scale * sum_i terms[i][k], K terms per item, one workgroup.
template <int K>
__global__ __launch_bounds__(1024) void k_terms(const double* terms, int64_t n, double scale,
                                                float* sums) {
  __shared__ double sm[K][16];
  double acc[K] = {};
  for (int64_t i = threadIdx.x; i < n; i += 1024)
#pragma unroll
    for (int k = 0; k < K; ++k) acc[k] += terms[K * i + k];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const double v = group_sum<1024>(acc[k], sm[k]);
    if (threadIdx.x == 0) sums[k] = (float)(v * scale);
  }
}

// ------------------------------------------------------------ preference loss
__device__ __forceinline__ int64_t bound(int64_t v, int64_t lo, int64_t hi) {
  return v < lo ? lo : (v > hi ? hi : v);
}

// One workgroup per pair: both sequences' sums in fp64, the loss, the margin
// and the gradient of their tokens.
__global__ __launch_bounds__(256) void k_preference(PrefArgs p) {
  __shared__ double sm[4][4];
  const int64_t pair = blockIdx.x;
  int64_t lo[2], hi[2];
  double sum[2] = {0.0, 0.0}, len[2] = {0.0, 0.0};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int64_t i = pair + q * p.P;
    lo[q] = bound(p.start[i], 0, p.T);
    hi[q] = bound(p.start[i + 1], lo[q], p.T);
    for (int64_t t = lo[q] + threadIdx.x; t < hi[q]; t += 256) {
      const double w = p.weight ? (double)p.weight[t] : 1.0;
      if (w != 0.0) {
        sum[q] += w * ((double)p.logprob[t] - (p.ref_logprob ? (double)p.ref_logprob[t] : 0.0));
        len[q] += w;
      }
    }
    sum[q] = group_sum<256>(sum[q], sm[2 * q]);
    len[q] = group_sum<256>(len[q], sm[2 * q + 1]);
  }
  double part[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) part[q] = !p.mean ? 1.0 : (len[q] > 0.0 ? 1.0 / len[q] : 0.0);
  const double z = p.beta * (sum[0] * part[0] - sum[1] * part[1]), e = p.smoothing;
  const double tail = log1p(exp(-fabs(z)));  // -log sigmoid(z) = tail + max(-z, 0)
  const double g = p.beta / (double)p.P * (1.0 / (1.0 + exp(-z)) - 1.0 + e);
  if (threadIdx.x == 0) {
    p.margin[pair] = (float)z;
    p.terms[pair] = tail + (z < 0.0 ? -(1.0 - e) * z : e * z);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const double gq = (q ? -g : g) * part[q];
    for (int64_t t = lo[q] + threadIdx.x; t < hi[q]; t += 256) {
      const double w = p.weight ? (double)p.weight[t] : 1.0;
      p.g_logprob[t] = w != 0.0 ? (float)(w * gq) : 0.f;
    }
  }
}

#define HLQ_ROWS(K, ...)                                                                      \
  if (dtype == 0)                                                                             \
    hipLaunchKernelGGL((K<0, 1024>), rows_grid(a.T), dim3(1024), 0, s, __VA_ARGS__);     \
  else                                                                                        \
    hipLaunchKernelGGL((K<1, 1024>), rows_grid(a.T), dim3(1024), 0, s, __VA_ARGS__)

hipError_t launch_logprob(const LogitArgs& a, int dtype, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  HLQ_ROWS(k_logprob, a);
  return hipGetLastError();
}

hipError_t launch_logprob_grad(const LogitArgs& a, int dtype, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  HLQ_ROWS(k_logprob_grad, a);
  return hipGetLastError();
}

hipError_t launch_policy_logits(const LogitArgs& a, const PolicyArgs& p, int dtype,
                                hipStream_t s) {
  if (a.T) { HLQ_ROWS(k_policy_logits, a, p); }
  hipLaunchKernelGGL(k_terms<3>, dim3(1), dim3(1024), 0, s, p.terms, p.T, 1.0, p.sums);
  return hipGetLastError();
}
#undef HLQ_ROWS

hipError_t launch_policy(const PolicyArgs& p, hipStream_t s) {
  if (p.T) hipLaunchKernelGGL(k_policy, dim3(cdiv(p.T, 256)), dim3(256), 0, s, p);
  hipLaunchKernelGGL(k_terms<3>, dim3(1), dim3(1024), 0, s, p.terms, p.T, 1.0, p.sums);
  return hipGetLastError();
}

hipError_t launch_preference(const PrefArgs& p, hipStream_t s) {
  hipLaunchKernelGGL(k_preference, dim3((unsigned)p.P), dim3(256), 0, s, p);
  hipLaunchKernelGGL(k_terms<1>, dim3(1), dim3(1024), 0, s, p.terms, p.P, 1.0 / (double)p.P,
                     p.loss);
  return hipGetLastError();
}

}  // namespace hlq
