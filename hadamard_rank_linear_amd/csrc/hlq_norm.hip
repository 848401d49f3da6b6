// gfx950 (CDNA4) kernels of the layer norm, forward and backward.
//
// With h the (residual-added) row, n = (h - mean) * rstd and u = g_y * weight:
//   y = n * weight + bias
//   g_x = rstd * (u - mean_c(u) - n * mean_c(u n)) + g_h
//   g_weight = sum_t g_y n,  g_bias = sum_t g_y
// Memory-bound: forward reads x and residual once and writes y and h, backward
// reads g_y, h and g_h once and writes g_x; a few operations per element.
// The variance is the mean of (h - mean)^2 with the mean known (not a
// difference of moments, which cancels when |mean| is large), in fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hlq_internal.h"
#include "hlq_rows.h"

namespace hlq {

// ------------------------------------------------------------ any row length
// One 256-thread workgroup per row; the row is read again for each pass (from
// cache: what a thread reads again it read or wrote itself).

template <int DT>
__global__ __launch_bounds__(256) void k_norm_fwd_wide(NormFwd a) {
  constexpr int N = Piece<DT>::N;
  __shared__ float sm[2][4];
  const int64_t C = a.C;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
  const int64_t base = row * C;
  const void* src = a.x;
  float sum = 0.f;
  for (int64_t c = threadIdx.x * N; c < C; c += 256 * N) {
    u32x4 r = load_piece<DT>(a.x, base + c, C - c);
    if (a.residual) {
      const u32x4 q = load_piece<DT>(a.residual, base + c, C - c);
      float v[N];
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = piece_at<DT>(r, k) + piece_at<DT>(q, k);
      r = make_piece<DT>(v);
      store_piece<DT>(a.h, base + c, C - c, r);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) sum += piece_at<DT>(r, k);
  }
  if (a.residual) src = a.h;
  const float mean = group_sum<256>(sum, sm[0]) / (float)C;
  float sq = 0.f;
  for (int64_t c = threadIdx.x * N; c < C; c += 256 * N) {
    const u32x4 r = load_piece<DT>(src, base + c, C - c);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float d = piece_at<DT>(r, k) - mean;
      sq += c + k < C ? d * d : 0.f;
    }
  }
  const float rstd = 1.0f / sqrtf(group_sum<256>(sq, sm[1]) / (float)C + a.eps);
  if (threadIdx.x == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  for (int64_t c = threadIdx.x * N; c < C; c += 256 * N) {
    const u32x4 r = load_piece<DT>(src, base + c, C - c);
    float w[N], b[N] = {}, y[N];
    load_params<N>(a.weight, a.param_dt, c, C, w);
    if (a.bias) load_params<N>(a.bias, a.param_dt, c, C, b);
#pragma unroll
    for (int k = 0; k < N; ++k) y[k] = (piece_at<DT>(r, k) - mean) * rstd * w[k] + b[k];
    store_piece<DT>(a.y, base + c, C - c, make_piece<DT>(y));
  }
  __syncthreads();
  }
}

template <int DT>
__global__ __launch_bounds__(256) void k_norm_gx_wide(NormBwd a) {
  constexpr int N = Piece<DT>::N;
  __shared__ float sm[2][4];
  const int64_t C = a.C;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
  const int64_t base = row * C;
  const float mean = a.mean[row], rstd = a.rstd[row];
  float su = 0.f, sn = 0.f;
  for (int64_t c = threadIdx.x * N; c < C; c += 256 * N) {
    const u32x4 g = load_piece<DT>(a.g_y, base + c, C - c);
    const u32x4 h = load_piece<DT>(a.h, base + c, C - c);
    float w[N];
    load_params<N>(a.weight, a.param_dt, c, C, w);  // zero past the row
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float u = piece_at<DT>(g, k) * w[k];
      su += u;
      sn += u * ((piece_at<DT>(h, k) - mean) * rstd);
    }
  }
  su = group_sum<256>(su, sm[0]) / (float)C;
  sn = group_sum<256>(sn, sm[1]) / (float)C;
  for (int64_t c = threadIdx.x * N; c < C; c += 256 * N) {
    const u32x4 g = load_piece<DT>(a.g_y, base + c, C - c);
    const u32x4 h = load_piece<DT>(a.h, base + c, C - c);
    float w[N], o[N];
    load_params<N>(a.weight, a.param_dt, c, C, w);
#pragma unroll
    for (int k = 0; k < N; ++k)
      o[k] = rstd * (piece_at<DT>(g, k) * w[k] - su - (piece_at<DT>(h, k) - mean) * rstd * sn);
    if (a.g_h) {
      const u32x4 q = load_piece<DT>(a.g_h, base + c, C - c);
#pragma unroll
      for (int k = 0; k < N; ++k) o[k] += piece_at<DT>(q, k);
    }
    store_piece<DT>(a.g_x, base + c, C - c, make_piece<DT>(o));
  }
  __syncthreads();
  }
}

// Column sums of one range of rows: blockIdx.x a tile of 64 pieces of columns,
// blockIdx.y the range; the four waves take every fourth row of it.
template <int DT>
__global__ __launch_bounds__(256) void k_norm_columns(NormBwd a) {
  constexpr int N = Piece<DT>::N;
  __shared__ float sm[4][64][2 * N + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t C = a.C, c = ((int64_t)blockIdx.x * 64 + lane) * N;
  const int64_t r0 = a.T * blockIdx.y / a.parts, r1 = a.T * (blockIdx.y + 1) / a.parts;
  float gw[N] = {}, gb[N] = {};
  if (c < C)
    for (int64_t r = r0 + wave; r < r1; r += 4) {
      const u32x4 g = load_piece<DT>(a.g_y, r * C + c, C - c);
      const u32x4 h = load_piece<DT>(a.h, r * C + c, C - c);
      const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float v = piece_at<DT>(g, k);
        gw[k] += v * ((piece_at<DT>(h, k) - mean) * rstd);
        gb[k] += v;
      }
    }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    sm[wave][lane][2 * k] = gw[k];
    sm[wave][lane][2 * k + 1] = gb[k];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 128 * N; e += 256) {
    const int l = e / (2 * N), k = e % (2 * N);
    const int64_t col = ((int64_t)blockIdx.x * 64 + l) * N + k / 2;
    if (col < C)
      a.part[((int64_t)blockIdx.y * 2 + (k & 1)) * C + col] =
          (sm[0][l][k] + sm[1][l][k]) + (sm[2][l][k] + sm[3][l][k]);
  }
}

// Fold of the partial column sums part [parts][2][C] in a fixed order:
// 64 columns per workgroup, the sixteen waves take every sixteenth part;
// blockIdx.y 0: g_weight, 1: g_bias.
__global__ __launch_bounds__(1024) void k_norm_fold(NormBwd a) {
  __shared__ double sm[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t C = a.C, c = (int64_t)blockIdx.x * 64 + lane;
  double s = 0.0;
  if (c < C) {
#pragma unroll 8
    for (int64_t p = wave; p < a.parts; p += 16) s += (double)a.part[(p * 2 + blockIdx.y) * C + c];
  }
  sm[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < C) {
    for (int w = 1; w < 16; ++w) s += sm[w][lane];
    void* out = blockIdx.y ? a.g_bias : a.g_weight;
    if (a.param_dt == 0) static_cast<float*>(out)[c] = (float)s;
    else static_cast<__bf16*>(out)[c] = (__bf16)(float)s;
  }
}

int64_t norm_parts(int64_t T, int64_t C, int dtype) {
  (void)C; (void)dtype;
  const int64_t p = (T + 31) / 32;
  return p > 256 ? 256 : p;
}

hipError_t launch_norm_forward(const NormFwd& a, int dtype, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  if (dtype == 0)
    hipLaunchKernelGGL(k_norm_fwd_wide<0>, rows_grid(a.T), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(k_norm_fwd_wide<1>, rows_grid(a.T), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormBwd& a, int dtype, hipStream_t s) {
  const int N = dtype == 0 ? 4 : 8;
  if (a.T) {
    const dim3 cols(cdiv(a.C, 64 * N), (unsigned)a.parts);
    if (dtype == 0) {
      hipLaunchKernelGGL(k_norm_gx_wide<0>, rows_grid(a.T), dim3(256), 0, s, a);
      hipLaunchKernelGGL(k_norm_columns<0>, cols, dim3(256), 0, s, a);
    } else {
      hipLaunchKernelGGL(k_norm_gx_wide<1>, rows_grid(a.T), dim3(256), 0, s, a);
      hipLaunchKernelGGL(k_norm_columns<1>, cols, dim3(256), 0, s, a);
    }
  }
  hipLaunchKernelGGL(k_norm_fold, dim3(cdiv(a.C, 64), a.g_bias ? 2 : 1), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace hlq
