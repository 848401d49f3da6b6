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

// ------------------------------------------------------------ rows in registers
// L lanes hold a row, M pieces each (L * M pieces cover it): one read of every
// operand, the statistics and the output from registers.  L up to 64: a
// workgroup of B threads takes B / L rows, sums over lanes alone; above: one
// row per workgroup (B = L).

// Sum over the L lanes of a row (every lane gets it).
template <int L>
__device__ __forceinline__ float row_sum(float v, float* sm) {
  if constexpr (L <= 64) return lanes_sum<L>(v);
  else return group_sum<L>(v, sm);
}

template <int DT, int L, int M, int B>
__global__ __launch_bounds__(B) void k_norm_fwd(NormFwd a) {
  constexpr int N = Piece<DT>::N, R = B / L;
  __shared__ float sm[2][16];
  const int lane = threadIdx.x % L;
  const int64_t C = a.C;
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < a.T; r0 += (int64_t)gridDim.x * R) {
    const int64_t row = r0 + threadIdx.x / L;
    // a group past the last row holds zeros and writes nothing
    const int64_t base = row * C, n = row < a.T ? C : 0;
    u32x4 x[M];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int64_t c = (int64_t)(lane + j * L) * N;
      x[j] = load_piece<DT>(a.x, base + c, n - c);
    }
    if (a.residual) {
      u32x4 q[M];
#pragma unroll
      for (int j = 0; j < M; ++j) {
        const int64_t c = (int64_t)(lane + j * L) * N;
        q[j] = load_piece<DT>(a.residual, base + c, n - c);
      }
#pragma unroll
      for (int j = 0; j < M; ++j) {
        const int64_t c = (int64_t)(lane + j * L) * N;
        float v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = piece_at<DT>(x[j], k) + piece_at<DT>(q[j], k);
        x[j] = make_piece<DT>(v);
        store_piece<DT>(a.h, base + c, n - c, x[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
      for (int k = 0; k < N; ++k) sum += piece_at<DT>(x[j], k);
    const float mean = row_sum<L>(sum, sm[0]) / (float)C;
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int64_t c = (int64_t)(lane + j * L) * N;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float d = piece_at<DT>(x[j], k) - mean;
        sq += c + k < C ? d * d : 0.f;
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<L>(sq, sm[1]) / (float)C + a.eps);
    if (lane == 0 && n) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int64_t c = (int64_t)(lane + j * L) * N;
      if (c < n) {
        float w[N], b[N] = {}, y[N];
        load_params<N>(a.weight, a.param_dt, c, C, w);
        if (a.bias) load_params<N>(a.bias, a.param_dt, c, C, b);
#pragma unroll
        for (int k = 0; k < N; ++k) y[k] = (piece_at<DT>(x[j], k) - mean) * rstd * w[k] + b[k];
        store_piece<DT>(a.y, base + c, n - c, make_piece<DT>(y));
      }
    }
    if constexpr (L > 64) __syncthreads();  // sm is used again
  }
}

// Gradient of the rows and, over the rows a group takes, its column sums in
// registers; at the end the groups of a workgroup join theirs (lanes of a wave
// first, then the waves through LDS) and write one partial.
template <int DT, int L, int M, int B>
__global__ __launch_bounds__(B) void k_norm_bwd(NormBwd a) {
  constexpr int N = Piece<DT>::N, R = B / L, COLS = L * M * N;
  __shared__ float sm[2][16];
  extern __shared__ float cols[];  // L <= 64: [B / 64][COLS]
  const int lane = threadIdx.x % L;
  const int64_t C = a.C;
  float gw[M][N] = {}, gb[M][N] = {};
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < a.T; r0 += (int64_t)gridDim.x * R) {
    const int64_t row = r0 + threadIdx.x / L;
    const int64_t base = row * C, n = row < a.T ? C : 0;
    u32x4 g[M], h[M], q[M];
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int64_t c = (int64_t)(lane + j * L) * N;
      g[j] = load_piece<DT>(a.g_y, base + c, n - c);
      h[j] = load_piece<DT>(a.h, base + c, n - c);
    }
    if (a.g_h) {
#pragma unroll
      for (int j = 0; j < M; ++j) {
        const int64_t c = (int64_t)(lane + j * L) * N;
        q[j] = load_piece<DT>(a.g_h, base + c, n - c);
      }
    }
    const float mean = n ? a.mean[row] : 0.f, rstd = n ? a.rstd[row] : 0.f;
    float su = 0.f, sn = 0.f;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int64_t c = (int64_t)(lane + j * L) * N;
      float w[N];
      load_params<N>(a.weight, a.param_dt, c, C, w);  // zero past the row
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float v = piece_at<DT>(g[j], k), x = (piece_at<DT>(h[j], k) - mean) * rstd;
        const float u = v * w[k];
        su += u;
        sn += u * x;
        gw[j][k] += v * x;
        gb[j][k] += v;
      }
    }
    su = row_sum<L>(su, sm[0]) / (float)C;
    sn = row_sum<L>(sn, sm[1]) / (float)C;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int64_t c = (int64_t)(lane + j * L) * N;
      if (c < n) {
        float w[N], o[N];
        load_params<N>(a.weight, a.param_dt, c, C, w);
#pragma unroll
        for (int k = 0; k < N; ++k)
          o[k] = rstd * (piece_at<DT>(g[j], k) * w[k] - su -
                         (piece_at<DT>(h[j], k) - mean) * rstd * sn);
        if (a.g_h) {
#pragma unroll
          for (int k = 0; k < N; ++k) o[k] += piece_at<DT>(q[j], k);
        }
        store_piece<DT>(a.g_x, base + c, n - c, make_piece<DT>(o));
      }
    }
    if constexpr (L > 64) __syncthreads();  // sm is used again
  }
  float* part = a.part + (int64_t)blockIdx.x * 2 * C;
  if constexpr (L > 64) {
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int64_t c = (int64_t)(lane + j * L) * N + k;
        if (c < C) {
          part[c] = gw[j][k];
          part[C + c] = gb[j][k];
        }
      }
  } else {
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      if (side) __syncthreads();
#pragma unroll
      for (int j = 0; j < M; ++j)
#pragma unroll
        for (int k = 0; k < N; ++k) {
          float v = side ? gb[j][k] : gw[j][k];
#pragma unroll
          for (int m = L; m < 64; m <<= 1) v += __shfl_xor(v, m);
          if ((threadIdx.x & 63) < L) cols[wave * COLS + (lane + j * L) * N + k] = v;
        }
      __syncthreads();
      for (int c = threadIdx.x; c < COLS; c += B)
        if (c < C) {
          float v = cols[c];
#pragma unroll
          for (int w = 1; w < B / 64; ++w) v += cols[w * COLS + c];
          part[side * C + c] = v;
        }
    }
  }
}

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

// Fold of the partial column sums part [parts][2][C] in a fixed order, in
// fp64: 16 columns per workgroup, its 64 groups of 16 lanes take every 64th
// part; blockIdx.y 0: g_weight, 1: g_bias.
__global__ __launch_bounds__(1024) void k_norm_fold(NormBwd a) {
  __shared__ double sm[64][17];
  const int lane = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const int64_t C = a.C, c = (int64_t)blockIdx.x * 16 + lane;
  double s = 0.0;
  if (c < C) {
#pragma unroll 8
    for (int64_t p = slot; p < a.parts; p += 64) s += (double)a.part[(p * 2 + blockIdx.y) * C + c];
  }
  sm[slot][lane] = s;
  __syncthreads();
  if (threadIdx.x < 16 && c < C) {
#pragma unroll 8
    for (int w = 1; w < 64; ++w) s += sm[w][lane];
    void* out = blockIdx.y ? a.g_bias : a.g_weight;
    if (a.param_dt == 0) static_cast<float*>(out)[c] = (float)s;
    else static_cast<__bf16*>(out)[c] = (__bf16)(float)s;
  }
}

// ------------------------------------------------------------ launches
// Lanes and pieces per row for rows of `pieces` 16-byte pieces.
enum NormRow { ROW_8x1, ROW_16x1, ROW_32x1, ROW_32x2, ROW_32x3, ROW_64x2, ROW_64x3, ROW_256x1,
               ROW_256x2, ROW_256x3, ROW_256x4, ROW_1024x2, ROW_1024x4, ROW_WIDE };

static NormRow norm_row(int64_t pieces, bool backward) {
  if (pieces <= 8) return ROW_8x1;
  if (pieces <= 16) return ROW_16x1;
  if (pieces <= 32) return ROW_32x1;
  if (pieces <= 64) return ROW_32x2;
  if (pieces <= 96) return ROW_32x3;
  if (pieces <= 128) return ROW_64x2;
  if (pieces <= 192) return ROW_64x3;
  if (pieces <= 256) return ROW_256x1;
  if (pieces <= 512) return ROW_256x2;
  if (pieces <= 768) return ROW_256x3;
  if (pieces <= 1024) return ROW_256x4;
  if (pieces <= 2048) return ROW_1024x2;
  // (the column sums of 4 pieces do not fit a thread's registers beside them)
  if (pieces <= 4096 && !backward) return ROW_1024x4;
  return ROW_WIDE;
}

#define HLQ_NORM_ROWS(F, BS)                                                                \
  case ROW_8x1: F(8, 1, BS); break;                                                         \
  case ROW_16x1: F(16, 1, BS); break;                                                       \
  case ROW_32x1: F(32, 1, BS); break;                                                       \
  case ROW_32x2: F(32, 2, BS); break;                                                       \
  case ROW_32x3: F(32, 3, BS); break;                                                       \
  case ROW_64x2: F(64, 2, BS); break;                                                       \
  case ROW_64x3: F(64, 3, BS); break;                                                       \
  case ROW_256x1: F(256, 1, 256); break;                                                    \
  case ROW_256x2: F(256, 2, 256); break;                                                    \
  case ROW_256x3: F(256, 3, 256); break;                                                    \
  case ROW_256x4: F(256, 4, 256); break;                                                    \
  case ROW_1024x2: F(1024, 2, 1024); break;

static int norm_lanes(NormRow r) {
  static const int lanes[] = {8, 16, 32, 32, 32, 64, 64, 256, 256, 256, 256, 1024, 1024};
  return lanes[r];
}
constexpr int NORM_BWD_THREADS = 512;  // workgroups of the backward kernel, L <= 64

// Workgroups of the backward kernel, each leaving one partial: up to 1024
// threads per CU.
int64_t norm_parts(int64_t T, int64_t C, int dtype) {
  const NormRow r = norm_row((C + (dtype == 0 ? 3 : 7)) / (dtype == 0 ? 4 : 8), true);
  if (r == ROW_WIDE) return (T + 31) / 32 < 256 ? (T + 31) / 32 : 256;
  const int L = norm_lanes(r), B = L <= 64 ? NORM_BWD_THREADS : L;
  const int64_t need = (T + B / L - 1) / (B / L), most = 256 * 1024 / B;
  return need < most ? need : most;
}

hipError_t launch_norm_forward(const NormFwd& a, int dtype, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  const int N = dtype == 0 ? 4 : 8;
  const NormRow r = norm_row((a.C + N - 1) / N, false);
#define HLQ_F(L, M, B)                                                                      \
  do {                                                                                      \
    const dim3 g = rows_grid((a.T + B / L - 1) / (B / L));                                  \
    if (dtype == 0) hipLaunchKernelGGL((k_norm_fwd<0, L, M, B>), g, dim3(B), 0, s, a);      \
    else hipLaunchKernelGGL((k_norm_fwd<1, L, M, B>), g, dim3(B), 0, s, a);                 \
  } while (0)
  switch (r) {
    HLQ_NORM_ROWS(HLQ_F, 256)
    case ROW_1024x4: HLQ_F(1024, 4, 1024); break;
    case ROW_WIDE:
      if (dtype == 0) hipLaunchKernelGGL(k_norm_fwd_wide<0>, rows_grid(a.T), dim3(256), 0, s, a);
      else hipLaunchKernelGGL(k_norm_fwd_wide<1>, rows_grid(a.T), dim3(256), 0, s, a);
  }
#undef HLQ_F
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormBwd& a, int dtype, hipStream_t s) {
  const int N = dtype == 0 ? 4 : 8;
  const NormRow r = norm_row((a.C + N - 1) / N, true);
  const dim3 g((unsigned)a.parts), wide(cdiv(a.C, 64 * N), (unsigned)a.parts);
#define HLQ_B(L, M, B)                                                                      \
  do {                                                                                      \
    const size_t lds = L <= 64 ? (size_t)B / 64 * L * M * N * 4 : 0;                        \
    if (dtype == 0) hipLaunchKernelGGL((k_norm_bwd<0, L, M, B>), g, dim3(B), lds, s, a);    \
    else hipLaunchKernelGGL((k_norm_bwd<1, L, M, B>), g, dim3(B), lds, s, a);               \
  } while (0)
  if (a.T) switch (r) {
    HLQ_NORM_ROWS(HLQ_B, NORM_BWD_THREADS)
    default:
      if (dtype == 0) {
        hipLaunchKernelGGL(k_norm_gx_wide<0>, rows_grid(a.T), dim3(256), 0, s, a);
        hipLaunchKernelGGL(k_norm_columns<0>, wide, dim3(256), 0, s, a);
      } else {
        hipLaunchKernelGGL(k_norm_gx_wide<1>, rows_grid(a.T), dim3(256), 0, s, a);
        hipLaunchKernelGGL(k_norm_columns<1>, wide, dim3(256), 0, s, a);
      }
  }
#undef HLQ_B
  hipLaunchKernelGGL(k_norm_fold, dim3(cdiv(a.C, 16), a.g_bias ? 2 : 1), dim3(1024), 0, s, a);
  return hipGetLastError();
}
#undef HLQ_NORM_ROWS

}  // namespace hlq
