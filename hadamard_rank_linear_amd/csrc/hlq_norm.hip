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
// L lanes hold a row, M quads (4 elements) each: one read of every operand,
// the statistics and the output from registers.  L up to 64: a workgroup of B
// threads takes B / L rows and sums over lanes alone; above: one row per
// workgroup (B = L).  Quads rather than 16-byte pieces of bf16: twice the
// lanes per row, so half the registers per thread and twice the waves, which
// is what hides the latency of a row.
//
// Addresses are a scalar base (the wave's first row) and a 32-bit byte offset
// per lane.  Rows are at least 4 long here.  When C is no multiple of 4, the
// last quad of a row is read ending at the row's end and shifted into place,
// so nothing outside the row is read, and it is written by elements.

template <int DT>
struct Quad {
  typedef typename std::conditional<DT == 0, u32x4, u32x2>::type Raw;
  static constexpr int BYTES = DT == 0 ? 16 : 8;
};

// The quad at element c of a row (lane's offset `off` bytes from base); skip =
// the elements by which a row's last quad passes its end; `last`: this is it.
template <int DT>
__device__ __forceinline__ typename Quad<DT>::Raw load_quad(const char* base, uint32_t off,
                                                            bool in_row, bool last, int skip) {
  typename Quad<DT>::Raw r = {};
  if (in_row) {
    const uint32_t back = last ? (uint32_t)skip * (Quad<DT>::BYTES / 4) : 0u;
    __builtin_memcpy(&r, base + (off - back), Quad<DT>::BYTES);
    if (last && skip) {
      if constexpr (DT == 0) {
        if (skip & 1) r = (u32x4){r[1], r[2], r[3], 0u};
        if (skip & 2) r = (u32x4){r[2], r[3], 0u, 0u};
      } else {
        if (skip & 1) r = (u32x2){(r[0] >> 16) | (r[1] << 16), r[1] >> 16};
        if (skip & 2) r = (u32x2){r[1], 0u};
      }
    }
  }
  return r;
}

template <int DT>
__device__ __forceinline__ float quad_at(const typename Quad<DT>::Raw& r, int k) {
  if constexpr (DT == 0) return __uint_as_float(r[k]);
  else return (k & 1) ? bf16_hi(r[k / 2]) : bf16_lo(r[k / 2]);
}

template <int DT>
__device__ __forceinline__ typename Quad<DT>::Raw make_quad(const float (&v)[4]) {
  if constexpr (DT == 0) return make_piece<0>(v);
  else return (u32x2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

template <int DT>
__device__ __forceinline__ void store_quad(char* base, uint32_t off, bool in_row, bool last,
                                           int skip, const typename Quad<DT>::Raw& r) {
  if (!in_row) return;
  if (!(last && skip)) {
    __builtin_memcpy(base + off, &r, Quad<DT>::BYTES);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k + skip < 4) {
        if constexpr (DT == 0) reinterpret_cast<uint32_t*>(base + off)[k] = r[k];
        else reinterpret_cast<uint16_t*>(base + off)[k] = (uint16_t)(r[k / 2] >> (16 * (k & 1)));
      }
  }
}

// Sum over the L lanes of a row (every lane gets it).
template <int L>
__device__ __forceinline__ float row_sum(float v, float* sm) {
  if constexpr (L <= 64) return lanes_sum<L>(v);
  else return group_sum<L>(v, sm);
}

// Two sums at once: one exchange through LDS.
template <int L>
__device__ __forceinline__ void row_sums(float (&v)[2], float (*sm)[16]) {
  if constexpr (L <= 64) {
    v[0] = lanes_sum<L>(v[0]);
    v[1] = lanes_sum<L>(v[1]);
  } else {
    v[0] = lanes_sum<64>(v[0]);
    v[1] = lanes_sum<64>(v[1]);
    if ((threadIdx.x & 63) == 0) {
      sm[0][threadIdx.x >> 6] = v[0];
      sm[1][threadIdx.x >> 6] = v[1];
    }
    __syncthreads();
    v[0] = lanes_sum<L / 64>(sm[0][threadIdx.x & (L / 64 - 1)]);
    v[1] = lanes_sum<L / 64>(sm[1][threadIdx.x & (L / 64 - 1)]);
  }
}

// Where a thread stands: lane of its row, and the wave's first row within a
// workgroup's B / L rows.
template <int L>
struct RowLane {
  int lane, wave_row, sub;  // row = workgroup's first + wave_row (scalar) + sub
  __device__ __forceinline__ RowLane() {
    lane = threadIdx.x % L;
    if constexpr (L <= 64) {
      wave_row = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * (64 / L);
      sub = (threadIdx.x & 63) / L;
    } else {
      wave_row = sub = 0;
    }
  }
};

// Four parameters (weight or bias) at element c, zero past the end.
__device__ __forceinline__ void load_quad_params(const void* base, int dt, uint32_t c, bool in_row,
                                                 bool last, int skip, float (&v)[4]) {
  if (dt == 0) {
    const u32x4 r = load_quad<0>(static_cast<const char*>(base), c * 4, in_row, last, skip);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = quad_at<0>(r, k);
  } else {
    const u32x2 r = load_quad<1>(static_cast<const char*>(base), c * 2, in_row, last, skip);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = quad_at<1>(r, k);
  }
}

// M quads of a row in registers: quad j of a lane is elements (lane + j L) 4
// and on.
template <int DT, int L, int M>
struct RowQuads {
  typename Quad<DT>::Raw v[M];
  __device__ __forceinline__ void load(const void* p, int64_t base, uint32_t off, uint32_t c0,
                                       uint32_t C, int skip, bool live) {
    constexpr int ES = DT == 0 ? 4 : 2;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const uint32_t c = c0 + j * L * 4;
      v[j] = load_quad<DT>(static_cast<const char*>(p) + base, off + c * ES, live && c < C,
                           c + 4 > C, skip);
    }
  }
  __device__ __forceinline__ float at(int j, int k) const { return quad_at<DT>(v[j], k); }
};

// Where a workgroup's group of L lanes reads its row of round r0.
template <int DT, int L>
struct RowAt {
  int64_t row, base;
  uint32_t c0, off;
  bool live;  // a group past the last row reads and writes nothing
  __device__ __forceinline__ RowAt(const RowLane<L>& at, int64_t r0, int64_t T, int64_t C) {
    const int64_t first = r0 + at.wave_row;
    row = first + at.sub;
    base = first * C * (DT == 0 ? 4 : 2);
    live = row < T;
    c0 = (uint32_t)at.lane * 4;
    off = (uint32_t)at.sub * (uint32_t)C * (DT == 0 ? 4 : 2);
    // computed anew for every row: else the compiler keeps a 64-bit pointer
    // per operand and quad across the loop instead of base + offset
    asm volatile("" : "+v"(c0), "+v"(off));
  }
};

// A workgroup takes rounds of B / L rows, the grid's width apart.  Weight and
// bias stay in registers (an fp32 weight is twice the bytes of a bf16 row, and
// reading it again for every row kept the vector L1 busier than the row did),
// and a round's operands are loaded while the one before is worked on.  With 64
// MiB operands, bf16: 45 us at 64 columns (65 with a workgroup per round), 46 at
// 768 (49), 44 at 4096 (50, and 47 without the loads ahead), 53 at 1100 (73);
// fp32 42 to 45 us, 256 MiB at 6 TB/s.
template <int DT, int L, int M, int B>
__global__ __launch_bounds__(B, 4) void k_norm_fwd(NormFwd a) {
  constexpr int R = B / L, ES = DT == 0 ? 4 : 2;
  __shared__ float sm[2][2][16];
  const RowLane<L> at;
  const uint32_t C = (uint32_t)a.C;
  const int skip = (4 - (int)(C & 3)) & 3;
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t r0 = (int64_t)blockIdx.x * R;
  RowQuads<DT, L, M> x, q;
  {
    const RowAt<DT, L> p(at, r0, a.T, a.C);
    x.load(a.x, p.base, p.off, p.c0, C, skip, p.live);
    if (a.residual) q.load(a.residual, p.base, p.off, p.c0, C, skip, p.live);
  }
  float w[M][4], b[M][4] = {};
#pragma unroll
  for (int j = 0; j < M; ++j) {
    const uint32_t c = (uint32_t)(at.lane + j * L) * 4;
    load_quad_params(a.weight, a.param_dt, c, c < C, c + 4 > C, skip, w[j]);
    if (a.bias) load_quad_params(a.bias, a.param_dt, c, c < C, c + 4 > C, skip, b[j]);
  }
  for (int turn = 0; r0 < a.T; r0 += step, turn ^= 1) {
    RowQuads<DT, L, M> nx, nq;
    {
      const RowAt<DT, L> n(at, r0 + step, a.T, a.C);
      nx.load(a.x, n.base, n.off, n.c0, C, skip, n.live);
      if (a.residual) nq.load(a.residual, n.base, n.off, n.c0, C, skip, n.live);
    }
    const RowAt<DT, L> p(at, r0, a.T, a.C);
    float sum = 0.f;
    if (a.residual) {
#pragma unroll
      for (int j = 0; j < M; ++j) {
        const uint32_t c = p.c0 + j * L * 4;
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = x.at(j, k) + q.at(j, k);
        x.v[j] = make_quad<DT>(v);
        store_quad<DT>(static_cast<char*>(a.h) + p.base, p.off + c * ES, p.live && c < C,
                       c + 4 > C, skip, x.v[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) sum += x.at(j, k);
    const float mean = row_sum<L>(sum, sm[turn][0]) / (float)C;
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const uint32_t c = p.c0 + j * L * 4;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float d = x.at(j, k) - mean;
        sq += c + k < C ? d * d : 0.f;
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<L>(sq, sm[turn][1]) / (float)C + a.eps);
    if (at.lane == 0 && p.live) {
      a.mean[p.row] = mean;
      a.rstd[p.row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const uint32_t c = p.c0 + j * L * 4;
      float y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = (x.at(j, k) - mean) * rstd * w[j][k] + b[j][k];
      store_quad<DT>(static_cast<char*>(a.y) + p.base, p.off + c * ES, p.live && c < C, c + 4 > C,
                     skip, make_quad<DT>(y));
    }
    x = nx;
    q = nq;
  }
}

// Column sum c of a workgroup's rows (side 0: of g_y n, 1: of g_y): a partial
// for the fold, or the output itself where there is one workgroup.
__device__ __forceinline__ void put_param(void* out, int dt, int64_t c, float v) {
  if (dt == 0) static_cast<float*>(out)[c] = v;
  else static_cast<__bf16*>(out)[c] = (__bf16)v;
}
__device__ __forceinline__ void put_column(const NormBwd& a, int64_t part, int side, int64_t c,
                                           float v) {
  if (a.parts > 1) a.part[(part * 2 + side) * a.C + c] = v;
  else if (side == 0) put_param(a.g_weight, a.param_dt, c, v);
  else if (a.g_bias) put_param(a.g_bias, a.param_dt, c, v);
}

// Gradient of the rows and, over the rows a group takes, its column sums in
// registers; at the end the groups of a workgroup join theirs (lanes of a wave
// first, then the waves through LDS) and write one partial.  These sums are fp32, as
// 8 M of them a lane in fp64 are more registers than the rows themselves, and
// only the fold is fp64: 32 rows a group at 16383 x 4096 leave an error of 1.2e-7
// (5.8e-8 with every sum in fp64).  The weight stays in
// registers (KEEP), except for four quads a lane in fp32, where there is no room
// and it is read again.  With 64 MiB operands, fold included: bf16 51 us at 64
// columns (70 with the weight read for every row and sums through ds_bpermute), 50
// at 768 (59), 49 at 1024 (59), 56 at 4096 (77); fp32 49 at 768 (50), 51 at 4096
// (71).  Loading the next round ahead as the forward kernel does changed nothing
// here (three operands in flight and 16 waves a CU cover the latency) and cost the
// registers.
template <int DT, int L, int M, int B>
__global__ __launch_bounds__(B, 4) void k_norm_bwd(NormBwd a) {
  constexpr int R = B / L, COLS = L * M * 4, ES = DT == 0 ? 4 : 2;
  constexpr bool KEEP = M < 4 || DT == 1;
  __shared__ float sm[2][2][16];
  __shared__ float cols[L <= 64 ? B / 64 * COLS : 1];
  const RowLane<L> at;
  const uint32_t C = (uint32_t)a.C;
  const int skip = (4 - (int)(C & 3)) & 3;
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t r0 = (int64_t)blockIdx.x * R;
  float keep[KEEP ? M : 1][4], gw[M][4] = {}, gb[M][4] = {};
  auto weight = [&](uint32_t c0, int j, float(&w)[4]) {
    const uint32_t c = c0 + j * L * 4;
    load_quad_params(a.weight, a.param_dt, c, c < C, c + 4 > C, skip, w);
  };
  if constexpr (KEEP) {
#pragma unroll
    for (int j = 0; j < M; ++j) weight((uint32_t)at.lane * 4, j, keep[j]);
  }
  for (int turn = 0; r0 < a.T; r0 += step, turn ^= 1) {
    const RowAt<DT, L> p(at, r0, a.T, a.C);
    RowQuads<DT, L, M> g, h, q;
    g.load(a.g_y, p.base, p.off, p.c0, C, skip, p.live);
    h.load(a.h, p.base, p.off, p.c0, C, skip, p.live);
    if (a.g_h) q.load(a.g_h, p.base, p.off, p.c0, C, skip, p.live);
    const float mean = p.live ? a.mean[p.row] : 0.f;
    const float rstd = p.live ? a.rstd[p.row] : 0.f;
    float s[2] = {0.f, 0.f};  // of u, of u n
#pragma unroll
    for (int j = 0; j < M; ++j) {
      float w[4];
      if constexpr (!KEEP) weight(p.c0, j, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = g.at(j, k), x = (h.at(j, k) - mean) * rstd;
        const float u = v * (KEEP ? keep[KEEP ? j : 0][k] : w[k]);
        s[0] += u;
        s[1] += u * x;
        gw[j][k] += v * x;
        gb[j][k] += v;
      }
    }
    row_sums<L>(s, sm[turn]);
    const float su = s[0] / (float)C, sn = s[1] / (float)C;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const uint32_t c = p.c0 + j * L * 4;
      float w[4], o[4];
      if constexpr (!KEEP) weight(p.c0, j, w);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        o[k] = rstd * (g.at(j, k) * (KEEP ? keep[KEEP ? j : 0][k] : w[k]) - su -
                       (h.at(j, k) - mean) * rstd * sn);
      if (a.g_h) {
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] += q.at(j, k);
      }
      store_quad<DT>(static_cast<char*>(a.g_x) + p.base, p.off + c * ES, p.live && c < C,
                     c + 4 > C, skip, make_quad<DT>(o));
    }
  }
  if constexpr (L > 64) {
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t c = (uint32_t)(at.lane + j * L) * 4 + k;
        if (c < C) {
          put_column(a, blockIdx.x, 0, c, gw[j][k]);
          put_column(a, blockIdx.x, 1, c, gb[j][k]);
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
        for (int k = 0; k < 4; ++k) {
          const float v = lanes_sum_across<L>(side ? gb[j][k] : gw[j][k]);
          if ((threadIdx.x & 63) < L) cols[wave * COLS + (at.lane + j * L) * 4 + k] = v;
        }
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < COLS; c += B)
        if (c < C) {
          float v = cols[c];
#pragma unroll
          for (int w = 1; w < B / 64; ++w) v += cols[w * COLS + c];
          put_column(a, blockIdx.x, side, c, v);
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
      put_column(a, blockIdx.y, k & 1, col,
                 (sm[0][l][k] + sm[1][l][k]) + (sm[2][l][k] + sm[3][l][k]));
  }
}

// Fold of the partial column sums part [parts][2][C] in a fixed order, in
// fp64: FOLD columns per workgroup from column col0 on, its 1024 / FOLD groups
// of lanes take the parts in turn and are joined within each wave, then across
// the 16 waves; blockIdx.y 0: g_weight, 1: g_bias.
// (16, 32 and 64 columns: the backward of 4096 columns fp32 takes 53.7, 51.2 and
// 51.9 us, of 768 48.7, 49.7 and 49.0.)
constexpr int FOLD = 32;
__global__ __launch_bounds__(1024) void k_norm_fold(NormBwd a, int64_t col0) {
  __shared__ double sm[16][FOLD];
  const int lane = threadIdx.x & (FOLD - 1), slot = threadIdx.x / FOLD;
  const int64_t C = a.C, c = col0 + (int64_t)blockIdx.x * FOLD + lane;
  double s = 0.0;
  if (c < C) {
#pragma unroll 8
    for (int64_t p = slot; p < a.parts; p += 1024 / FOLD)
      s += (double)a.part[(p * 2 + blockIdx.y) * C + c];
  }
  s = lanes_sum_across<FOLD>(s);
  if ((threadIdx.x & 63) < FOLD) sm[threadIdx.x >> 6][lane] = s;
  __syncthreads();
  if (threadIdx.x >= FOLD || c >= C) return;
  s = 0.0;
#pragma unroll
  for (int q = 0; q < 16; ++q) s += sm[q][lane];
  put_param(blockIdx.y ? a.g_bias : a.g_weight, a.param_dt, c, (float)s);
}

// ------------------------------------------------------------ launches
// Lanes and quads per row, by the length of the row.  A wave has a row up to 1024
// columns, without a barrier (forward of 1000 bf16 columns with 64 x 4 and 128 x 2:
// 46 and 51 us); above, more lanes rather than a fourth quad (8192 columns fp32 with
// 512 x 4 and 1024 x 2: 48 and 45), which the backward kernel has no registers for.
enum NormRow { ROW_8x1, ROW_16x1, ROW_32x1, ROW_64x1, ROW_64x2, ROW_64x3, ROW_64x4, ROW_128x3,
               ROW_256x2, ROW_256x3, ROW_512x2, ROW_512x3, ROW_1024x2, ROW_1024x3, ROW_1024x4,
               ROW_WIDE };
static const int norm_lanes[] = {8, 16, 32, 64, 64, 64, 64, 128, 256, 256, 512, 512, 1024, 1024,
                                 1024};
static const int norm_quads[] = {1, 1, 1, 1, 2, 3, 4, 3, 2, 3, 2, 3, 2, 3, 4};

static NormRow norm_row(int64_t C) {
  if (C < 4) return ROW_WIDE;
  for (int r = 0; r < ROW_WIDE; ++r)
    if (C <= 4 * norm_lanes[r] * norm_quads[r]) return (NormRow)r;
  return ROW_WIDE;
}

#define HLQ_NORM_ROWS(F, BS)                                                                \
  case ROW_8x1: F(8, 1, BS); break;                                                         \
  case ROW_16x1: F(16, 1, BS); break;                                                       \
  case ROW_32x1: F(32, 1, BS); break;                                                       \
  case ROW_64x1: F(64, 1, BS); break;                                                       \
  case ROW_64x2: F(64, 2, BS); break;                                                       \
  case ROW_64x3: F(64, 3, BS); break;                                                       \
  case ROW_64x4: F(64, 4, BS); break;                                                    \
  case ROW_128x3: F(128, 3, 128); break;                                                    \
  case ROW_256x2: F(256, 2, 256); break;                                                    \
  case ROW_256x3: F(256, 3, 256); break;                                                    \
  case ROW_512x2: F(512, 2, 512); break;                                                    \
  case ROW_512x3: F(512, 3, 512); break;                                                    \
  case ROW_1024x2: F(1024, 2, 1024); break;                                                 \
  case ROW_1024x3: F(1024, 3, 1024); break;                                                 \
  case ROW_1024x4: F(1024, 4, 1024); break;

constexpr int NORM_BWD_THREADS = 512;  // workgroups of the backward kernel, L <= 64

// At most `most` workgroups for `need` rounds of one, all with as many rounds.
static int64_t even_rounds(int64_t need, int64_t most) {
  const int64_t rounds = (need + most - 1) / most;
  return (need + rounds - 1) / rounds;
}

// Workgroups of the backward kernel, each leaving one partial: up to 1024
// threads per CU, which all run at once (so not evened out as above: 512 of them
// take ViT-B's 1576 rounds in 19.8 us, 394 in 21.7), and half for fp32 rows of
// three quads a lane, which have as many bytes in flight and are more columns to
// fold (64 MiB operands, 512 and 1024 threads: 1200 columns 56.6 and 60.1 us, 1500
// 54.7 and 61.8, 2500 52.6 and 59.2, 3000 53.9 and 61.6, 4200 57.7 and 57.0, 6144
// 54.6 and 56.9; bf16 the other way about from 1200, 68.3 and 62.7, to 4200, 77.6 and
// 60.1), except where a row takes 1024 lanes: half of the CUs would have none (10000
// columns 73.9 and 60.1).  Few rows are one workgroup's, which writes the parameters'
// gradients itself: up to NORM_ALONE rounds of it (GPU time of 1, 2 and 4 rounds
// in one launch, and of as many rows in two: 768 columns 4.0, 5.2, 7.5 and 6.0 us;
// 4096 4.4, 5.5, 7.6 and 6.7; the second launch costs the host 2.3 us).
constexpr int NORM_ALONE = 2;
int64_t norm_parts(int64_t T, int64_t C, int dtype) {
  const NormRow r = norm_row(C);
  if (r == ROW_WIDE) return (T + 31) / 32 < 256 ? (T + 31) / 32 : 256;
  const int L = norm_lanes[r], B = L <= 64 ? NORM_BWD_THREADS : L;
  const int threads = dtype == 0 && L > 64 && L <= 512 && norm_quads[r] == 3 ? 512 : 1024;
  const int64_t need = (T + B / L - 1) / (B / L), most = 256 * threads / B;
  if (T == 0) return 0;
  if (need <= NORM_ALONE) return 1;
  return need < most ? need : most;
}

hipError_t launch_norm_forward(const NormFwd& a, int dtype, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
#define HLQ_F(L, M, B)                                                                      \
  do {                                                                                      \
    const dim3 g((unsigned)even_rounds((a.T + B / L - 1) / (B / L), 256 * 2048 / B));       \
    if (dtype == 0) return launch(k_norm_fwd<0, L, M, B>, g, B, s, a);                      \
    return launch(k_norm_fwd<1, L, M, B>, g, B, s, a);                                      \
  } while (0)
  switch (norm_row(a.C)) {
    HLQ_NORM_ROWS(HLQ_F, 256)
    default: break;
  }
#undef HLQ_F
  if (dtype == 0) return launch(k_norm_fwd_wide<0>, rows_grid(a.T), 256, s, a);
  return launch(k_norm_fwd_wide<1>, rows_grid(a.T), 256, s, a);
}

// g_x and the partial column sums.
static hipError_t launch_norm_gx(const NormBwd& a, int dtype, hipStream_t s) {
  const int N = dtype == 0 ? 4 : 8;
  const dim3 g((unsigned)a.parts), wide(cdiv(a.C, 64 * N), (unsigned)a.parts);
#define HLQ_B(L, M, B)                                                                      \
  do {                                                                                      \
    if (dtype == 0) return launch(k_norm_bwd<0, L, M, B>, g, B, s, a);                      \
    return launch(k_norm_bwd<1, L, M, B>, g, B, s, a);                                      \
  } while (0)
  switch (norm_row(a.C)) {
    HLQ_NORM_ROWS(HLQ_B, NORM_BWD_THREADS)
    default: break;
  }
#undef HLQ_B
  const hipError_t e = dtype == 0 ? launch(k_norm_gx_wide<0>, rows_grid(a.T), 256, s, a)
                                  : launch(k_norm_gx_wide<1>, rows_grid(a.T), 256, s, a);
  if (e != hipSuccess) return e;
  if (dtype == 0) return launch(k_norm_columns<0>, wide, 256, s, a);
  return launch(k_norm_columns<1>, wide, 256, s, a);
}

hipError_t launch_norm_backward(const NormBwd& a, int dtype, hipStream_t s) {
  hipError_t e = a.T ? launch_norm_gx(a, dtype, s) : hipSuccess;
  if (a.parts == 1) return e;
  // 2^24 columns a launch (a launch holds fewer than 2^32 threads)
  for (int64_t c = 0; c < a.C && e == hipSuccess; c += 1 << 24) {
    const int64_t n = a.C - c < (1 << 24) ? a.C - c : 1 << 24;
    e = launch(k_norm_fold, dim3(cdiv(n, FOLD), a.g_bias ? 2 : 1), 1024, s, a, c);
  }
  return e;
}
#undef HLQ_NORM_ROWS

}  // namespace hlq
