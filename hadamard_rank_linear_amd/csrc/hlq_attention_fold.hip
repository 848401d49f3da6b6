// What follows the attention kernels: the join of the keys' shares of a row, and
// the sums of the position bias's gradient over the work items.
#include "hlq_rows.h"

namespace hlq {
namespace {

// A wave a row of (token, head): with (m_p, l_p) of share p in powers of two and M
// the largest m, o = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p.  Lane p holds
// share p's factor (at most 64 shares).  The shares' sums are loaded AHEAD at a time,
// also those that no share has written, and are not used then.  Bound by latency: 256
// rows of 16 shares 5 us, one at a time 6.5.
template <int DT>
__global__ __launch_bounds__(256) void k_attention_join(AttnFwd a) {
  typedef typename Piece<DT>::Elem E;
  constexpr int AHEAD = 8;
  const AttnShape& g = a.g;
  const int lane = threadIdx.x & 63;
  const int64_t rows = g.Tq * g.heads;
  for (int64_t r = blockIdx.x * 4ll + (threadIdx.x >> 6); r < rows; r += gridDim.x * 4ll) {
    float m = -__builtin_inff(), l = 0.f;
    if (lane < g.splits) {
      const float2 v = *reinterpret_cast<const float2*>(a.ml + (lane * rows + r) * 2);
      m = v.x;
      l = v.y;
    }
    const float top = lanes_max(m), base = top == -__builtin_inff() ? 0.f : top;
    const float f = __builtin_amdgcn_exp2f(m - base);
    const float total = lanes_sum<64>(f * l);
    const int64_t token = r / g.heads;
    const int head = (int)(r % g.heads);
    E* const o = static_cast<E*>(a.o.data) + token * a.o.token + head * a.o.head;
    for (int d = lane; d - lane < g.D; d += 64) {
      const float* const part = a.po + r * g.D + min(d, g.D - 1);
      float v = 0.f;
      for (int p0 = 0; p0 < g.splits; p0 += AHEAD) {
        float x[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          x[i] = part[min(p0 + i, (int)g.splits - 1) * rows * g.D];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const int p = min(p0 + i, 63);
          const float w = __shfl(f, p), k = __shfl(l, p);
          // a share that has seen no key (or is none) has written no sums
          if (k != 0.f) v += w * x[i];
        }
      }
      v = total == 0.f ? 0.f : v / total;
      if (d < g.D) {
        if constexpr (DT == 0) o[d] = v;
        else o[d] = (uint16_t)pack_bf16(v, 0.f);
      }
    }
    if (lane == 0)
      a.lse[head * g.Tq + token] = total == 0.f
                                       ? -__builtin_inff()
                                       : (top + __builtin_amdgcn_logf(total)) * 0.69314718055994530942f;
  }
}

// g_bias[bucket][head]: a workgroup a head; thread t adds bucket t % buckets of
// every 1024 / buckets-th item, four at a time, then one sum over the threads of a
// bucket.  fp64, always in the same order.  A sequence's items lie together, those of
// two sequences heads * tiles apart.  Bound by latency: 144 items a head 5.2 us, with 256
// threads and a division an item 9.
__global__ __launch_bounds__(1024) void k_attention_bias(const float* part, int64_t S, unsigned tiles,
                                                         int heads, int buckets, int param_dt,
                                                         void* g_bias) {
  __shared__ double sm[1024];
  const int head = blockIdx.x, ways = 1024 / buckets;
  const int b = (int)threadIdx.x % buckets, way = (int)threadIdx.x / buckets;
  double v = 0.0;
  if (way < ways) {
    const float* const mine = part + (int64_t)head * tiles * buckets + b;
    const int64_t next = (int64_t)heads * tiles * buckets;
    const auto at = [&](int64_t s, unsigned t) {
      return s < S ? mine[s * next + (int64_t)t * buckets] : 0.f;
    };
    int64_t s = way / tiles;
    unsigned t = way % tiles;
    const unsigned ds = ways / tiles, dt = ways % tiles;
    while (s < S) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = at(s, t);
        s += ds;
        t += dt;
        if (t >= tiles) {
          t -= tiles;
          ++s;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v += x[i];
    }
  }
  sm[threadIdx.x] = v;
  __syncthreads();
  if (way == 0) {
    for (int w = 1; w < ways; ++w) v += sm[w * buckets + b];
    const int64_t at = (int64_t)b * heads + head;
    if (param_dt == 0) static_cast<float*>(g_bias)[at] = (float)v;
    else static_cast<uint16_t*>(g_bias)[at] = (uint16_t)pack_bf16((float)v, 0.f);
  }
}

}  // namespace

hipError_t launch_attention_join(const AttnFwd& a, int dtype, hipStream_t s) {
  const int64_t groups = (a.g.Tq * a.g.heads + 3) / 4;
  const dim3 grid((unsigned)(groups < (1 << 20) ? groups : 1 << 20));
  return launch(dtype == 0 ? k_attention_join<0> : k_attention_join<1>, grid, 256, s, a);
}

hipError_t launch_attention_bias(const float* part, int64_t S, int64_t tiles, int heads,
                                 int buckets, int param_dt, void* g_bias, hipStream_t s) {
  return launch(k_attention_bias, dim3((unsigned)heads), 1024, s, part, S, (unsigned)tiles, heads, buckets,
                param_dt, g_bias);
}

}  // namespace hlq
