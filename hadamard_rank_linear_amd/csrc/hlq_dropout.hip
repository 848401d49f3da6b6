// Dropout with the residual addition.  The mask is a function of the element's
// index: block i / 8 of Philox 4x32 with seven rounds (Salmon, Moraes, Dror, Shaw:
// "Parallel random numbers: as easy as 1, 2, 3", 2011; seven rounds are the
// fewest that passed the paper's tests) gives eight elements 16 bits each, and
// the backward pass draws them again.  Memory bound: 16 bytes of each operand a
// thread and step, about 20 integer operations an element between them.  12608 x 768
// bf16 with the residual 10.2 us (5.7 TB/s, the caches help), the backward pass of 117
// million elements 87 us (5.4 TB/s).
#include "hlq_rows.h"

namespace hlq {
namespace {

struct Words {
  uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                        uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)q;
    c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

// Eight elements a step: one piece in bf16, two in fp32.
template <int DT, bool RES>
__global__ __launch_bounds__(256) void k_dropout(DropArgs a) {
  constexpr int P = DT == 0 ? 2 : 1, N = Piece<DT>::N;
  const uint64_t key = (uint64_t)a.seed[0], step = (uint64_t)a.seed[1];
  const int64_t blocks = (a.n + 7) / 8, stride = (int64_t)gridDim.x * 256;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < blocks; i += stride) {
    u32x4 x[P], r[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t e = i * 8 + p * N;
      x[p] = r[p] = (u32x4){0u, 0u, 0u, 0u};
      if (e < a.n) {
        x[p] = load_piece<DT>(a.x, e, a.n - e);
        if constexpr (RES) r[p] = load_piece<DT>(a.residual, e, a.n - e);
      }
    }
    const Words w = philox((uint32_t)i, a.site, (uint32_t)step, (uint32_t)(step >> 32),
                           (uint32_t)key, (uint32_t)(key >> 32));
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t e = i * 8 + p * N;
      if (e >= a.n) continue;
      float y[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int j = p * N + k;
        const uint32_t bits = j & 1 ? w.w[j / 2] >> 16 : w.w[j / 2] & 0xFFFFu;
        y[k] = bits >= a.limit ? piece_at<DT>(x[p], k) * a.scale : 0.f;
        if constexpr (RES) y[k] = piece_at<DT>(r[p], k) + y[k];
      }
      store_piece<DT>(a.y, e, a.n - e, make_piece<DT>(y));
    }
  }
}

}  // namespace

hipError_t launch_dropout(const DropArgs& a, int dtype, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  const int64_t groups = ((a.n + 7) / 8 + 255) / 256;
  const dim3 grid((unsigned)(groups < 4096 ? groups : 4096));
  if (dtype == 0)
    return launch(a.residual ? k_dropout<0, true> : k_dropout<0, false>, grid, 256, s, a);
  return launch(a.residual ? k_dropout<1, true> : k_dropout<1, false>, grid, 256, s, a);
}

}  // namespace hlq
