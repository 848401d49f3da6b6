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

// exp(scale d) for d <= 0, scale log2(e) = c_hi + c_lo.  c rounded to fp32
// alone shifts every exponential of a sum the same way (2e-7 of a typical log
// probability, and a sequence adds hundreds); c_lo > 0, so -inf stays -inf.
__device__ __forceinline__ float exp_scaled(float d, float c_hi, float c_lo) {
  return exp2_hw(__builtin_fmaf(d, c_hi, d * c_lo));
}

// ------------------------------------------------------------ pieces of a row
// A row is split into 16-byte pieces at 16-byte boundaries, thread i of W taking
// pieces i, i + W, ...  Positions count elements from the boundary at or before
// the row's start, so the row is positions head .. end - 1; addresses are a
// scalar base and a 32-bit byte offset.  Rows of an odd length start anywhere:
// pieces cut at the row's own start would cross boundaries in every access
// (the gradient of 4096 x 32003 bf16 takes 115 us that way, 87 here).
// What lies outside the row reads as -inf, which adds nothing to the sum.  The
// first and the last piece are read where they lie whole within the row and
// shifted into place (rows shorter than a piece: by elements).
//
// ST (streaming): non-temporal accesses, for rows that together would pass
// through the last-level cache without being found there again.  Scoring 4096 x
// 128256 bf16 takes 154 us instead of 174, 8190 x 32000 60 instead of 100, the
// policy loss over 2048 x 128256 184 instead of 192.  The gradient kernel is the
// other way about (148 us with, 140 without, at 8190 x 32000 after its scoring).

template <int DT, bool ST>
struct Row {
  static constexpr int N = Piece<DT>::N, ES = DT == 0 ? 4 : 2;
  static constexpr uint32_t FILL = DT == 0 ? 0xFF800000u : 0xFF80FF80u;
  const char* base;  // of position 0 (uniform)
  uint32_t head, end;

  __device__ __forceinline__ Row(const void* x, int64_t row, int64_t ld, int64_t V) {
    base = static_cast<const char*>(x) + row * ld * ES;
    head = (uint32_t)(reinterpret_cast<uintptr_t>(base) & 15u) / ES;
    base -= head * ES;
    end = head + (uint32_t)V;
  }

  __device__ __forceinline__ u32x4 at(uint32_t p) const {
    const Loose* q = reinterpret_cast<const Loose*>(base + p * ES);
    if constexpr (ST) return __builtin_nontemporal_load(q);
    else return *q;
  }

  // The piece at position p (a multiple of N).
  __device__ __forceinline__ u32x4 load(uint32_t p) const {
    u32x4 r = {FILL, FILL, FILL, FILL};
    if (p >= head && p + N <= end) r = at(p);
    else if (p < end) edge(p, r);
    return r;
  }

  __device__ __forceinline__ void edge(uint32_t p, u32x4& r) const {
    if (end - head < (uint32_t)N) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (p + k >= head && p + k < end) {
          if constexpr (DT == 0) {
            r[k] = reinterpret_cast<const uint32_t*>(base)[p + k];
          } else {
            const uint32_t v = reinterpret_cast<const uint16_t*>(base)[p + k];
            r[k / 2] = (k & 1) ? (r[k / 2] & 0xFFFFu) | (v << 16) : (r[k / 2] & 0xFFFF0000u) | v;
          }
        }
    } else if (p < head) {
      r = at(head);
      const uint32_t up = head - p;
      if constexpr (DT == 0) {
        if (up & 1) r = (u32x4){FILL, r[0], r[1], r[2]};
        if (up & 2) r = (u32x4){FILL, FILL, r[0], r[1]};
      } else {
        if (up & 1)
          r = (u32x4){(FILL >> 16) | (r[0] << 16), (r[0] >> 16) | (r[1] << 16),
                      (r[1] >> 16) | (r[2] << 16), (r[2] >> 16) | (r[3] << 16)};
        if (up & 2) r = (u32x4){FILL, r[0], r[1], r[2]};
        if (up & 4) r = (u32x4){FILL, FILL, r[0], r[1]};
      }
    } else {
      r = at(end - N);
      const uint32_t down = p + N - end;
      if constexpr (DT == 0) {
        if (down & 1) r = (u32x4){r[1], r[2], r[3], FILL};
        if (down & 2) r = (u32x4){r[2], r[3], FILL, FILL};
      } else {
        if (down & 1)
          r = (u32x4){(r[0] >> 16) | (r[1] << 16), (r[1] >> 16) | (r[2] << 16),
                      (r[2] >> 16) | (r[3] << 16), (r[3] >> 16) | (FILL << 16)};
        if (down & 2) r = (u32x4){r[1], r[2], r[3], FILL};
        if (down & 4) r = (u32x4){r[2], r[3], FILL, FILL};
      }
    }
  }

  __device__ __forceinline__ float element(uint32_t t) const {
    return load1<DT>(base, head + t);
  }
};

// Stores a piece of a row of the gradient, positions as in its row of logits.
template <int DT, bool ST>
struct OutRow {
  static constexpr int N = Piece<DT>::N, ES = DT == 0 ? 4 : 2;
  char* base;
  uint32_t head, end;

  __device__ __forceinline__ OutRow(const LogitArgs& a, int64_t row, uint32_t head_)
      : head(head_), end(head_ + (uint32_t)a.V) {
    base = static_cast<char*>(a.g_x) + row * a.g_ld * ES - head * ES;
  }
  __device__ __forceinline__ void store(uint32_t p, const u32x4& r) const {
    if (p >= head && p + N <= end) {
      Loose* q = reinterpret_cast<Loose*>(base + p * ES);
      if constexpr (ST) __builtin_nontemporal_store(r, q);
      else *q = r;
    } else if (p < end) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (p + k >= head && p + k < end) {
          if constexpr (DT == 0) reinterpret_cast<uint32_t*>(base)[p + k] = r[k];
          else reinterpret_cast<uint16_t*>(base)[p + k] = (uint16_t)(r[k / 2] >> (16 * (k & 1)));
        }
    }
  }
};

// Makes the compiler unpack a piece again where it is used next, instead of
// keeping its elements in a register each from one use to the other.
__device__ __forceinline__ void keep_packed(u32x4& r) { asm volatile("" : "+v"(r)); }

// Maximum and sum relative to it of P pieces at positions e0, e0 + step, ...,
// joined to a thread's running (m, s).  Pieces past the row's end cost nothing
// where the whole wave's are.  The sum is fp32: a thread adds V / threads terms and
// the threads join over a tree, off by 4.5e-8 of a log probability at 128256 logits.
// An fp64 sum (2.5e-8) would be a conversion and a wider addition for every logit.
template <int DT, int P>
__device__ __forceinline__ void accumulate(u32x4 (&r)[P], uint32_t e0, uint32_t step, uint32_t end,
                                           const LogitArgs& a, float& m, float& s) {
  constexpr int N = Piece<DT>::N;
  float top = m;
#pragma unroll
  for (int j = 0; j < P; ++j)
    if (e0 + j * step < end) {
#pragma unroll
      for (int k = 0; k < N; ++k) top = fmaxf(top, piece_at<DT>(r[j], k));
    }
  const float ref = ref_of(top);
  float t = s * exp_scaled(m - ref, a.c_hi, a.c_lo);
#pragma unroll
  for (int j = 0; j < P; ++j)
    if (e0 + j * step < end) {
      keep_packed(r[j]);
#pragma unroll
      for (int k = 0; k < N; ++k) t += exp_scaled(piece_at<DT>(r[j], k) - ref, a.c_hi, a.c_lo);
    }
  m = top;
  s = t;
}

// Joins the threads' (m, s) over a workgroup of W; every thread gets the row's.  sm: [2][16] floats.
template <int W>
__device__ __forceinline__ void join_stats(const LogitArgs& a, float (*sm)[16], float& m,
                                           float& s) {
  float top = lanes_max(m);
  s = lanes_sum<64>(s * exp_scaled(m - ref_of(top), a.c_hi, a.c_lo));
  if constexpr (W > 64) {
    if ((threadIdx.x & 63) == 0) {
      sm[0][threadIdx.x >> 6] = top;
      sm[1][threadIdx.x >> 6] = s;
    }
    __syncthreads();
    m = sm[0][threadIdx.x & (W / 64 - 1)];
    s = sm[1][threadIdx.x & (W / 64 - 1)];
    top = lanes_max<W / 64>(m);
    s = lanes_sum<W / 64>(s * exp_scaled(m - ref_of(top), a.c_hi, a.c_lo));
  }
  m = top;
}

template <int DT, bool ST>
__device__ __forceinline__ Row<DT, ST> row_of(const LogitArgs& a, int64_t row) {
  return Row<DT, ST>(a.logits, row, a.ld, a.V);
}

// scale (x_t - m) - log s; s is 0 (nothing but -inf), NaN, or at least 1.  The
// logarithm splits off the exponent, so fp32 suffices for the rest of it: off
// by 2^-25, where log(double) costs a row about as much as all its reductions.
__device__ __forceinline__ double logprob_of(float xt, float m, float s, double scale) {
  if (!(s >= 1.f)) return s == 0.f ? -__builtin_huge_val() : (double)s;
  const uint32_t b = __float_as_uint(s);
  int e = (int)(b >> 23) - 127;
  float f = __uint_as_float((b & 0x7FFFFFu) | 0x3F800000u);
  if (f >= 1.5f) {
    f *= 0.5f;
    ++e;
  }
  return ((double)xt - (double)m) * scale - ((double)e * 0.69314718055994530942 + (double)logf(f));
}

// Log probabilities: a workgroup of W threads per row, P pieces of a thread in
// flight at a time.
template <int DT, bool ST, int W, int P>
__global__ __launch_bounds__(W) void k_logprob(LogitArgs a) {
  constexpr int N = Piece<DT>::N;
  __shared__ float sm[2][16];
  const int64_t row = a.row0 + blockIdx.x, t = a.targets[row];
  float m = 0.f, s = 1.f, lp = 0.f;
  if (t >= 0 && t < a.V) {
    const Row<DT, ST> x = row_of<DT, ST>(a, row);
    const float xt = x.element((uint32_t)t);
    m = -__builtin_huge_valf();
    s = 0.f;
    for (uint32_t e0 = threadIdx.x * N; e0 < x.end; e0 += W * N * P) {
      u32x4 r[P];
#pragma unroll
      for (int j = 0; j < P; ++j) r[j] = x.load(e0 + j * W * N);
      accumulate<DT, P>(r, e0, W * N, x.end, a, m, s);
    }
    join_stats<W>(a, sm, m, s);
    if (threadIdx.x == 0) lp = (float)logprob_of(xt, m, s, a.scale);
  }
  if (threadIdx.x == 0) {
    a.logprob[row] = lp;
    a.stats[2 * row] = m;
    a.stats[2 * row + 1] = s;
  }
}

// Gradient of a row's piece at position e: f ([v = t] - e_v / s), k_s = -f / s,
// t the target's position.  The exponent has c in one word: off by 2^-24 of itself
// and as much from the product, 1e-6 of an exponential 20 below the maximum (which is
// 2e-9), and unlike in the sum nothing adds these errors up.
template <int DT>
__device__ __forceinline__ u32x4 gradient_piece(const u32x4& r, uint32_t e, uint32_t t, float c,
                                                float f, float k_s, float m) {
  constexpr int N = Piece<DT>::N;
  float o[N];
#pragma unroll
  for (int k = 0; k < N; ++k) o[k] = k_s * exp2_hw((piece_at<DT>(r, k) - m) * c);
  if (t - e < (uint32_t)N) {
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] += t - e == (uint32_t)k ? f : 0.f;
  }
  return make_piece<DT>(o);
}

template <int DT, bool ST, int W>
__device__ __forceinline__ void zero_row(const OutRow<DT, ST>& g) {
  const u32x4 z = {0u, 0u, 0u, 0u};
  for (uint32_t e = threadIdx.x * g.N; e < g.end; e += W * g.N) g.store(e, z);
}

// The gradient of a row whose f is infinite (a banned target under a KL term): its
// limit, zero where [v = t] - e_v / s is, instead of inf * 0.  Rare, so the row is
// read again, from `first` on, whatever the kernel holds of it.
template <int DT, bool ST>
__device__ __forceinline__ void limit_row(const Row<DT, ST>& x, const OutRow<DT, ST>& g,
                                          uint32_t first, uint32_t step, uint32_t t, float c,
                                          float f, float m, float s) {
  constexpr int N = Piece<DT>::N;
  for (uint32_t e = first; e < x.end; e += step) {
    const u32x4 r = x.load(e);
    float o[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float d = (t - e == (uint32_t)k ? 1.f : 0.f) - exp2_hw((piece_at<DT>(r, k) - m) * c) / s;
      o[k] = d == 0.f ? 0.f : f * d;
    }
    g.store(e, make_piece<DT>(o));
  }
}

// Reads a row again and writes its gradient, P pieces of a thread in flight.  Where
// rows are few, gridDim.y workgroups share one (SHARED; a stride known only at run
// time costs 8190 x 32000 bf16 9 us of 146 otherwise).
template <int DT, int W, int P, bool SHARED>
__global__ __launch_bounds__(W) void k_logprob_grad(LogitArgs a) {
  constexpr int N = Piece<DT>::N;
  const int64_t row = a.row0 + blockIdx.x, t = a.targets[row];
  const bool live = t >= 0 && t < a.V;
  const float f = live ? a.g_logprob[row] * (float)a.scale : 0.f;
  const float m = a.stats[2 * row], s = a.stats[2 * row + 1];
  const Row<DT, false> x = row_of<DT, false>(a, row);
  const OutRow<DT, false> g(a, row, x.head);
  const uint32_t first = ((SHARED ? blockIdx.y * W : 0) + threadIdx.x) * N;
  const uint32_t step = (SHARED ? gridDim.y : 1) * W * N;
  if (f == 0.f || s == 0.f) {
    const u32x4 z = {0u, 0u, 0u, 0u};
    for (uint32_t e = first; e < g.end; e += step) g.store(e, z);
    return;
  }
  if (__builtin_isinf(f)) {
    limit_row(x, g, first, step, x.head + (uint32_t)t, a.c, f, m, s);
    return;
  }
  const float k_s = -f / s;
  for (uint32_t e0 = first; e0 < x.end; e0 += step * P) {
    u32x4 r[P];
#pragma unroll
    for (int j = 0; j < P; ++j) r[j] = x.load(e0 + j * step);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const uint32_t e = e0 + j * step;
      if (e < x.end) g.store(e, gradient_piece<DT>(r[j], e, x.head + (uint32_t)t, a.c, f, k_s, m));
    }
  }
}

// ------------------------------------------------------------ policy loss
// What a token brings to the loss besides its log probability.
struct PolicyToken {
  float old, advantage, weight, ref;
};
__device__ __forceinline__ PolicyToken policy_load(const PolicyArgs& p, int64_t i) {
  return PolicyToken{p.old_logprob[i], p.advantage[i], p.weight ? p.weight[i] : 1.f,
                     p.ref_logprob ? p.ref_logprob[i] : 0.f};
}

// The terms of one token, in fp64 from the log probability: w times the loss,
// the KL estimate and whether the clamped ratio counted; returns the gradient.
__device__ __forceinline__ double policy_token(const PolicyArgs& p, const PolicyToken& q, double lp,
                                               double (&term)[3]) {
  const double w = (double)q.weight, A = (double)q.advantage;
  const double r = exp(lp - (double)q.old);
  const double lo = 1.0 - p.clip_low, hi = 1.0 + p.clip_high;
  const double bounded = r < lo ? lo : (r > hi ? hi : r);
  // a ratio past the range counts as a finite one under an advantage of zero
  const double free_ = A == 0.0 && r == __builtin_huge_val() ? 0.0 : r * A, clipped = bounded * A;
  const bool cut = clipped < free_;
  double kl = 0.0, g = cut ? 0.0 : -free_;
  if (p.ref_logprob) {
    const double d = (double)q.ref - lp, x = expm1(d);
    kl = x == __builtin_huge_val() ? x : x - d;  // d = inf too, where lp is -inf
    g -= p.kl_coef * x;
  }
  term[0] = w * (p.kl_coef * kl - (cut ? clipped : free_));
  term[1] = w * kl;
  term[2] = cut ? w : 0.0;
  return w * g;
}

// The row's loss terms and the gradient of its log probability, by thread 0;
// every thread gets the gradient.
__device__ __forceinline__ float policy_row(const LogitArgs& a, const PolicyArgs& p, int64_t row,
                                            const PolicyToken& q, bool live, float xt, float m,
                                            float s, float* sg) {
  if (threadIdx.x == 0) {
    double term[3] = {0.0, 0.0, 0.0}, lp = 0.0, g = 0.0;
    if (live) {
      lp = logprob_of(xt, m, s, a.scale);
      g = policy_token(p, q, lp, term);
    }
    a.logprob[row] = (float)lp;
#pragma unroll
    for (int k = 0; k < 3; ++k) p.terms[3 * row + k] = term[k];
    *sg = (float)g * (float)a.scale;
  }
  __syncthreads();
  return *sg;
}

// Rows of up to W * P pieces: held in registers between the statistics and the
// gradient, so that the logits are read once.
template <int DT, bool ST, int W, int P>
__global__ __launch_bounds__(W, 4) void k_policy_regs(LogitArgs a, PolicyArgs p) {
  constexpr int N = Piece<DT>::N;
  __shared__ float sm[2][16], sg;
  const int64_t row = a.row0 + blockIdx.x, t = a.targets[row];
  const PolicyToken q = policy_load(p, row);
  const bool live = t >= 0 && t < a.V && q.weight != 0.f;
  const Row<DT, ST> x = row_of<DT, ST>(a, row);
  u32x4 r[P];
  float m = -__builtin_huge_valf(), s = 0.f, xt = 0.f;
  if (live) {
    xt = x.element((uint32_t)t);
#pragma unroll
    for (int j = 0; j < P; ++j) r[j] = x.load((threadIdx.x + j * W) * N);
    accumulate<DT, P>(r, threadIdx.x * N, W * N, x.end, a, m, s);
    join_stats<W>(a, sm, m, s);
  }
  const float f = policy_row(a, p, row, q, live, xt, m, s, &sg);
  const OutRow<DT, ST> g(a, row, x.head);
  if (f == 0.f || s == 0.f) {
    zero_row<DT, ST, W>(g);
    return;
  }
  if (__builtin_isinf(f)) {
    limit_row(x, g, threadIdx.x * N, W * N, x.head + (uint32_t)t, a.c, f, m, s);
    return;
  }
  const float k_s = -f / s;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    keep_packed(r[j]);
    const uint32_t e = (threadIdx.x + j * W) * N;
    if (e < x.end)
      g.store(e, gradient_piece<DT>(r[j], e, x.head + (uint32_t)t, a.c, f, k_s, m));
  }
}

// Longer rows: the first W * H pieces are held, the others are read twice, the
// second time from the last-level cache (524 x 100003 fp32, H 0, 8 and 16: 122, 98
// and 96 us; 400 x 131072: 117, 91 and 87).
template <int DT, int W, int P, int H>
__global__ __launch_bounds__(W, 4) void k_policy_long(LogitArgs a, PolicyArgs p) {
  constexpr int N = Piece<DT>::N;
  constexpr uint32_t REST = W * H * N;
  __shared__ float sm[2][16], sg;
  const int64_t row = a.row0 + blockIdx.x, t = a.targets[row];
  const PolicyToken q = policy_load(p, row);
  const bool live = t >= 0 && t < a.V && q.weight != 0.f;
  const Row<DT, false> x = row_of<DT, false>(a, row);
  const Row<DT, true> once = row_of<DT, true>(a, row);
  u32x4 held[H];
  float m = -__builtin_huge_valf(), s = 0.f, xt = 0.f;
  if (live) {
    xt = x.element((uint32_t)t);
    for (uint32_t e0 = REST + threadIdx.x * N; e0 < x.end; e0 += W * N * P) {
      u32x4 r[P];
#pragma unroll
      for (int j = 0; j < P; ++j) r[j] = x.load(e0 + j * W * N);
      accumulate<DT, P>(r, e0, W * N, x.end, a, m, s);
    }
#pragma unroll
    for (int j = 0; j < H; ++j) held[j] = once.load((threadIdx.x + j * W) * N);
    accumulate<DT, H>(held, threadIdx.x * N, W * N, x.end, a, m, s);
    join_stats<W>(a, sm, m, s);
  }
  const float f = policy_row(a, p, row, q, live, xt, m, s, &sg);
  const OutRow<DT, true> g(a, row, x.head);
  if (f == 0.f || s == 0.f) {
    zero_row<DT, true, W>(g);
    return;
  }
  if (__builtin_isinf(f)) {
    limit_row(once, g, threadIdx.x * N, W * N, x.head + (uint32_t)t, a.c, f, m, s);
    return;
  }
  const float k_s = -f / s;
  const uint32_t at = x.head + (uint32_t)t;
#pragma unroll
  for (int j = 0; j < H; ++j) {
    keep_packed(held[j]);
    const uint32_t e = (threadIdx.x + j * W) * N;
    g.store(e, gradient_piece<DT>(held[j], e, at, a.c, f, k_s, m));
  }
  for (uint32_t e0 = REST + threadIdx.x * N; e0 < x.end; e0 += W * N * P) {
    u32x4 r[P];
#pragma unroll
    for (int j = 0; j < P; ++j) r[j] = x.load(e0 + j * W * N);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const uint32_t e = e0 + j * W * N;
      if (e < x.end) g.store(e, gradient_piece<DT>(r[j], e, at, a.c, f, k_s, m));
    }
  }
}

__global__ __launch_bounds__(256) void k_policy(PolicyArgs p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.T) return;
  double term[3] = {0.0, 0.0, 0.0}, g = 0.0;
  const PolicyToken q = policy_load(p, i);
  if (q.weight != 0.f) g = policy_token(p, q, (double)p.logprob[i], term);
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
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < n; i += 1024)
#pragma unroll
    for (int k = 0; k < K; ++k) acc[k] += terms[K * i + k];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    acc[k] = lanes_sum<64>(acc[k]);
    if ((threadIdx.x & 63) == 0) sm[k][threadIdx.x >> 6] = acc[k];
  }
  __syncthreads();
  if (threadIdx.x < 16)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const double v = lanes_sum<16>(sm[k][threadIdx.x]);
      if (threadIdx.x == 0) sums[k] = (float)(v * scale);
    }
}

// ------------------------------------------------------------ preference loss
__device__ __forceinline__ int64_t bound(int64_t v, int64_t lo, int64_t hi) {
  return v < lo ? lo : (v > hi ? hi : v);
}

// One group of G threads per pair (a workgroup, or a wave of it: G = 64): both
// sequences' sums in fp64, then the margin, the loss and the gradient of their
// tokens.  Returns the pair's loss.
template <int G>
__device__ __forceinline__ double preference_pair(const PrefArgs& p, int64_t pair, double (*sm)[4]) {
  const int lane = threadIdx.x % G;
  int64_t lo[2], hi[2];
  double v[4] = {0.0, 0.0, 0.0, 0.0};  // sum and weight of the chosen, of the rejected one
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int64_t i = pair + q * p.P;
    lo[q] = bound(p.start[i], 0, p.T);
    hi[q] = bound(p.start[i + 1], lo[q], p.T);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll 4
    for (int64_t t = lo[q] + lane; t < hi[q]; t += G) {
      const float w = p.weight ? p.weight[t] : 1.f;
      const float lp = p.logprob[t], ref = p.ref_logprob ? p.ref_logprob[t] : 0.f;
      v[2 * q] += w != 0.f ? (double)w * ((double)lp - (double)ref) : 0.0;
      v[2 * q + 1] += (double)w;
    }
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = lanes_sum<64>(v[k]);
  if constexpr (G > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < 4; ++k) sm[wave][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = lanes_sum<G / 64>(sm[threadIdx.x & (G / 64 - 1)][k]);
  }
  double part[2] = {1.0, 1.0};
  if (p.mean) {
    part[0] = v[1] > 0.0 ? 1.0 / v[1] : 0.0;
    part[1] = v[3] > 0.0 ? 1.0 / v[3] : 0.0;
  }
  const double z = p.beta * (v[0] * part[0] - v[2] * part[1]), e = p.smoothing;
  // with x = exp(-|z|): -log sigmoid(z) = log(1 + x) + max(-z, 0), and
  // sigmoid(z) - 1 = -x / (1 + x) for z >= 0, -1 / (1 + x) below
  const double x = exp(-fabs(z)), share = 1.0 / (1.0 + x);
  const double g = p.beta / (double)p.P * ((z < 0.0 ? -share : -x * share) + e);
  if (lane == 0) p.margin[pair] = (float)z;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const double gq = (q ? -g : g) * part[q];
#pragma unroll 4
    for (int64_t t = lo[q] + lane; t < hi[q]; t += G) {
      const float w = p.weight ? p.weight[t] : 1.f;
      p.g_logprob[t] = w != 0.f ? (float)((double)w * gq) : 0.f;
    }
  }
  if (pair == 0) {  // tokens of no sequence, before the first bound or from the last one on
    const int64_t before = bound(p.start[0], 0, p.T), from = bound(p.start[2 * p.P], before, p.T);
    for (int64_t t = lane; t < before; t += G) p.g_logprob[t] = 0.f;
    for (int64_t t = from + lane; t < p.T; t += G) p.g_logprob[t] = 0.f;
  }
  // an infinite margin counts where its side has a share (e or 1 - e), else not at all
  const double part_z = z < 0.0 ? 1.0 - e : e;
  return log1p(x) + (part_z == 0.0 ? 0.0 : part_z * fabs(z));
}

__global__ __launch_bounds__(1024) void k_preference(PrefArgs p) {
  __shared__ double sm[16][4];
  const int64_t pair = p.pair0 + blockIdx.x;
  const double loss = preference_pair<1024>(p, pair, sm);
  if (threadIdx.x == 0) p.terms[pair] = loss;
}

// All pairs in one workgroup, a wave per pair: one launch, no partials.
__global__ __launch_bounds__(1024) void k_preference_small(PrefArgs p) {
  __shared__ double sm[16];
  double loss = 0.0;
  for (int64_t pair = threadIdx.x >> 6; pair < p.P; pair += 16)
    loss += preference_pair<64>(p, pair, nullptr);
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = loss;
  __syncthreads();
  if (threadIdx.x < 16) {
    loss = lanes_sum<16>(sm[threadIdx.x]);
    if (threadIdx.x == 0) *p.loss = (float)(loss / (double)p.P);
  }
}

// ------------------------------------------------------------ launches
// Threads per row of n pieces: a wave for short rows, 512 for long ones (scored
// with 64, 256, 512 and 1024 threads a row, inputs displaced from the caches: 8190 x
// 1000 bf16 6.5, 10.9, 18.1 and 32.2 us; 15728 x 3000 20.9, 25.3, 40.4 and 70.5;
// 12790 x 4099 fp32 35.2, 36.9, 45.5 and 72.7; 8190 x 32000 bf16 87.3, 82.6, 78.2 and
// 87.1; 4096 x 128256 183, 162, 159 and 153, the one shape where 1024 would be ahead),
// and more where the rows are too few to fill the chip (3 x 32003: 16.0, 6.2, 5.7
// and 5.6; what is left there is the arithmetic of one CU, 10 us for a row of
// 131072, the same with 8 or 16 pieces of a thread in flight).
static int score_threads(int64_t T, int64_t n) {
  if (T < 256) return n <= 64 ? 64 : (n <= 512 ? 256 : 1024);
  return n <= 600 ? 64 : (n <= 2048 ? 256 : 512);
}

// The same for the gradient of 256 rows and more (4096 x 128256 bf16 with 64, 256,
// 512 and 1024 threads: 425, 420, 412 and 388 us; 8190 x 32000: 218, 206, 194 and
// 176; 8190 x 1000: 8.8, 11.2, 19.6 and 32.4; 15728 x 3000: 39.8, 35.8, 60.1 and 83.5;
// 12790 x 4099 fp32: 89.0, 78.3, 80.2 and 145).
static int grad_threads(int64_t n) {
  return n <= 256 ? 64 : (n <= 1024 ? 256 : n <= 2560 ? 512 : 1024);
}

// Pieces of a row, at most: one more where rows do not start at a boundary.
static int64_t row_pieces(const LogitArgs& a, int dtype) {
  const int64_t N = dtype == 0 ? 4 : 8;
  const bool at_boundary = (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 && a.ld % N == 0;
  return (a.V + (at_boundary ? 0 : N - 1) + N - 1) / N;
}

// One workgroup per row (or pair), 2^20 of them a launch (a launch holds fewer than
// 2^32 threads); `first` is where the kernel reads a launch's first one.
template <typename F>
static hipError_t for_rows(int64_t& first, int64_t n, F f) {
  hipError_t e = hipSuccess;
  for (first = 0; first < n && e == hipSuccess; first += 1 << 20) e = f(rows_grid(n - first));
  return e;
}
template <typename F>
static hipError_t for_rows(LogitArgs& a, F f) {
  return for_rows(a.row0, a.T, f);
}

template <int W, int P>
static hipError_t logprob_rows(LogitArgs& a, int dtype, hipStream_t s) {
  return for_rows(a, [&](dim3 g) {
    if (dtype == 0)
      return a.stream ? launch(k_logprob<0, true, W, P>, g, W, s, a)
                      : launch(k_logprob<0, false, W, P>, g, W, s, a);
    return a.stream ? launch(k_logprob<1, true, W, P>, g, W, s, a)
                    : launch(k_logprob<1, false, W, P>, g, W, s, a);
  });
}

hipError_t launch_logprob(LogitArgs a, int dtype, hipStream_t s) {
  switch (score_threads(a.T, row_pieces(a, dtype))) {
    case 64: return logprob_rows<64, 4>(a, dtype, s);
    case 256: return logprob_rows<256, 4>(a, dtype, s);
    case 512: return logprob_rows<512, 4>(a, dtype, s);
    default: return logprob_rows<1024, 4>(a, dtype, s);
  }
}

template <int W, int P, bool SHARED = false>
static hipError_t grad_rows(LogitArgs& a, int dtype, hipStream_t s, unsigned share = 1) {
  return for_rows(a, [&](dim3 g) {
    g.y = share;
    return dtype == 0 ? launch(k_logprob_grad<0, W, P, SHARED>, g, W, s, a)
                      : launch(k_logprob_grad<1, W, P, SHARED>, g, W, s, a);
  });
}

hipError_t launch_logprob_grad(LogitArgs a, int dtype, hipStream_t s) {
  const int64_t n = row_pieces(a, dtype);
  if (a.T && a.T < 256) {
    // rows shared by workgroups of 256 threads, four pieces a thread, two
    // workgroups a CU (1, 16 and 64 rows of 131072 bf16 logits 2.9, 3.5 and 6.6 us,
    // with 1024 threads a row 9.5, 10.1 and 11.8)
    const int64_t share = 512 / a.T, most = (n + 1023) / 1024;
    return grad_rows<256, 4, true>(a, dtype, s, (unsigned)(share < most ? share : most));
  }
  switch (grad_threads(n)) {
    case 64: return grad_rows<64, 2>(a, dtype, s);
    case 256: return grad_rows<256, 2>(a, dtype, s);
    case 512: return grad_rows<512, 4>(a, dtype, s);
    default: return grad_rows<1024, 4>(a, dtype, s);
  }
}

template <int W, int P>
static hipError_t policy_rows(LogitArgs& a, const PolicyArgs& p, int dtype, hipStream_t s) {
  return for_rows(a, [&](dim3 g) {
    if (dtype == 0)
      return a.stream ? launch(k_policy_regs<0, true, W, P>, g, W, s, a, p)
                      : launch(k_policy_regs<0, false, W, P>, g, W, s, a, p);
    return a.stream ? launch(k_policy_regs<1, true, W, P>, g, W, s, a, p)
                    : launch(k_policy_regs<1, false, W, P>, g, W, s, a, p);
  });
}

static hipError_t policy_long_rows(LogitArgs& a, const PolicyArgs& p, int dtype, hipStream_t s) {
  return for_rows(a, [&](dim3 g) {
    return dtype == 0 ? launch(k_policy_long<0, 1024, 4, 16>, g, 1024, s, a, p)
                      : launch(k_policy_long<1, 1024, 4, 16>, g, 1024, s, a, p);
  });
}

hipError_t launch_policy_logits(LogitArgs a, const PolicyArgs& p, int dtype,
                                hipStream_t s) {
  // threads and pieces a thread for rows of n pieces; more threads where there
  // are fewer rows than CUs (3276 x 32000 bf16 with 256 x 16 and 1024 x 4: 81
  // and 75 us; 15728 x 3000 with 64 x 8 and 256 x 4: 44 and 49, but 11520 x 2048
  // fp32 43 and 38)
  const int64_t n = row_pieces(a, dtype);
  const bool few = a.T < 256;
  hipError_t e;
  if (n <= 256 && !(few && n > 64)) e = policy_rows<64, 4>(a, p, dtype, s);
  else if (n <= 1024 && !(few && n > 256)) e = policy_rows<256, 4>(a, p, dtype, s);
  else if (n <= 2048 && !few) e = policy_rows<256, 8>(a, p, dtype, s);
  else if (n <= 4096) e = policy_rows<1024, 4>(a, p, dtype, s);
  else if (n <= 8192) e = policy_rows<512, 16>(a, p, dtype, s);
  else if (n <= 12288) e = policy_rows<1024, 12>(a, p, dtype, s);
  else if (n <= 16384) e = policy_rows<1024, 16>(a, p, dtype, s);
  else e = policy_long_rows(a, p, dtype, s);
  if (e != hipSuccess) return e;
  return launch(k_terms<3>, dim3(1), 1024, s, p.terms, p.T, 1.0, p.sums);
}

hipError_t launch_policy(const PolicyArgs& p, hipStream_t s) {
  const hipError_t e = p.T ? launch(k_policy, dim3(cdiv(p.T, 256)), 256, s, p) : hipSuccess;
  if (e != hipSuccess) return e;
  return launch(k_terms<3>, dim3(1), 1024, s, p.terms, p.T, 1.0, p.sums);
}

hipError_t launch_preference(PrefArgs p, hipStream_t s) {
  // one launch where a wave has one pair, and a short one in the mean (2 pairs
  // of 150 tokens: 4.8 us instead of 4.8 + 1.8 and a launch's gap; 32 pairs of
  // 256 tokens, ragged: 20 us instead of 6.8 + 4)
  if (p.P <= 16 && p.T <= 256 * p.P) return launch(k_preference_small, dim3(1), 1024, s, p);
  const hipError_t e =
      for_rows(p.pair0, p.P, [&](dim3 g) { return launch(k_preference, g, 1024, s, p); });
  if (e != hipSuccess) return e;
  return launch(k_terms<1>, dim3(1), 1024, s, p.terms, p.P, 1.0 / (double)p.P, p.loss);
}

}  // namespace hlq
