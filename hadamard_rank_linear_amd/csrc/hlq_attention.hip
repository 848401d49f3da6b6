// Attention over packed sequences, forward and backward, for head sizes up to
// HLQ_ATTN_D (built once per value).
//
// With S = scale q k^T + bias, P = exp(S - lse), delta_i = sum_d g_o o:
//   o = P v,   g_v = P^T g_o,   dS = P (g_o v^T - delta),
//   g_q = scale dS k,   g_k = scale dS^T q,   g_bias = sums of dS by bucket.
// Scores and statistics are fp32, in powers of two (c = scale log2 e).
//
// Every product is written so that its result's columns (a lane each) are what
// stays in a wave: a wave's 32 query rows in the forward pass and the gradient
// of q, its 32 keys in the gradients of k and v.  Then P and dS leave the matrix
// unit in the registers in which the next product takes them in, row statistics
// are one value a lane, and nothing but the other operand's tiles goes through LDS.
//
// Bound by the matrix unit for long sequences, by memory and the waits of a workgroup's
// start for short ones.  Measured in bf16, where a large product reaches 1138 TFLOP/s
// and a large copy 4.84 TB/s:
//  - forward, 8192 tokens, 32 heads of 128 on 8: 1180 us (930 TFLOP/s), causal 577 to 667
//    (952 to 824, with the inputs and the card's state); ViT-B (64 x 197 tokens, 12 heads of
//    64) 29 us for 78 MB; 8 tokens against 32700 keys 51 us with the join (2.6 TB/s);
//  - backward, 8192 ragged causal tokens, 32 heads of 128 on 8: 343 us for q (matrix units
//    busy 50% of the time), 552 for k and v (34%: one wave a SIMD, of whose cycles a
//    quarter go into its turns of the tiles' loads), under the profiler; ViT-B 48 + 59.
#include <algorithm>
#include <utility>

#include "hlq_attn.h"

#ifndef HLQ_ATTN_D
#error "HLQ_ATTN_D: the padded head size"
#endif

namespace hlq {
namespace {

constexpr float kInf = __builtin_inff();

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float max_halves(float v) {
  return lanes_stage<32>(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float sum_halves(float v) {
  return lanes_stage<32>(v, [](float a, float b) { return a + b; });
}

template <int DT, typename R>
__device__ __forceinline__ char* row_at(const R& t, int64_t token, int64_t head) {
  return static_cast<char*>(t.data) + (token * t.token + head * t.head) * (DT == 0 ? 4 : 2);
}

// Outputs of tokens that belong to no sequence: zeros.  A thread of `groups` workgroups
// has a 16-byte piece of every so many rows.
template <int DT>
__device__ void clear_tokens(const AttnRows& t, int64_t from, int64_t to, unsigned heads, int D,
                             unsigned group, unsigned groups) {
  constexpr int N = Piece<DT>::N;
  const unsigned pieces = (unsigned)(D + N - 1) / N, per = 256 / pieces;
  const unsigned piece = threadIdx.x % pieces, mine = threadIdx.x / pieces;
  if (mine >= per) return;
  const unsigned rows = (unsigned)(to - from) * heads;  // fewer than 2^30
  for (unsigned r = group * per + mine; r < rows; r += groups * per)
    store_piece<DT>(row_at<DT>(t, from + r / heads, r % heads), piece * N, D - (int)piece * N,
                    (u32x4){0u, 0u, 0u, 0u});
}
__device__ __forceinline__ int64_t bound(const int64_t* start, int64_t s, int64_t T) {
  const int64_t a = start[s];
  return a < 0 ? 0 : a > T ? T : a;
}

// What a wave knows of its 32 query rows: lane l has row l & 31.
struct RowInfo {
  bool valid;
  int token, head;  // in the sequence; query head
  int pos;          // position among the keys
  int limit;        // keys before it are visible
};
__device__ __forceinline__ RowInfo row_info(const AttnShape& g, int row, int rows, int head0,
                                            int off, int nk) {
  RowInfo r;
  r.valid = row < rows;
  r.token = row;
  r.head = head0;
  if (g.pack > 1) {
    r.token = (int)((unsigned)row / (unsigned)g.pack);
    r.head = head0 + row - r.token * g.pack;
  }
  r.pos = r.token + off;
  r.limit = nk;
  if (g.causal) r.limit = max(0, min(nk, r.pos + 1));
  return r;
}

__device__ __forceinline__ int wave_min(int v) {
  return lanes_join<64>(v, [](int a, int b) { return a < b ? a : b; });
}
__device__ __forceinline__ int wave_max_int(int v) {
  return lanes_join<64>(v, [](int a, int b) { return a > b ? a : b; });
}

// Scores of a 32 x 32 block plus their bias, in powers of two (s holds q k^T).  lo
// .. hi: the block's distances (key position - query position); base: the lane's
// of row 0, from which row r of the block is r up, or down where its rows are
// queries.
template <bool DOWN>
__device__ __forceinline__ void add_bias(const AttnShape& g, const float* line, f32x16& s, int lo,
                                         int hi, int base) {
  const int reach = g.bias.reach;
  if (lo >= reach || hi <= -reach) {
    const float b = line[lo >= reach ? 2 * (reach + BIAS_MARGIN) : 0];
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = __builtin_fmaf(s[r], g.c, b);
    return;
  }
  const float* at = line + base + reach + BIAS_MARGIN;
#pragma unroll
  for (int r = 0; r < 16; ++r)
    s[r] = __builtin_fmaf(s[r], g.c, DOWN ? at[-acc_row(r)] : at[acc_row(r)]);
}

// Address of the kernel's dynamic LDS.
__device__ __forceinline__ uint32_t lds_place(char* lds) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
}

typedef std::true_type Yes;
typedef std::false_type No;

// A chain of matrix products whose fragments come from LDS, in steps whose order the
// compiler keeps: fragment i + AHEAD is read, product i starts, and what the matrix
// unit does not need runs beside it.  Left alone the compiler reads a fragment, waits
// and multiplies: with one or two waves a SIMD the backward pass of 8192 ragged tokens
// took 1203 us, in this order 814.  Reading 8 or 12 products ahead gains nothing.
// read and use get the step's number as a constant.
constexpr int AHEAD = 4;
template <int I>
using Step = std::integral_constant<int, I>;
template <int DT, int N, typename Read, typename Use, int... I>
__device__ __forceinline__ void steps(std::integer_sequence<int, I...>, Read read, Use use) {
  Frag<DT> ring[AHEAD + 1];
  const auto one = [&](auto step) {
    constexpr int i = decltype(step)::value;
    if constexpr (i == 0) {
      ring[0] = read(Step<0>());
      if constexpr (N > 1 && AHEAD > 1) ring[1] = read(Step<1>());
      if constexpr (N > 2 && AHEAD > 2) ring[2] = read(Step<2>());
      if constexpr (N > 3 && AHEAD > 3) ring[3] = read(Step<3>());
    }
    if constexpr (i + AHEAD < N) ring[(i + AHEAD) % (AHEAD + 1)] = read(Step<i + AHEAD>());
    use(step, ring[i % (AHEAD + 1)]);
    __builtin_amdgcn_sched_barrier(0);
  };
  (one(Step<I>()), ...);
}
template <int DT, int N, typename Read, typename Use>
__device__ __forceinline__ void steps(Read read, Use use) {
  static_assert(AHEAD <= 4, "the first reads are written out");
  steps<DT, N>(std::make_integer_sequence<int, N>(), read, use);
}
// Of `all` pieces of work beside steps 1 .. n - 1 (the step before has the results
// they need still under way), the first that belongs to step i.
__device__ __forceinline__ constexpr int beside(int i, int n, int all) {
  return i <= 0 ? 0 : i >= n ? all : all * (i - 1) / (n - 1);
}

// ------------------------------------------------------------ forward

// A work item is a tile of query rows of one sequence and head group: 32 rows a wave
// and every key, or, FEW, 32 rows in all and a share of the keys, of which each wave
// takes a quarter, joined through LDS at the end.
template <int DT, int DP, bool FEW>
struct FwdShape {
  typedef Tile<DT, DP> T;
  static constexpr int ROWS = FEW ? ATTN_FEW : ATTN_ROWS;
  static constexpr int KEYS = FEW ? 128 : DT == 0 ? 32 : 64;  // of a tile
  static constexpr int MINE = FEW ? 32 : KEYS;                // of them a wave's
  static constexpr int TILE_BYTES = KEYS * T::ROW_BYTES;
  static constexpr int JOIN_BYTES = FEW ? 4 * DP * 33 * 4 + 4 * 32 * 8 : 0;
  // buffers of a tile of keys and of values: one where two leave no room for a second
  // workgroup, which then loads while this one computes (1 token against 65536 keys, with
  // equal shares, 96 -> 67 us)
  static constexpr int BUFS = TILE_BYTES > 16384 ? 1 : 2;
  static constexpr int LDS =
      2 * BUFS * TILE_BYTES > JOIN_BYTES ? 2 * BUFS * TILE_BYTES : JOIN_BYTES;
};

// Workgroups a CU: three of heads up to 64 (ViT-B 36 -> 31 us; a fourth costs spills),
// one in fp32, whose fragments are twice as large.
template <int DT, int DP, bool BIAS, bool FEW, bool VEC>
__global__ __launch_bounds__(256, DT == 0 ? 1 : DP <= 64 && !FEW ? 3 : 2) void k_attention_forward(AttnFwd a) {
  typedef FwdShape<DT, DP, FEW> F;
  typedef Tile<DT, DP> T;
  constexpr int DB = DP / 32, DC = DP / 16, SB = F::MINE / 32, ES = DT == 0 ? 4 : 2;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int16_t* const first_of = reinterpret_cast<int16_t*>(lds + F::LDS);
  float* const line = reinterpret_cast<float*>(first_of + BIAS_FIRST);
  const uint32_t row_lane = lds_place(lds) + T::row_lane(), col_lane = lds_place(lds) + T::col_lane();
  const AttnShape& g = a.g;
  const int lane = threadIdx.x & 63, half = lane >> 5, wave = threadIdx.x >> 6;

  if (blockIdx.x >= g.launched) {  // tokens of no sequence
    const unsigned group = blockIdx.x - g.launched, groups = gridDim.x - g.launched;
    const int64_t from = bound(g.start_q, 0, g.Tq), to = bound(g.start_q, g.S, g.Tq);
    for (int part = 0; part < 2; ++part) {
      const int64_t x = part ? max(from, to) : 0, y = part ? g.Tq : from;
      const unsigned tokens = (unsigned)(y - x), rows = tokens * g.heads;
      if (FEW && a.po) {
        for (unsigned p = 0; p < g.splits; ++p)
          for (unsigned i = group * 256 + threadIdx.x; i < rows; i += groups * 256) {
            float* ml = a.ml + ((p * g.Tq + x) * g.heads + i) * 2;
            ml[0] = -kInf;
            ml[1] = 0.f;
          }
        continue;
      }
      clear_tokens<DT>(a.o, x, y, g.heads, g.D, group, groups);
      for (unsigned i = group * 256 + threadIdx.x; i < rows; i += groups * 256)
        a.lse[(int64_t)(i / tokens) * g.Tq + x + i % tokens] = -kInf;
    }
    return;
  }

  for (unsigned item = blockIdx.x; item < g.items; item += g.launched) {
    unsigned u, t;
    if (!item_of(g, item, u, t)) continue;
    const int split = FEW ? (int)(t % g.splits) : 0;
    const unsigned tile0 = g.tiles - 1 - (FEW ? t / g.splits : t);  // the longest first
    const unsigned per = g.kv_heads * g.groups;
    const int64_t seq = u / per;
    const int unit = (int)(u % per), head0 = unit * g.pack, kvh = unit / g.groups;
    int q0, nq, k0, nk;
    sequence(g.start_q, seq, g.Tq, q0, nq);
    sequence(g.start_k, seq, g.Tk, k0, nk);
    const int rows = nq * g.pack, off = nk - nq;
    if ((int64_t)tile0 * F::ROWS >= rows) continue;
    if constexpr (BIAS) {
      __syncthreads();
      load_bias_first(g.bias, first_of);
      load_bias_line(g.bias, first_of, head0, g.heads, line);
    }
    const char* const kb = row_at<DT>(a.k, k0, kvh);
    const char* const vb = row_at<DT>(a.v, k0, kvh);
    const int64_t kt = a.k.token * ES, vt = a.v.token * ES;
    Feed<DT, DP, F::KEYS, VEC> sk, sv;
    sk.init((uint32_t)kt, 0, 1);
    sv.init((uint32_t)vt, 0, 1);

    for (int64_t tile = tile0; tile * F::ROWS < rows; tile += g.tiles) {
      const int row0 = (int)tile * F::ROWS + (FEW ? 0 : wave * 32);
      const RowInfo me = row_info(g, row0 + (lane & 31), rows, head0, off, nk);
      // keys of the tile's last row: every wave of the group goes that far
      int end = nk;
      if (g.causal) {
        const int r = min(rows, (int)(tile + 1) * F::ROWS) - 1;
        end = max(0, min(nk, (int)((unsigned)r / (unsigned)g.pack) + off + 1));
      }
      // where it is known to be zero the compiler runs out of scalar registers (ViT-B 28.0
      // -> 29.3 us)
      int from = 0;
      if (!FEW) asm volatile("" : "+s"(from));
      if (FEW && g.splits > 1) {
        const int share =
            max(g.share, (int)(((end + F::KEYS - 1) / F::KEYS + g.splits - 1) / g.splits) * F::KEYS);
        from = (int)min((int64_t)end, (int64_t)split * share);
        end = min(end, from + share);
      }
      const int limit = min(me.limit, end);
      const int first = wave_min(me.valid ? limit : end);     // keys that all rows see
      const int last = wave_max_int(me.valid ? limit : from);  // and that any does

      Frag<DT> qf[DC];
      {
        const char* p = row_at<DT>(a.q, q0 + (me.valid ? me.token : 0), me.head);
#pragma unroll
        for (int c = 0; c < DC; ++c)
          qf[c] = me.valid ? global_frag<DT, VEC>(p, 16 * c + 8 * half, g.D) : zero_frag<DT>();
      }
      f32x16 o[DB];
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] = (f32x16)(0.f);
      float m = -kInf, l = 0.f;

      // One tile of keys, from key0 on in this wave.
      // COUNT blocks of 32 keys from key0 on; rl, cl: the lane's place in the keys'
      // tile, by rows and by columns, the values' follow.  MASK: some rows do not see
      // some of the keys; bad: those of them whose values are not finite.
      const auto blocks = [&](auto count, auto mask, int key0, uint32_t rl, uint32_t cl,
                              uint32_t bad) {
        constexpr int COUNT = decltype(count)::value, ND = 2 * DB, PV = COUNT * DC;
        constexpr bool MASK = decltype(mask)::value;
        // fragments in the order of use: rows of k by blocks, columns of v by blocks
        const auto read = [&](auto step) {
          constexpr int i = decltype(step)::value;
          if constexpr (i < PV) {
            return T::row_frag(rl, 32 * (i / DC), i % DC);
          } else {
            constexpr int j = i - PV;
            return T::col_frag(cl, F::KEYS + 32 * (j / ND) + 16 * (j % ND / DB), j % DB);
          }
        };
        Frag<DT> pf[2];
        f32x16 s[COUNT];
        float base = 0.f, keep = 1.f, sum = 0.f;
        bool moved = false;  // the maximum; uniform
        // A block's scores are there: bias, mask, the running maximum, and the factor
        // that the sums so far then need.
        const auto enter = [&](int b) {
          if constexpr (MASK) {
#pragma unroll
            for (int r = 0; r < 16; ++r)
              if (key0 + 32 * b + acc_row(r) + 4 * half >= limit) s[b][r] = -kInf;
          }
          float top = s[b][0];
#pragma unroll
          for (int r = 1; r < 16; ++r) top = fmaxf(top, s[b][r]);
          top = max_halves(top);
          if constexpr (!BIAS) top *= g.c;
          top = fmaxf(m, top);
          base = top == -kInf ? 0.f : top;  // a row that has seen no key yet
          moved = __any(top != m);
          if (moved) {
            keep = exp2_fast(m - base);
            l *= keep;
            m = top;
          }
        };
        const auto rescale = [&] {
          if (!moved) return;
#pragma unroll
          for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[d][r] *= keep;
        };
        const auto probability = [&](int b, int r) {
          s[b][r] = exp2_fast(BIAS ? s[b][r] - base : __builtin_fmaf(s[b][r], g.c, -base));
          sum += s[b][r];
        };
        const auto leave = [&](int b) {
          if (MASK && (bad & bit_range(0, limit - key0 - 32 * b))) sum = __builtin_nanf("");
          l += sum;
          sum = 0.f;
          pf[0] = acc_frag<DT>(s[b], 0);
          pf[1] = acc_frag<DT>(s[b], 1);
        };
        steps<DT, PV + COUNT * ND>(read, [&](auto step, const Frag<DT>& f) {
          constexpr int i = decltype(step)::value;
          if constexpr (i < PV) {
            constexpr int b = i / DC, j = i % DC;
            if constexpr (j == 0) s[b] = (f32x16)(0.f);
            s[b] = mma(f, qf[j], s[b]);
            if constexpr (BIAS && j == DC - 1) {
              const int dist = key0 + 32 * b - (row0 + off);  // of the first row; later ones less
              add_bias<false>(g, line, s[b], dist - 31, dist + 31, key0 + 32 * b - me.pos + 4 * half);
            }
            if constexpr (COUNT == 1 && j == DC - 1) {
              enter(0);
              rescale();
#pragma unroll
              for (int r = 0; r < 16; ++r) probability(0, r);
              leave(0);
            }
            if constexpr (b > 0) {
              // beside the second block's scores: the first one's probabilities
              if constexpr (j == 1) {
                enter(0);
                rescale();
              }
#pragma unroll
              for (int r = beside(j, DC, 16); r < beside(j + 1, DC, 16); ++r) probability(0, r);
              if constexpr (j == DC - 1) leave(0);
            }
          } else {
            constexpr int b = (i - PV) / ND, j = (i - PV) % ND;
            o[j % DB] = mma(only_finite<DT>(f, MASK && bad), pf[j / DB], o[j % DB]);
            if constexpr (b + 1 < COUNT) {
              // beside the first block's values: the second one's probabilities
              if constexpr (j == 1) enter(1);
#pragma unroll
              for (int r = beside(j, ND, 16); r < beside(j + 1, ND, 16); ++r) probability(1, r);
              if constexpr (j == ND - 1) {
                rescale();
                leave(1);
              }
            }
          }
        });
      };
      // A tile of keys, of which this wave's begin at key0 and in LDS at `tile`.
      const auto attend = [&](int key0, int tile) {
        uint32_t rl = row_lane + tile, cl = col_lane + tile;
        if (key0 + F::MINE <= first) {
          blocks(Step<SB>(), No(), key0, rl, cl, 0);
          return;
        }
#pragma unroll 1
        for (int b = 0; b < SB && key0 < last; ++b, key0 += 32) {
          blocks(Step<1>(), Yes(), key0, rl, cl,
                 g.causal ? rows_not_finite<DT, DP>(rl, F::KEYS) : 0);
          rl += 32 * T::ROW_BYTES;
          cl += 32 * T::ROW_BYTES;
        }
      };

      const auto feed = [&](int key, int buf) {
        const uint32_t at = lds_place(lds) + buf * 2 * F::TILE_BYTES;
        sk.issue(kb + key * kt, end - key, g.D, at);
        sv.issue(vb + key * vt, end - key, g.D, at + F::TILE_BYTES);
      };
      __syncthreads();  // the previous tile's reads are done
      if (F::BUFS == 2 && from < end) feed(from, 0);
      int buf = 0;
      for (int key = from; key < end; key += F::KEYS, buf ^= F::BUFS - 1) {
        if (F::BUFS == 1) {
          __syncthreads();
          feed(key, 0);
        }
        feed_wait();
        if (F::BUFS == 2 && key + F::KEYS < end) feed(key + F::KEYS, buf ^ 1);
        const int mine = FEW ? 32 * wave : 0, key0 = key + mine;
        if (key0 >= last) continue;
        const int at = buf * 2 * F::TILE_BYTES + mine * T::ROW_BYTES;
        attend(key0, at);
      }
      l = sum_halves(l);

      const auto& z = *again<AttnFwd>();
      if constexpr (!FEW) {
        if (!me.valid) continue;
        const int64_t token = (int64_t)q0 + me.token;
        if (half == 0)
          z.lse[me.head * z.g.Tq + token] =
              l == 0.f ? -kInf : (m + __builtin_amdgcn_logf(l)) * kLn2;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        char* p = row_at<DT>(z.o, token, me.head);
        const int D = z.g.D;
        const bool vec = z.o.vec;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int r = 0; r < 16; r += 4)
            store4<DT>(p, 32 * d + acc_row(r) + 4 * half, D, vec, o[d][r] * inv, o[d][r + 1] * inv,
                       o[d][r + 2] * inv, o[d][r + 3] * inv);
      } else {
        // the waves' shares of the keys: [wave][d][row], rows 33 apart
        float* const jo = reinterpret_cast<float*>(lds);
        float2* const jm = reinterpret_cast<float2*>(lds + 4 * DP * 33 * 4);
        __syncthreads();
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            jo[(wave * DP + 32 * d + acc_row(r) + 4 * half) * 33 + (lane & 31)] = o[d][r];
        if (half == 0) jm[wave * 32 + lane] = make_float2(m, l);
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * DP; i += 256) {
          const int r = i / DP, d = i % DP;
          const RowInfo it = row_info(g, (int)tile * F::ROWS + r, rows, head0, off, nk);
          if (!it.valid || d >= z.g.D) continue;
          float top = -kInf, total = 0.f, v = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) top = fmaxf(top, jm[w * 32 + r].x);
          const float base = top == -kInf ? 0.f : top;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float f = exp2_fast(jm[w * 32 + r].x - base);
            total += f * jm[w * 32 + r].y;
            v += f * jo[(w * DP + d) * 33 + r];
          }
          const int64_t token = (int64_t)q0 + it.token;
          if (z.po) {
            const int64_t at = ((int64_t)split * z.g.Tq + token) * z.g.heads + it.head;
            z.po[at * z.g.D + d] = v;
            if (d == 0) {
              z.ml[2 * at] = top;
              z.ml[2 * at + 1] = total;
            }
            continue;
          }
          if (d == 0)
            z.lse[it.head * z.g.Tq + token] =
                total == 0.f ? -kInf : (top + __builtin_amdgcn_logf(total)) * kLn2;
          const float y = total == 0.f ? 0.f : v / total;
          char* p = row_at<DT>(z.o, token, it.head);
          if constexpr (DT == 0) reinterpret_cast<float*>(p)[d] = y;
          else reinterpret_cast<uint16_t*>(p)[d] = (uint16_t)pack_bf16(y, 0.f);
        }
        __syncthreads();
      }
    }
  }
}

// ------------------------------------------------------------ gradient of q

// FEW: a tile of 32 rows (keys), of which each wave takes a quarter of the keys
// (rows); the waves' sums are joined through LDS.
template <int DT, int DP, bool FEW, bool SKEWED = false>
struct BwdShape {
  typedef Tile<DT, DP> T;
  static constexpr int OWN = FEW ? ATTN_FEW : ATTN_ROWS;      // rows (keys) of a workgroup
  static constexpr int KEYS = FEW ? 128 : DT == 0 ? 32 : 64;  // keys, or rows, of a tile
  static constexpr int BLOCKS = FEW ? 1 : KEYS / 32;          // of them a wave's
  static constexpr int TILE_BYTES = KEYS * T::ROW_BYTES;
  // SKEWED: the sums of a bias's gradient need room too
  static constexpr int BUFS = TILE_BYTES > (SKEWED ? 16384 : 32768) ? 1 : 2;
  static constexpr int JOIN_BYTES = FEW ? 4 * DP * 33 * 4 : 0;
  static constexpr int LDS =
      2 * BUFS * TILE_BYTES > JOIN_BYTES ? 2 * BUFS * TILE_BYTES : JOIN_BYTES;
};

// Sums of the four waves, each [d][lane] in `mine` (plus poison, 0 or NaN), times scale
// into the lanes' rows: row(i) is the address of lane i's output or null.  All
// threads; LDS is free before and after.
template <int DT, int DP, typename Row>
__device__ __forceinline__ void join_waves(char* lds, const f32x16 (&mine)[DP / 32], float poison,
                                           float scale, int D, Row row) {
  typedef typename Piece<DT>::Elem E;
  float* const sums = reinterpret_cast<float*>(lds);
  const int lane = threadIdx.x & 63, half = lane >> 5, wave = threadIdx.x >> 6;
  __syncthreads();
#pragma unroll
  for (int d = 0; d < DP / 32; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      sums[(wave * DP + 32 * d + acc_row(r) + 4 * half) * 33 + (lane & 31)] =
          mine[d][r] + poison;
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * DP; i += 256) {
    const int d = i % DP, at = d * 33 + i / DP;
    char* const p = row(i / DP);
    if (!p || d >= D) continue;
    const float v = ((sums[at] + sums[DP * 33 + at]) +
                     (sums[2 * DP * 33 + at] + sums[3 * DP * 33 + at])) * scale;
    if constexpr (DT == 0) reinterpret_cast<E*>(p)[d] = v;
    else reinterpret_cast<E*>(p)[d] = (uint16_t)pack_bf16(v, 0.f);
  }
  __syncthreads();
}

// Waves as in the forward pass.  Writes delta for the gradients of k and v, and
// with a bias the sums of dS by bucket over the item: each wave adds its blocks'
// diagonals to a line of distances of its own in LDS, blocks beyond reach in
// registers (8190 ragged tokens, 12 heads of 64: 100 us).  Three workgroups a CU of
// heads up to 64 as above (ViT-B 48 -> 44 us, at 44 bytes of scratch a lane), two where the
// line takes registers too.
template <int DT, int DP, bool BIAS, bool FEW, bool VEC>
__global__ __launch_bounds__(256, DT == 0 ? 1 : DP <= 64 && !BIAS && !FEW ? 3 : 2) void k_attention_backward_q(AttnBwd a) {
  typedef BwdShape<DT, DP, FEW, BIAS> F;
  typedef Tile<DT, DP> T;
  constexpr int DB = DP / 32, DC = DP / 16, ES = DT == 0 ? 4 : 2;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const uint32_t row_lane = lds_place(lds) + T::row_lane(), col_lane = lds_place(lds) + T::col_lane();
  const AttnShape& g = a.g;
  const int lines = BIAS ? bias_line_size(g.bias) : 0;
  int16_t* const first_of = reinterpret_cast<int16_t*>(lds + F::LDS);
  float* const skew = reinterpret_cast<float*>(first_of + BIAS_FIRST);  // [4][SKEW_SIZE]
  float* const far = skew + (BIAS ? 4 * SKEW_SIZE : 0);                 // [4][2]
  float* const sums = far + 8;                                          // [4][lines]
  float* const line = sums + 4 * lines;
  const int lane = threadIdx.x & 63, half = lane >> 5, wave = threadIdx.x >> 6;

  if (blockIdx.x >= g.launched) {
    const unsigned group = blockIdx.x - g.launched, groups = gridDim.x - g.launched;
    const int64_t from = bound(g.start_q, 0, g.Tq), to = bound(g.start_q, g.S, g.Tq);
    clear_tokens<DT>(a.g_q, 0, from, g.heads, g.D, group, groups);
    clear_tokens<DT>(a.g_q, max(from, to), g.Tq, g.heads, g.D, group, groups);
    return;
  }

  for (unsigned item = blockIdx.x; item < g.items; item += g.launched) {
    unsigned u, t;
    if (!item_of(g, item, u, t)) continue;
    const unsigned tile0 = g.tiles - 1 - t, per = g.kv_heads * g.groups;
    const int64_t seq = u / per;
    const int unit = (int)(u % per), head0 = unit * g.pack, kvh = unit / g.groups;
    float* const bucket_sums = a.g_line + ((int64_t)u * g.tiles + tile0) * g.bias.buckets;
    int q0, nq, k0, nk;
    sequence(g.start_q, seq, g.Tq, q0, nq);
    sequence(g.start_k, seq, g.Tk, k0, nk);
    const int rows = nq * g.pack, off = nk - nq;
    if ((int64_t)tile0 * F::OWN >= rows) {
      if constexpr (BIAS)
        for (int b = threadIdx.x; b < g.bias.buckets; b += 256)
          bucket_sums[b] = 0.f;
      continue;
    }
    float far_low = 0.f, far_high = 0.f;
    if constexpr (BIAS) {
      __syncthreads();
      load_bias_first(g.bias, first_of);
      load_bias_line(g.bias, first_of, head0, g.heads, line);
      for (int i = threadIdx.x; i < 4 * lines; i += 256) sums[i] = 0.f;
      for (int i = threadIdx.x; i < 4 * SKEW_SIZE; i += 256) skew[i] = 0.f;
    }
    const char* const kb = row_at<DT>(a.k, k0, kvh);
    const char* const vb = row_at<DT>(a.v, k0, kvh);
    const int64_t kt = a.k.token * ES, vt = a.v.token * ES;
    Feed<DT, DP, F::KEYS, VEC> sk, sv;
    sk.init((uint32_t)kt, 0, 1);
    sv.init((uint32_t)vt, 0, 1);

    for (int64_t tile = tile0; tile * F::OWN < rows; tile += g.tiles) {
      const int row0 = (int)tile * F::OWN + (FEW ? 0 : wave * 32);
      RowInfo me = row_info(g, row0 + (lane & 31), rows, head0, off, nk);
      // Rows past the end are computed for nothing, but not for the bias's gradient.
      if (BIAS && !me.valid) me.limit = 0;
      const int first = wave_min(BIAS || me.valid ? me.limit : nk);
      const int last = wave_max_int(me.valid ? me.limit : 0);
      int end = nk;
      if (g.causal) {
        const int r = min(rows, (int)(tile + 1) * F::OWN) - 1;
        end = max(0, min(nk, (int)((unsigned)r / (unsigned)g.pack) + off + 1));
      }

      const auto feed = [&](int key, int buf) {
        const uint32_t at = lds_place(lds) + buf * 2 * F::TILE_BYTES;
        sk.issue(kb + key * kt, end - key, g.D, at);
        sv.issue(vb + key * vt, end - key, g.D, at + F::TILE_BYTES);
      };
      __syncthreads();  // the previous tile's reads are done
      if (F::BUFS == 2 && end > 0) feed(0, 0);

      Frag<DT> qf[DC], gf[DC];
      float lse = kInf, delta = 0.f;
      const int64_t token = (int64_t)q0 + (me.valid ? me.token : 0);
      {
        const auto& z = *again<AttnBwd>();
        const char* pq = row_at<DT>(z.q, token, me.head);
        const char* pg = row_at<DT>(z.g_o, token, me.head);
        const char* po = row_at<DT>(z.o, token, me.head);
        const int D = z.g.D;
#pragma unroll
        for (int c = 0; c < DC; ++c) {
          qf[c] = gf[c] = zero_frag<DT>();
          if (me.valid) {
            const int d = 16 * c + 8 * half;
            qf[c] = global_frag<DT, VEC>(pq, d, D);
            gf[c] = global_frag<DT, VEC>(pg, d, D);
            const Frag<DT> of = global_frag<DT, VEC>(po, d, D);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              delta = __builtin_fmaf((float)gf[c][e], (float)of[e], delta);
          }
        }
        delta = sum_halves(delta);
        if (me.valid) {
          if (half == 0) z.delta[me.head * z.g.Tq + token] = delta;
          lse = z.lse[me.head * z.g.Tq + token] * kLog2e;
          if (lse == -kInf) lse = kInf;  // no key seen: probabilities of zero
        }
      }
      f32x16 dq[DB];
#pragma unroll
      for (int d = 0; d < DB; ++d) dq[d] = (f32x16)(0.f);
      float poison = 0.f;

      // A block of 32 keys from key on; see the forward pass.
      const auto block = [&](auto mask, int key, uint32_t rl, uint32_t cl, uint32_t bad) {
        constexpr bool MASK = decltype(mask)::value;
        const int dist = key - (row0 + off), limit = me.limit - key;
        // fragments in the order of use: rows of k, rows of v, columns of k
        const auto read = [&](auto step) {
          constexpr int i = decltype(step)::value;
          if constexpr (i < 2 * DC) return T::row_frag(rl, i < DC ? 0 : F::KEYS, i % DC);
          else return T::col_frag(cl, 16 * ((i - 2 * DC) / DB), (i - 2 * DC) % DB);
        };
        Frag<DT> df[2], rest[2];
        f32x16 s = (f32x16)(0.f), dp = (f32x16)(0.f);
        steps<DT, 2 * DC + 2 * DB>(read, [&](auto step, const Frag<DT>& f) {
          constexpr int i = decltype(step)::value;
          if constexpr (i < DC) {
            s = mma(f, qf[i], s);
            if constexpr (BIAS && i == DC - 1)
              add_bias<false>(g, line, s, dist - 31, dist + 31, key - me.pos + 4 * half);
          } else if constexpr (i < 2 * DC) {
            dp = mma(f, gf[i - DC], dp);
            constexpr int j = i - DC;
#pragma unroll
            for (int r = beside(j, DC, 16); r < beside(j + 1, DC, 16); ++r)
              s[r] = exp2_fast(BIAS ? s[r] - lse : __builtin_fmaf(s[r], g.c, -lse));
            if constexpr (j == DC - 1) {
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                s[r] *= dp[r] - delta;
                if (MASK && acc_row(r) + 4 * half >= limit) s[r] = 0.f;
              }
              if constexpr (BIAS) {  // its gradient
                if (dist - 31 >= g.bias.reach || dist + 31 <= -g.bias.reach) {
                  float sum = 0.f;
#pragma unroll
                  for (int r = 0; r < 16; ++r) sum += s[r];
                  if (dist > 0) far_high += sum;
                  else far_low += sum;
                } else {
                  const float sum = diagonal_sum(skew + wave * SKEW_SIZE, s);
                  // lane i: distance i - 31 from the block's first row and column
                  if (lane < 63)
                    sums[wave * lines + dist - 31 + lane + g.bias.reach + BIAS_MARGIN] += sum;
                }
              }
              if (MASK && (bad & bit_range(0, limit))) poison = __builtin_nanf("");
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                df[c] = acc_frag<DT>(s, c);
                if constexpr (DT == 1) rest[c] = acc_rest(s, c, df[c]);
              }
            }
          } else {
            constexpr int j = i - 2 * DC;
            const Frag<DT> k = only_finite<DT>(f, MASK && bad);
            dq[j % DB] = mma(k, df[j / DB], dq[j % DB]);
            if constexpr (DT == 1) dq[j % DB] = mma(k, rest[j / DB], dq[j % DB]);
          }
        });
      };
      // A tile of keys, of which this wave's begin at key and in LDS at `tile`.
      const auto attend = [&](int key, int tile) {
        uint32_t rl = row_lane + tile, cl = col_lane + tile;
#pragma unroll 1
        for (int b = 0; b < F::BLOCKS && key < last; ++b, key += 32) {
          if (key + 32 <= first) block(No(), key, rl, cl, 0);
          else block(Yes(), key, rl, cl, g.causal ? rows_not_finite<DT, DP>(rl, 0) : 0);
          rl += 32 * T::ROW_BYTES;
          cl += 32 * T::ROW_BYTES;
        }
      };
      int buf = 0;
      for (int key = 0; key < end; key += F::KEYS, buf ^= F::BUFS - 1) {
        if (F::BUFS == 1) {
          __syncthreads();
          feed(key, 0);
        }
        feed_wait();
        if (F::BUFS == 2 && key + F::KEYS < end) feed(key + F::KEYS, buf ^ 1);
        const int mine = FEW ? 32 * wave : 0;
        attend(key + mine, buf * 2 * F::TILE_BYTES + mine * T::ROW_BYTES);
      }
      if constexpr (FEW) {
        const auto& z = *again<AttnBwd>();
        join_waves<DT, DP>(lds, dq, poison, z.g.scale, z.g.D, [&](int i) -> char* {
          const RowInfo it = row_info(g, row0 + i, rows, head0, off, nk);
          return it.valid ? row_at<DT>(z.g_q, (int64_t)q0 + it.token, it.head) : nullptr;
        });
        continue;
      }
      if (me.valid) {
        const auto& z = *again<AttnBwd>();
        char* p = row_at<DT>(z.g_q, token, me.head);
        const int D = z.g.D;
        const bool vec = z.g_q.vec;
        const float scale = z.g.scale + poison;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int r = 0; r < 16; r += 4)
            store4<DT>(p, 32 * d + acc_row(r) + 4 * half, D, vec, dq[d][r] * scale,
                       dq[d][r + 1] * scale, dq[d][r + 2] * scale, dq[d][r + 3] * scale);
      }
    }

    if constexpr (BIAS) {
      far_low = lanes_sum<64>(far_low);
      far_high = lanes_sum<64>(far_high);
      if (lane == 0) {
        far[2 * wave] = far_low;
        far[2 * wave + 1] = far_high;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < lines; i += 256)
        line[i] = (sums[i] + sums[lines + i]) + (sums[2 * lines + i] + sums[3 * lines + i]);
      __syncthreads();
      const int end = g.bias.reach + BIAS_MARGIN;
      for (int b = threadIdx.x; b < g.bias.buckets; b += 256) {
        int from, to;
        bucket_range(g.bias, first_of, b, from, to);
        float v = 0.f;
        for (int i = from; i <= to; ++i) v += line[i + end];
        for (int w = 0; w < 4; ++w) {
          if (from <= -end && -end <= to) v += far[2 * w];
          if (from <= end && end <= to) v += far[2 * w + 1];
        }
        bucket_sums[b] = v;
      }
    }
  }
}

// ------------------------------------------------------------ gradients of k and v

// A work item is 128 keys of one sequence and key head, 32 a wave (FEW: 32 keys, a
// quarter of the rows a wave); it goes through the query rows of the heads that share
// them.  Both gradients of 32 keys, keys and values stay in registers: 64 keys a wave
// spill (ViT-B 59 -> 90 us), and heads of 128 leave room for one wave a SIMD.  The
// probabilities are computed once more than in one kernel for all three gradients,
// which would have to add up g_q over workgroups: with atomics, in any order.
template <int DT, int DP, bool BIAS, bool FEW, bool VEC>
__global__ __launch_bounds__(256, DT == 1 && DP <= 64 ? 2 : 1) void k_attention_backward_kv(
    AttnBwd a) {
  typedef BwdShape<DT, DP, FEW> F;
  typedef Tile<DT, DP> T;
  constexpr int DB = DP / 32, DC = DP / 16, ES = DT == 0 ? 4 : 2;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  float* const stats = reinterpret_cast<float*>(lds + F::LDS);  // lse, delta of the rows, twice
  int16_t* const first_of = reinterpret_cast<int16_t*>(stats + 4 * F::KEYS);
  float* const line = reinterpret_cast<float*>(first_of + BIAS_FIRST);
  const uint32_t row_lane = lds_place(lds) + T::row_lane(), col_lane = lds_place(lds) + T::col_lane();
  const AttnShape& g = a.g;
  const int lane = threadIdx.x & 63, half = lane >> 5, wave = threadIdx.x >> 6;

  if (blockIdx.x >= g.launched) {
    const unsigned group = blockIdx.x - g.launched, groups = gridDim.x - g.launched;
    const int64_t from = bound(g.start_k, 0, g.Tk), to = bound(g.start_k, g.S, g.Tk);
    for (int part = 0; part < 2; ++part) {
      const int64_t x = part ? max(from, to) : 0, y = part ? g.Tk : from;
      clear_tokens<DT>(a.g_k, x, y, g.kv_heads, g.D, group, groups);
      clear_tokens<DT>(a.g_v, x, y, g.kv_heads, g.D, group, groups);
    }
    return;
  }

  for (unsigned item = blockIdx.x; item < g.items; item += g.launched) {
    unsigned u, tile0;  // first keys are seen by most rows
    if (!item_of(g, item, u, tile0)) continue;
    const int64_t seq = u / (unsigned)g.kv_heads;
    const int kvh = (int)(u % (unsigned)g.kv_heads);
    int q0, nq, k0, nk;
    sequence(g.start_q, seq, g.Tq, q0, nq);
    sequence(g.start_k, seq, g.Tk, k0, nk);
    const int rows = nq * g.pack, off = nk - nq;
    if ((int64_t)tile0 * F::OWN >= nk) continue;
    const int64_t qt = a.q.token * ES, gt = a.g_o.token * ES;
    Feed<DT, DP, F::KEYS, VEC> sq, sg;
    sq.init((uint32_t)qt, (uint32_t)(a.q.head * ES), g.pack);
    sg.init((uint32_t)gt, (uint32_t)(a.g_o.head * ES), g.pack);

    for (int64_t tile = tile0; tile * F::OWN < nk; tile += g.tiles) {
      const int wkey = (int)tile * F::OWN + (FEW ? 0 : wave * 32), key = wkey + (lane & 31);
      const bool valid = key < nk;
      Frag<DT> kf[DC], vf[DC];
      {
        const auto& z = *again<AttnBwd>();
        const int64_t token = (int64_t)k0 + (valid ? key : 0);
        const char* pk = row_at<DT>(z.k, token, kvh);
        const char* pv = row_at<DT>(z.v, token, kvh);
        const int D = z.g.D;
#pragma unroll
        for (int c = 0; c < DC; ++c) {
          const int d = 16 * c + 8 * half;
          kf[c] = valid ? global_frag<DT, VEC>(pk, d, D) : zero_frag<DT>();
          vf[c] = valid ? global_frag<DT, VEC>(pv, d, D) : zero_frag<DT>();
        }
      }
      f32x16 dk[DB], dv[DB];
#pragma unroll
      for (int d = 0; d < DB; ++d) dk[d] = dv[d] = (f32x16)(0.f);
      float poison_k = 0.f, poison_v = 0.f;
      // first row that sees the tile's first key, in whole tiles; this wave's first key
      int begin = 0, mine = 0;
      if (g.causal) {
        begin = max(0, (int)tile * F::OWN - off) * g.pack / F::KEYS * F::KEYS;
        mine = max(0, wkey - off) * g.pack;
      }
      const int sees = g.causal ? max(0, key - off) * g.pack : 0;       // first row of this key
      const int most = g.causal ? max(0, wkey + 31 - off) * g.pack : 0;  // of the wave's last

      // A block of 32 rows from row on; stat: their lse, and delta after a tile's.
      const auto block = [&](auto mask, int row, uint32_t rl, uint32_t cl, const float* stat,
                             uint32_t bad_q, uint32_t bad_g) {
        constexpr bool MASK = decltype(mask)::value;
        constexpr int ND = 2 * DB;
        const int low = sees - row, high = rows - row;
        // fragments in the order of use: rows of q, rows of g_o, columns of g_o, of q
        const auto read = [&](auto step) {
          constexpr int i = decltype(step)::value;
          if constexpr (i < 2 * DC) {
            return T::row_frag(rl, i < DC ? 0 : F::KEYS, i % DC);
          } else {
            constexpr int j = (i - 2 * DC) % ND;
            return T::col_frag(cl, (i < 2 * DC + ND ? F::KEYS : 0) + 16 * (j / DB), j % DB);
          }
        };
        Frag<DT> pf[2], df[2];
        f32x16 s = (f32x16)(0.f), dp = (f32x16)(0.f);
        f32x4 lse[4], del[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float* p = stat + 8 * q + 4 * half;
          lse[q] = *reinterpret_cast<const f32x4*>(p);
          del[q] = *reinterpret_cast<const f32x4*>(p + F::KEYS);
        }
        const auto hidden = [&](int r) {
          const int i = acc_row(r) + 4 * half;
          return MASK && (i < low || i >= high);
        };
        steps<DT, 2 * (DC + ND)>(read, [&](auto step, const Frag<DT>& f) {
          constexpr int i = decltype(step)::value;
          if constexpr (i < DC) {
            s = mma(f, kf[i], s);
            if constexpr (BIAS && i == DC - 1) {
              const int dist = wkey - (row + off);
              add_bias<true>(g, line, s, dist - 31, dist + 31, key - (row + off) - 4 * half);
            }
          } else if constexpr (i < 2 * DC) {
            dp = mma(f, vf[i - DC], dp);
            constexpr int j = i - DC;
#pragma unroll
            for (int r = beside(j, DC, 16); r < beside(j + 1, DC, 16); ++r) {
              const float ls = lse[r / 4][r % 4];
              s[r] = exp2_fast(BIAS ? s[r] - ls : __builtin_fmaf(s[r], g.c, -ls));
              if (hidden(r)) s[r] = 0.f;
            }
            if constexpr (j == DC - 1) {
              if (MASK && (bad_q | bad_g)) {
                const uint32_t seen = bit_range(low, high);
                if (bad_q & seen) poison_k = __builtin_nanf("");
                if (bad_g & seen) poison_v = __builtin_nanf("");
              }
              pf[0] = acc_frag<DT>(s, 0);
              pf[1] = acc_frag<DT>(s, 1);
            }
          } else if constexpr (i < 2 * DC + ND) {
            constexpr int j = i - 2 * DC;
            dv[j % DB] = mma(only_finite<DT>(f, MASK && bad_g), pf[j / DB], dv[j % DB]);
#pragma unroll
            for (int r = beside(j, ND, 16); r < beside(j + 1, ND, 16); ++r) {
              s[r] *= dp[r] - del[r / 4][r % 4];
              if (hidden(r)) s[r] = 0.f;
            }
            if constexpr (j == ND - 1) {
              df[0] = acc_frag<DT>(s, 0);
              df[1] = acc_frag<DT>(s, 1);
            }
          } else {
            constexpr int j = i - 2 * DC - ND;
            dk[j % DB] = mma(only_finite<DT>(f, MASK && bad_q), df[j / DB], dk[j % DB]);
          }
        });
      };
      // A tile of rows, of which this wave's begin at row and in LDS at `tile`.  Rows past
      // the end are zeros with a probability of zero; with a bias they are masked (a
      // table may hold infinities that no pair needs).
      const int stop = wkey < nk ? rows : 0;  // a wave without keys has nothing to do
      const auto attend = [&](int row, int tile, const float* stat) {
        uint32_t rl = row_lane + tile, cl = col_lane + tile;
#pragma unroll 1
        for (int b = 0; b < F::BLOCKS && row < stop; ++b) {
          if (row >= most && (!BIAS || row + 32 <= rows)) {
            block(No(), row, rl, cl, stat, 0, 0);
          } else if (row + 32 > mine) {
            uint32_t bad_q = 0, bad_g = 0;
            if (g.causal) {
              bad_q = rows_not_finite<DT, DP>(rl, 0);
              bad_g = rows_not_finite<DT, DP>(rl, F::KEYS);
            }
            block(Yes(), row, rl, cl, stat, bad_q, bad_g);
          }
          rl += 32 * T::ROW_BYTES;
          cl += 32 * T::ROW_BYTES;
          stat += 32;
          row += 32;
        }
      };

      for (int group = 0; group < g.groups; ++group) {
        const int head0 = (kvh * g.groups + group) * g.pack;
        __syncthreads();  // the previous rows' reads are done
        if constexpr (BIAS) {
          load_bias_first(g.bias, first_of);
          load_bias_line(g.bias, first_of, head0, g.heads, line);
        }
        const char* const qb = row_at<DT>(a.q, q0, head0);
        const char* const gb = row_at<DT>(a.g_o, q0, head0);
        float st = 0.f;
        // The rows' statistics go through a register, into the buffer at the next turn.
        const auto fetch = [&](int row, int buf) {
          if (threadIdx.x < 2 * F::KEYS) {
            const int r = row + (int)threadIdx.x % F::KEYS;
            const bool first = threadIdx.x < F::KEYS;
            st = first ? -kInf : 0.f;
            if (r < rows) {
              const int t = (int)((unsigned)r / (unsigned)g.pack);
              const int64_t i = (head0 + r - t * g.pack) * g.Tq + q0 + t;
              st = first ? a.lse[i] : a.delta[i];
            }
          }
          const int64_t tok = row / g.pack;  // KEYS is a multiple of pack
          const uint32_t at = lds_place(lds) + buf * 2 * F::TILE_BYTES;
          sq.issue(qb + tok * qt, rows - row, g.D, at);
          sg.issue(gb + tok * gt, rows - row, g.D, at + F::TILE_BYTES);
        };
        if (F::BUFS == 2 && begin < rows) fetch(begin, 0);
        int buf = 0;
        for (int row = begin; row < rows; row += F::KEYS, buf ^= F::BUFS - 1) {
          if (F::BUFS == 1) {
            __syncthreads();
            fetch(row, 0);
          }
          float* const stat = stats + buf * 2 * F::KEYS;
          if (threadIdx.x < F::KEYS) st = st == -kInf ? kInf : st * kLog2e;  // no key: P = 0
          if (threadIdx.x < 2 * F::KEYS) stat[threadIdx.x] = st;
          feed_wait();
          if (F::BUFS == 2 && row + F::KEYS < rows) fetch(row + F::KEYS, buf ^ 1);
          const int skip = FEW ? 32 * wave : 0;
          attend(row + skip, buf * 2 * F::TILE_BYTES + skip * T::ROW_BYTES, stat + skip);
        }
      }
      if constexpr (FEW) {
        const auto& z = *again<AttnBwd>();
        const auto out = [&](const auto& t, int i) -> char* {
          const int k = (int)tile * F::OWN + i;
          return k < nk ? row_at<DT>(t, (int64_t)k0 + k, kvh) : nullptr;
        };
        join_waves<DT, DP>(lds, dv, poison_v, 1.f, z.g.D, [&](int i) { return out(z.g_v, i); });
        join_waves<DT, DP>(lds, dk, poison_k, z.g.scale, z.g.D, [&](int i) { return out(z.g_k, i); });
        continue;
      }
      if (valid) {
        const auto& z = *again<AttnBwd>();
        char* pk = row_at<DT>(z.g_k, (int64_t)k0 + key, kvh);
        char* pv = row_at<DT>(z.g_v, (int64_t)k0 + key, kvh);
        const int D = z.g.D;
        const bool kvec = z.g_k.vec, vvec = z.g_v.vec;
        const float scale = z.g.scale + poison_k, one = 1.f + poison_v;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int r = 0; r < 16; r += 4) {
            const int e = 32 * d + acc_row(r) + 4 * half;
            store4<DT>(pv, e, D, vvec, dv[d][r] * one, dv[d][r + 1] * one, dv[d][r + 2] * one,
                       dv[d][r + 3] * one);
            store4<DT>(pk, e, D, kvec, dk[d][r] * scale, dk[d][r + 1] * scale, dk[d][r + 2] * scale,
                       dk[d][r + 3] * scale);
          }
      }
    }
  }
}

// ------------------------------------------------------------ launches

// Workgroups for the tokens of no sequence, of which only the device knows how many
// there are: one for each 64 KB that all tokens would take, at most 256 (8192 tokens of 32
// heads of 128 with as many behind them 586 us, with 64 workgroups 595, without the padding
// 655; 64 x 197 tokens of 12 heads of 64 and 8192 behind them 29, with 64 workgroups 31).
constexpr int64_t GAP_GROUPS = 256;
unsigned gap_groups(const int64_t* start, int64_t rows, int D, int dtype) {
  const int64_t bytes = rows * D * (dtype == 0 ? 4 : 2);
  return start ? (unsigned)std::max<int64_t>(1, std::min(GAP_GROUPS, bytes >> 16)) : 0;
}

// Workgroups for the items: at most 2^20 (a launch holds fewer than 2^32
// threads; the rest go by the loop), a multiple of 8 so that the loop keeps to an XCD.
unsigned groups_for(unsigned items) { return items < (1u << 20) ? items : 1u << 20; }

template <typename A>
hipError_t launch_items(void (*kernel)(A), A a, int bytes, unsigned gaps, hipStream_t s) {
  a.g.launched = groups_for(a.g.items);
  if (bytes > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) {
      (void)hipGetLastError();
      return e;
    }
  }
  void* at[] = {&a};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel),
                                       dim3(a.g.launched + gaps), dim3(256), at,
                                       bytes, s);
  if (e != hipSuccess) (void)hipGetLastError();
  return e;
}

// LDS for a bias: the buckets' first distances and `lines` lines.
int bias_bytes(const AttnShape& g, int lines) {
  return g.bias.table ? 2 * BIAS_FIRST + (2 * (g.bias.reach + BIAS_MARGIN) + 1) * 4 * lines : 0;
}

// The variant for what the call needs: type, bias, and whether every row consists of
// whole 16-byte chunks.
template <typename F>
hipError_t choose(int dtype, bool bias, bool vec, F f) {
  typedef std::integral_constant<int, 0> F32;
  typedef std::integral_constant<int, 1> Bf16;
  const auto pick = [&](auto t) {
    if (bias) return vec ? f(t, std::true_type(), std::true_type())
                         : f(t, std::true_type(), std::false_type());
    return vec ? f(t, std::false_type(), std::true_type())
               : f(t, std::false_type(), std::false_type());
  };
  return dtype == 0 ? pick(F32()) : pick(Bf16());
}

}  // namespace

template <>
hipError_t launch_attention_forward<HLQ_ATTN_D>(const AttnFwd& a, int dtype, bool few,
                                                hipStream_t s) {
  const unsigned gaps = gap_groups(a.g.start_q, a.g.Tq * a.g.heads, a.g.D, dtype);
  return choose(dtype, a.g.bias.table, a.q.vec && a.k.vec && a.v.vec, [&](auto t, auto b, auto v) {
    constexpr int DT = decltype(t)::value, DP = HLQ_ATTN_D;
    constexpr bool BIAS = decltype(b)::value, VEC = decltype(v)::value;
    if (few)
      return launch_items(k_attention_forward<DT, DP, BIAS, true, VEC>, a,
                          FwdShape<DT, DP, true>::LDS + bias_bytes(a.g, 1), gaps, s);
    return launch_items(k_attention_forward<DT, DP, BIAS, false, VEC>, a,
                        FwdShape<DT, DP, false>::LDS + bias_bytes(a.g, 1), gaps, s);
  });
}

template <>
hipError_t launch_attention_backward_q<HLQ_ATTN_D>(const AttnBwd& a, int dtype, bool few,
                                                   hipStream_t s) {
  const bool vec = a.q.vec && a.k.vec && a.v.vec && a.o.vec && a.g_o.vec;
  const int extra = bias_bytes(a.g, 5) + (a.g.bias.table ? (4 * SKEW_SIZE + 8) * 4 : 0);
  return choose(dtype, a.g.bias.table, vec, [&](auto t, auto b, auto v) {
    constexpr int DT = decltype(t)::value, DP = HLQ_ATTN_D;
    constexpr bool BIAS = decltype(b)::value, VEC = decltype(v)::value;
    const unsigned gaps = gap_groups(a.g.start_q, a.g.Tq * a.g.heads, a.g.D, DT);
    if constexpr (attn_few_q(BIAS, DT, DP))
      if (few)
        return launch_items(k_attention_backward_q<DT, DP, BIAS, true, VEC>, a,
                            BwdShape<DT, DP, true, BIAS>::LDS + extra, gaps, s);
    return launch_items(k_attention_backward_q<DT, DP, BIAS, false, VEC>, a,
                        BwdShape<DT, DP, false, BIAS>::LDS + extra, gaps, s);
  });
}

template <>
hipError_t launch_attention_backward_kv<HLQ_ATTN_D>(const AttnBwd& a, int dtype, bool few,
                                                    hipStream_t s) {
  const bool vec = a.q.vec && a.k.vec && a.v.vec && a.g_o.vec;
  return choose(dtype, a.g.bias.table, vec, [&](auto t, auto b, auto v) {
    constexpr int DT = decltype(t)::value, DP = HLQ_ATTN_D;
    constexpr bool BIAS = decltype(b)::value, VEC = decltype(v)::value;
    const unsigned gaps = gap_groups(a.g.start_k, a.g.Tk * a.g.kv_heads, a.g.D, DT);
    const int extra = bias_bytes(a.g, 1);
    if (few)
      return launch_items(
          k_attention_backward_kv<DT, DP, BIAS, true, VEC>, a,
          BwdShape<DT, DP, true>::LDS + 16 * BwdShape<DT, DP, true>::KEYS + extra, gaps, s);
    return launch_items(
        k_attention_backward_kv<DT, DP, BIAS, false, VEC>, a,
        BwdShape<DT, DP, false>::LDS + 16 * BwdShape<DT, DP, false>::KEYS + extra, gaps, s);
  });
}

}  // namespace hlq
