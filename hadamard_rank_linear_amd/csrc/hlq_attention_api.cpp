// C ABI of the attention block's operators: attention over packed sequences,
// forward and backward, with the relative position bias, and dropout.  Argument
// validation, workspace sizes and launches; the arithmetic is in
// hlq_attention.hip, hlq_attention_fold.hip and hlq_dropout.hip.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <initializer_list>
#include <stdint.h>

#include "../../include/hlq.h"
#include "hlq_internal.h"

namespace {

using hlq::AttnBwd;
using hlq::AttnFwd;
using hlq::AttnRows;
using hlq::AttnShape;

constexpr int64_t kRows = int64_t(1) << 30;    // queries times heads, and keys times heads
constexpr int64_t kStride = int64_t(1) << 40;  // elements
// Tokens (fewer elements than this apart): a tile's 128 rows are within 32-bit offsets.
constexpr int64_t kTokenStride = int64_t(1) << 22;

bool dtype_ok(int dt) { return dt == HLQ_F32 || dt == HLQ_BF16; }
size_t esize(int dt) { return dt == HLQ_F32 ? 4 : 2; }
bool aligned(const void* p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// First distances of the buckets exact .. side - 1 of a side:
//   exact + floor((side - exact) log(n / exact) / log(reach / exact)) = k.
// The share of a distance that begins a bucket is a whole number up to rounding, or not
// whole.  Over all sizes allowed here (counted in whole numbers: it is whole when (n /
// exact)^(side - exact) is a power of reach / exact) the whole ones come out at most 2^-47
// off, the others at least 2^-36.4 (side 21, reach 1006, distance 435; the next 2^-31.3): 2^-40
// tells the two apart.
void bucket_bounds(hlq::AttnBias& b) {
  const double span = std::log((double)b.reach / b.exact);
  int k = b.exact;
  b.first[k] = (int16_t)b.exact;
  for (int n = b.exact; n <= b.reach; ++n) {
    const double share = (b.side - b.exact) * (std::log((double)n / b.exact) / span);
    const int at = std::min(b.side - 1, b.exact + (int)std::floor(share + 0x1p-40));
    while (k < at) b.first[++k] = (int16_t)n;
  }
}

hlq_status check_shape(const hlq_attention* a) {
  if (!a) return HLQ_ERR_NULL;
  if (!dtype_ok(a->dtype) || (a->bias && !dtype_ok(a->bias_dtype))) return HLQ_ERR_DTYPE;
  if (a->queries < 0 || a->keys < 0 || a->sequences < 1 || a->heads < 1 || a->kv_heads < 1 ||
      a->heads % a->kv_heads || a->head_dim < 1 || a->head_dim > 128 || a->max_len < 0)
    return HLQ_ERR_SHAPE;
  if (a->heads >= (1 << 16) || a->sequences >= kRows / a->heads || a->queries >= kRows / a->heads ||
      a->keys >= kRows / a->heads)
    return HLQ_ERR_SHAPE;
  if (!a->start_q && (a->sequences != 1 || a->start_k)) return HLQ_ERR_SHAPE;
  if (!a->start_k && a->start_q && a->queries != a->keys) return HLQ_ERR_SHAPE;
  if (!(a->scale > 0.0) || !(a->scale <= 0x1p64) || a->scale < 0x1p-64) return HLQ_ERR_VALUE;
  if (a->bias) {
    const int side = a->bidirectional ? a->buckets / 2 : a->buckets;
    if (a->buckets > 128 || (a->bidirectional && a->buckets % 2) || side < 2 ||
        a->max_distance <= side / 2 || a->max_distance > 1024)
      return HLQ_ERR_VALUE;
    if (!aligned(a->bias, esize(a->bias_dtype))) return HLQ_ERR_ALIGN;
  }
  if (!aligned(a->start_q, 8) || !aligned(a->start_k, 8)) return HLQ_ERR_ALIGN;
  return HLQ_OK;
}

// Pointer and strides of a tensor of `tokens` x `heads` rows; out: rows that do not
// overlap.
hlq_status check_rows(const hlq_attention* a, const hlq_tokens* t, int64_t tokens, int heads,
                      bool out) {
  if (!t) return HLQ_ERR_NULL;
  if (tokens == 0) return HLQ_OK;
  if (!t->data) return HLQ_ERR_NULL;
  if (!aligned(t->data, esize(a->dtype))) return HLQ_ERR_ALIGN;
  if (t->token_stride < 0 || t->head_stride < 0 || (tokens > 1 && t->token_stride >= kTokenStride) ||
      (heads > 1 && t->head_stride >= kStride))
    return HLQ_ERR_SHAPE;
  if (out) {
    const int64_t D = a->head_dim, ts = t->token_stride, hs = t->head_stride;
    const bool tokens_outside = heads == 1 ? ts >= D : hs >= D && ts >= (heads - 1) * hs + D;
    const bool heads_outside = tokens == 1 ? hs >= D : ts >= D && hs >= (tokens - 1) * ts + D;
    if (tokens > 1 && heads > 1 && !tokens_outside && !heads_outside) return HLQ_ERR_SHAPE;
    if (tokens > 1 && heads == 1 && ts < D) return HLQ_ERR_SHAPE;
    if (tokens == 1 && heads > 1 && hs < D) return HLQ_ERR_SHAPE;
  }
  return HLQ_OK;
}

// Whether an output starts where another operand does.
struct Operand {
  const hlq_tokens* t;
  int64_t tokens;
};
bool meets(const Operand& out, std::initializer_list<Operand> others) {
  for (const Operand& x : others)
    if (out.tokens && x.tokens && out.t->data == x.t->data) return true;
  return false;
}

// The kernels' form of them: the stride of a single token, or head, is not looked at.
AttnRows rows_of(const hlq_attention* a, const hlq_tokens* t, int64_t tokens, int heads) {
  const int64_t es = (int64_t)esize(a->dtype);
  AttnRows r = {t->data, tokens > 1 ? t->token_stride : 0, heads > 1 ? t->head_stride : 0, 0};
  r.vec = aligned(t->data, 16) && r.token * es % 16 == 0 && r.head * es % 16 == 0 &&
          a->head_dim * es % 16 == 0;
  return r;
}

AttnShape shape_of(const hlq_attention* a) {
  AttnShape g = {};
  g.start_q = a->start_q;
  g.start_k = a->start_k ? a->start_k : a->start_q;
  g.S = a->sequences;
  g.Tq = a->queries;
  g.Tk = a->keys;
  g.heads = a->heads;
  g.kv_heads = a->kv_heads;
  g.D = a->head_dim;
  g.causal = a->causal != 0;
  g.scale = (float)a->scale;
  g.c = (float)(a->scale * 1.4426950408889634074);
  g.splits = 1;
  const int shared = a->heads / a->kv_heads;
  g.pack = a->bias ? 1 : shared;
  g.groups = shared / g.pack;
  if (a->bias) {
    hlq::AttnBias& b = g.bias;
    b.table = a->bias;
    b.dtype = a->bias_dtype;
    b.buckets = a->buckets;
    b.reach = a->max_distance;
    b.bidirectional = a->bidirectional != 0;
    b.side = b.bidirectional ? a->buckets / 2 : a->buckets;
    b.exact = b.side / 2;
    bucket_bounds(b);
  }
  return g;
}

// How long the sequences are taken to be, where the launch needs a number: one without
// bounds has all tokens; else the caller's longest one (of queries, and of keys with the
// same bounds), or twice the mean.  Longer ones are looped over.
int64_t expected(const hlq_attention* a, int64_t total, bool keys = false) {
  if (!a->start_q) return std::max<int64_t>(1, total);
  const int64_t mean = (total + a->sequences - 1) / a->sequences;
  const int64_t guess = std::min(total, 2 * mean);
  return std::max<int64_t>(
      1, a->max_len && !(keys && a->start_k) ? std::min(total, a->max_len) : guess);
}

// Numbers a launch's work items.  Tiles beyond 2^30 items are looped over.  A unit's
// items (which read the same keys and values, or rows) go to one XCD, where they meet
// in its L2, if that leaves the eight equally busy.  With a causal mask long tiles come
// first, of all units, so that the last to end are short (8192 causal tokens 823 us in
// plain order, 602 so); without one a unit's tiles stay together (8190 ragged tokens
// with a bias, backward, 215 us tile by tile, 168 so).
void number(AttnShape& g, int64_t tiles, int64_t units, int64_t splits) {
  g.splits = (unsigned)splits;
  g.units = (unsigned)units;
  g.tiles = (unsigned)std::max<int64_t>(1, std::min(tiles, (int64_t(1) << 30) / (units * splits)));
  g.by_xcd = units % 8 == 0 || units >= 64;
  g.by_tile = g.causal;
  g.items = g.tiles * g.splits * (g.by_xcd ? (g.units + 7) / 8 * 8 : g.units);
}

struct FwdPlan {
  bool few;
  int64_t tiles, units, splits, share;
};

// Tiles of 128 rows (or keys) that leave compute units without work are cut into
// four, the waves of a workgroup sharing the other side: 2048 causal tokens, 8 heads
// of 64 take 23 us and backward 53, with tiles of 128 39 and 104; ViT-B's 1536 tiles
// 28 and 101 as they are, cut 86 and 200.  With a causal mask the longest tile decides
// up to twice as many (4096 such tokens 72 -> 51 and 195 -> 131 us, 6000 103 -> 91 and
// 286 -> 224), but not where a cut tile fills the LDS (heads of 128, 256 tiles: 32 -> 43
// and 101 -> 133).  All of this is bf16.  The rule takes fp32 along, where small tiles gain
// up to here too (1024 causal tokens, 16 heads of 64: 40 and 111, whole 85 and 261) and
// would beyond, in the forward pass and under a causal mask (4096 causal tokens, 8 heads of
// 64: 323 and 980 as they are, cut 187 and 602; ViT-B 227 and 845, cut 204 and 720; 2048
// tokens, 16 heads, no mask 170 and 505, cut 162 and 590).
constexpr int64_t kUnits = 256;
bool few_tiles(const hlq_attention* a, int64_t rows, int64_t units) {
  const bool small = a->head_dim * esize(a->dtype) <= 128;
  return rows <= hlq::ATTN_FEW || (rows + hlq::ATTN_ROWS - 1) / hlq::ATTN_ROWS * units <
                                      (a->causal && small ? 2 * kUnits : kUnits);
}
// A launch has a sequence's tiles for each of them, and a bias's gradient a line of
// buckets for each tile, so a sequence that is far longer than the rest pays for them all:
// at most kSkew times the tiles that `all` rows can have, a longer one loops over its own
// (131072 causal tokens in 1024 sequences, the longest 32768, 16 heads of 64: forward 6.8
// ms, backward with a bias 25.6; 7.6 and 31.1 with four times as many, 9.4 and 38.9 and 540
// MB of lines without a limit, 15.1 and 38.5 with a quarter).
constexpr int64_t kSkew = 16;
int64_t tiles_of(const hlq_attention* a, int64_t rows, int64_t all, bool few) {
  const int per = few ? hlq::ATTN_FEW : hlq::ATTN_ROWS;
  return std::min((rows + per - 1) / per, kSkew * (all / per + a->sequences) / a->sequences);
}

// If that is too few still, the keys are shared out: in shares of equal length, of
// which all sequences together have about two a CU, 256 keys each at least.  As many
// as the longest sequence is expected to need (at most 64); a longer one's are longer.
// (8 tokens against 32700 keys 51 us, with eight shares a sequence whatever its length
// 59; shares of 128 keys, or more than two a CU: up to 20% slower.)  The shares' sums
// cost what they are long: tiles full of rows are left whole where they occupy half of
// the CUs (512 causal tokens 11 us, shared out 14; 1024 tokens, 32 heads of 128 on 8, 32
// and 61), single tokens only where every CU has one (48 of 700 keys 32, whole 34; 32 of
// 1024, 256 items, 42 and 35).
// Every query has room in the workspace for every share.  A true hint has up to 32 x 256
// rows of queries and heads here, and 40960 with their shares: there are more where tokens
// belong to no sequence, or where the hint is wrong, and then fewer shares (one sequence
// of 65536 tokens, 32 heads of 128, said to be single tokens: 70 GB without that limit).
constexpr int64_t kShareRows = int64_t(1) << 18;
FwdPlan plan_forward(const hlq_attention* a) {
  const int shared = a->bias ? 1 : a->heads / a->kv_heads;
  const int64_t rows = expected(a, a->queries) * shared;
  FwdPlan p;
  p.units = a->sequences * (a->heads / shared);
  p.few = few_tiles(a, rows, p.units);
  p.tiles = tiles_of(a, rows, a->queries * shared, p.few);
  p.splits = 1;
  p.share = 0;
  const int64_t slots = 2 * kUnits, groups = p.tiles * p.units;
  const int64_t mean = a->keys / a->sequences, longest = std::min(a->keys, 2 * mean);
  if (!p.few || groups >= (rows <= hlq::ATTN_FEW ? kUnits : kUnits / 2) || mean < 512) return p;
  const int64_t share = std::max<int64_t>(256, (mean * groups + slots - 1) / slots);
  const int64_t room = kShareRows / std::max<int64_t>(1, a->queries * a->heads);
  p.splits = std::max<int64_t>(1, std::min({int64_t(64), room, (longest + share - 1) / share}));
  p.share = ((longest + p.splits - 1) / p.splits + 127) / 128 * 128;
  return p;
}

size_t forward_bytes(const hlq_attention* a, const FwdPlan& p) {
  if (p.splits == 1) return 0;
  return (size_t)p.splits * a->queries * a->heads * (a->head_dim + 2) * 4;
}

// The gradient of q's items, by which a bias's partial sums are laid out.
AttnShape backward_q_shape(const hlq_attention* a, bool* few) {
  AttnShape g = {};
  const int shared = a->bias ? 1 : a->heads / a->kv_heads;
  g.causal = a->causal != 0;
  const int64_t rows = expected(a, a->queries) * shared;
  const int64_t units = a->sequences * (a->heads / shared);
  *few = few_tiles(a, rows, units) && hlq::attn_few_q(a->bias != nullptr, a->dtype, a->head_dim);
  number(g, tiles_of(a, rows, a->queries * shared, *few), units, 1);
  return g;
}

size_t delta_bytes(const hlq_attention* a) {
  return ((size_t)a->queries * a->heads * 4 + 15) / 16 * 16;
}

template <typename F32, typename F64, typename F96, typename F128>
hipError_t by_size(int D, F32 f32, F64 f64, F96 f96, F128 f128) {
  return D <= 32 ? f32() : D <= 64 ? f64() : D <= 96 ? f96() : f128();
}
#define HLQ_BY_SIZE(D, f, ...)                                                             \
  by_size(D, [&] { return hlq::f<32>(__VA_ARGS__); }, [&] { return hlq::f<64>(__VA_ARGS__); }, \
          [&] { return hlq::f<96>(__VA_ARGS__); }, [&] { return hlq::f<128>(__VA_ARGS__); })

}  // namespace

#define HLQ_TRY(expr)                             \
  do {                                            \
    if ((expr) != hipSuccess) return HLQ_ERR_HIP; \
  } while (0)
#define HLQ_CHECK(expr)                  \
  do {                                   \
    const hlq_status st_ = (expr);       \
    if (st_ != HLQ_OK) return st_;       \
  } while (0)

extern "C" {

int hlq_relative_bucket(int distance, int buckets, int max_distance, int bidirectional) {
  hlq::AttnBias b = {};
  b.side = bidirectional ? buckets / 2 : buckets;
  if (buckets > 128 || (bidirectional && buckets % 2) || b.side < 2 || max_distance <= b.side / 2 ||
      max_distance > 1024)
    return -1;
  b.exact = b.side / 2;
  b.reach = max_distance;
  bucket_bounds(b);
  const int64_t d = distance;
  const int64_t n = bidirectional ? std::llabs(d) : std::max<int64_t>(-d, 0);
  int k = (int)std::min<int64_t>(n, b.exact);
  if (n >= b.exact)
    for (int i = b.exact + 1; i < b.side; ++i) k += n >= b.first[i];
  return k + (bidirectional && d > 0 ? b.side : 0);
}

size_t hlq_attention_forward_workspace_size(const hlq_attention* a) {
  if (check_shape(a) != HLQ_OK) return 0;
  return forward_bytes(a, plan_forward(a));
}

hlq_status hlq_attention_forward(const hlq_attention* a, const hlq_tokens* q, const hlq_tokens* k,
                                 const hlq_tokens* v, const hlq_tokens* o, float* lse,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  HLQ_CHECK(check_shape(a));
  HLQ_CHECK(check_rows(a, q, a->queries, a->heads, false));
  HLQ_CHECK(check_rows(a, k, a->keys, a->kv_heads, false));
  HLQ_CHECK(check_rows(a, v, a->keys, a->kv_heads, false));
  HLQ_CHECK(check_rows(a, o, a->queries, a->heads, true));
  if (a->queries && !lse) return HLQ_ERR_NULL;
  if (!aligned(lse, 4)) return HLQ_ERR_ALIGN;
  const FwdPlan p = plan_forward(a);
  const size_t need = forward_bytes(a, p);
  if (need && (!workspace || workspace_bytes < need)) return HLQ_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return HLQ_ERR_ALIGN;
  // other workgroups still read keys and values when one writes its rows
  if (meets({o, a->queries}, {{k, a->keys}, {v, a->keys}})) return HLQ_ERR_VALUE;
  if (a->queries == 0) return HLQ_OK;
  AttnFwd f = {};
  f.g = shape_of(a);
  f.q = rows_of(a, q, a->queries, a->heads);
  f.k = rows_of(a, k, a->keys, a->kv_heads);
  f.v = rows_of(a, v, a->keys, a->kv_heads);
  f.o = rows_of(a, o, a->queries, a->heads);
  f.lse = lse;
  number(f.g, p.tiles, p.units, p.splits);
  f.g.share = (int)p.share;
  if (need) {
    f.ml = static_cast<float*>(workspace);
    f.po = f.ml + (size_t)p.splits * a->queries * a->heads * 2;
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  HLQ_TRY(HLQ_BY_SIZE(a->head_dim, launch_attention_forward, f, a->dtype, p.few, s));
  if (need) HLQ_TRY(hlq::launch_attention_join(f, a->dtype, s));
  return HLQ_OK;
}

size_t hlq_attention_backward_workspace_size(const hlq_attention* a) {
  if (check_shape(a) != HLQ_OK) return 0;
  size_t bytes = delta_bytes(a);
  bool few;
  if (a->bias)
    bytes += (size_t)backward_q_shape(a, &few).tiles * a->sequences * a->heads * a->buckets * 4;
  return bytes;
}

hlq_status hlq_attention_backward(const hlq_attention* a, const hlq_tokens* g_o,
                                  const hlq_tokens* q, const hlq_tokens* k, const hlq_tokens* v,
                                  const hlq_tokens* o, const float* lse, const hlq_tokens* g_q,
                                  const hlq_tokens* g_k, const hlq_tokens* g_v, void* g_bias,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  HLQ_CHECK(check_shape(a));
  HLQ_CHECK(check_rows(a, g_o, a->queries, a->heads, false));
  HLQ_CHECK(check_rows(a, q, a->queries, a->heads, false));
  HLQ_CHECK(check_rows(a, k, a->keys, a->kv_heads, false));
  HLQ_CHECK(check_rows(a, v, a->keys, a->kv_heads, false));
  HLQ_CHECK(check_rows(a, o, a->queries, a->heads, false));
  HLQ_CHECK(check_rows(a, g_q, a->queries, a->heads, true));
  HLQ_CHECK(check_rows(a, g_k, a->keys, a->kv_heads, true));
  HLQ_CHECK(check_rows(a, g_v, a->keys, a->kv_heads, true));
  if ((a->queries && !lse) || (a->bias != nullptr) != (g_bias != nullptr)) return HLQ_ERR_NULL;
  if (!aligned(lse, 4) || (g_bias && !aligned(g_bias, esize(a->bias_dtype)))) return HLQ_ERR_ALIGN;
  const size_t need = hlq_attention_backward_workspace_size(a);
  if (need && (!workspace || workspace_bytes < need)) return HLQ_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return HLQ_ERR_ALIGN;
  // the gradients of k and v come from q and g_o after that of q is written
  const Operand Q = {q, a->queries}, G = {g_o, a->queries}, GQ = {g_q, a->queries};
  const Operand GK = {g_k, a->keys}, GV = {g_v, a->keys};
  if (meets(GQ, {Q, G, {k, a->keys}, {v, a->keys}, GK, GV}) || meets(GK, {Q, G, GV}) || meets(GV, {Q, G}))
    return HLQ_ERR_VALUE;
  AttnBwd b = {};
  b.g = shape_of(a);
  b.q = rows_of(a, q, a->queries, a->heads);
  b.k = rows_of(a, k, a->keys, a->kv_heads);
  b.v = rows_of(a, v, a->keys, a->kv_heads);
  b.o = rows_of(a, o, a->queries, a->heads);
  b.g_o = rows_of(a, g_o, a->queries, a->heads);
  b.g_q = rows_of(a, g_q, a->queries, a->heads);
  b.g_k = rows_of(a, g_k, a->keys, a->kv_heads);
  b.g_v = rows_of(a, g_v, a->keys, a->kv_heads);
  b.lse = lse;
  b.delta = static_cast<float*>(workspace);
  b.g_line = reinterpret_cast<float*>(static_cast<char*>(workspace) + delta_bytes(a));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  bool few;
  const AttnShape n = backward_q_shape(a, &few);
  number(b.g, n.tiles, n.units, 1);
  // with a bias also for no queries: the table's gradient is then zero
  if (a->queries || a->bias)
    HLQ_TRY(HLQ_BY_SIZE(a->head_dim, launch_attention_backward_q, b, a->dtype, few, s));
  if (a->bias)
    HLQ_TRY(hlq::launch_attention_bias(b.g_line, a->sequences, b.g.tiles, a->heads, a->buckets,
                                       a->bias_dtype, g_bias, s));
  if (a->keys) {
    // Rows that are read through LDS are packed where the heads are a power of two
    // that divides the rows a thread steps over, and near enough for 32-bit offsets.
    const int shared = a->heads / a->kv_heads;
    const int64_t far = std::max(b.q.head, b.g_o.head) * (int64_t)esize(a->dtype) * shared;
    if ((shared & (shared - 1)) || shared > hlq::ATTN_PACK || far >= (int64_t(1) << 30)) b.g.pack = 1;
    b.g.groups = shared / b.g.pack;
    const int64_t keys = expected(a, a->keys, true), units = a->sequences * a->kv_heads;
    few = few_tiles(a, keys, units);
    number(b.g, tiles_of(a, keys, a->keys, few), units, 1);
    HLQ_TRY(HLQ_BY_SIZE(a->head_dim, launch_attention_backward_kv, b, a->dtype, few, s));
  }
  return HLQ_OK;
}

static hlq_status dropout(const void* x, const void* residual, int dtype, int64_t n, double p,
                          const int64_t* seed, uint32_t site, void* y, void* stream) {
  if (!seed || (n && (!x || !y))) return HLQ_ERR_NULL;
  if (!dtype_ok(dtype)) return HLQ_ERR_DTYPE;
  if (n < 0 || n >= (int64_t(1) << 35)) return HLQ_ERR_SHAPE;
  if (!(p >= 0.0 && p <= 1.0)) return HLQ_ERR_VALUE;
  if (!aligned(x, esize(dtype)) || !aligned(residual, esize(dtype)) || !aligned(y, esize(dtype)) ||
      !aligned(seed, 8))
    return HLQ_ERR_ALIGN;
  hlq::DropArgs a = {x, residual, y, n, seed, site, 0, 0.f};
  a.limit = (uint32_t)std::nearbyint(p * 65536.0);  // ties to even, as in the definition
  a.scale = a.limit < 65536 ? (float)(65536.0 / (65536 - a.limit)) : 0.f;
  HLQ_TRY(hlq::launch_dropout(a, dtype, static_cast<hipStream_t>(stream)));
  return HLQ_OK;
}

hlq_status hlq_dropout_forward(const void* x, const void* residual, int dtype, int64_t n, double p,
                               const int64_t* seed, uint32_t site, void* y, void* stream) {
  return dropout(x, residual, dtype, n, p, seed, site, y, stream);
}

hlq_status hlq_dropout_backward(const void* g_y, int dtype, int64_t n, double p,
                                const int64_t* seed, uint32_t site, void* g_x, void* stream) {
  return dropout(g_y, nullptr, dtype, n, p, seed, site, g_x, stream);
}

}  // extern "C"
