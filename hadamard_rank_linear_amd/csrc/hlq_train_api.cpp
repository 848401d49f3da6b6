// C ABI of the operators of a training step around the linear layer: layer
// norm, token log probabilities with the policy and preference losses, and
// gradient clipping.  Argument validation, workspace sizes and launches; all
// arithmetic happens in the kernels of hlq_norm.hip, hlq_logprob.hip and
// hlq_clip.hip.
#include <hip/hip_runtime.h>

#include <cmath>
#include <stdint.h>

#include "../../include/hlq.h"
#include "hlq_internal.h"

namespace {

constexpr int64_t kMax = int64_t(1) << 31;
// Data of this size and more is read past the last-level cache (256 MB): with
// what is written beside it, it would not be found there again, and filling the
// cache evicts what earlier kernels left there to be written back.  Measured
// with inputs another kernel has just displaced: scoring 1023 x 48003 fp32 (196
// MB) 34 us past the cache and 57 through it, 4096 x 32000 bf16 46 and 76;
// clipping 48, 100 and 220 MB 33, 59 and 122 us and 39, 75 and 159.  With inputs
// just written: clipping 32 and 64 MB 30 and 43 us, and 24 and 38; the gradient
// after scoring 500 and 1024 x 32000 bf16 14 and 24 us, and 11 and 22.
constexpr int64_t kStreamBytes = int64_t(96) << 20;

bool dtype_ok(int dt) { return dt == HLQ_F32 || dt == HLQ_BF16; }
size_t esize(int dt) { return dt == HLQ_F32 ? 4 : 2; }

bool aligned(const void* p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

bool any_null(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p) return true;
  return false;
}

bool all_aligned(size_t bytes, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, bytes)) return false;
  return true;
}

bool positive(double v) { return v > 0.0 && std::isfinite(v); }
bool not_negative(double v) { return v >= 0.0 && std::isfinite(v); }

hlq_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need && (!ws || have < need)) return HLQ_ERR_WORKSPACE;
  return aligned(ws, 16) ? HLQ_OK : HLQ_ERR_ALIGN;
}

bool norm_shape_ok(int64_t T, int64_t C) { return T >= 0 && T < kMax && C >= 1 && C < kMax; }

// Rows of logits: T x V at pitch ld.  A row's bytes are addressed in 32 bits.
bool rows_ok(int64_t T, int64_t V, int64_t ld) {
  return T >= 0 && T < kMax && V >= 1 && V < kMax / 2 && ld >= V && ld < (int64_t(1) << 40);
}

// Its exponent scale * log2(e) splits into two normal fp32 numbers.
bool scale_ok(double v) { return v >= 0x1p-64 && v <= 0x1p64; }

hlq::LogitArgs logit_args(const void* logits, int dtype, int64_t ld, const int64_t* targets,
                          int64_t T, int64_t V, double scale) {
  hlq::LogitArgs a = {};
  a.logits = logits;
  a.targets = targets;
  a.T = T; a.V = V; a.ld = ld; a.g_ld = V;
  a.stream = T * V * (int64_t)esize(dtype) > kStreamBytes;
  a.scale = scale;
  const double c = scale * 1.4426950408889634074;
  a.c = (float)c;
  a.c_hi = std::nextafter((float)c, 0.f);
  a.c_lo = (float)(c - (double)a.c_hi);
  return a;
}

bool policy_values_ok(double lo, double hi, double kl) {
  return not_negative(lo) && lo <= 1.0 && not_negative(hi) && not_negative(kl);
}

}  // namespace

#define HLQ_TRY(expr)                             \
  do {                                            \
    if ((expr) != hipSuccess) return HLQ_ERR_HIP; \
  } while (0)

extern "C" {

hlq_status hlq_layer_norm_forward(const void* x, const void* residual, int dtype,
                                  const void* weight, const void* bias, int param_dtype,
                                  int64_t T, int64_t C, double eps, void* y, void* h,
                                  float* mean, float* rstd, void* stream) {
  if (!weight || (T && any_null({x, y, mean, rstd}))) return HLQ_ERR_NULL;
  if (T && (residual == nullptr) != (h == nullptr)) return HLQ_ERR_NULL;
  if (!dtype_ok(dtype) || !dtype_ok(param_dtype)) return HLQ_ERR_DTYPE;
  if (!norm_shape_ok(T, C)) return HLQ_ERR_SHAPE;
  if (!not_negative(eps)) return HLQ_ERR_VALUE;
  if (!all_aligned(esize(dtype), {x, residual, y, h}) ||
      !all_aligned(esize(param_dtype), {weight, bias}) || !all_aligned(4, {mean, rstd}))
    return HLQ_ERR_ALIGN;
  const hlq::NormFwd a = {x, residual, weight, bias, param_dtype, T, C, (float)eps,
                          y, h,        mean,   rstd};
  HLQ_TRY(hlq::launch_norm_forward(a, dtype, static_cast<hipStream_t>(stream)));
  return HLQ_OK;
}

size_t hlq_layer_norm_backward_workspace_size(int64_t T, int64_t C, int dtype) {
  if (!norm_shape_ok(T, C) || !dtype_ok(dtype)) return 0;
  return (size_t)hlq::norm_parts(T, C, dtype) * 2 * (size_t)C * 4;
}

hlq_status hlq_layer_norm_backward(const void* g_y, const void* h, const void* g_h, int dtype,
                                   const float* mean, const float* rstd, const void* weight,
                                   int param_dtype, int64_t T, int64_t C, void* g_x,
                                   void* g_weight, void* g_bias, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (any_null({weight, g_weight}) || (T && any_null({g_y, h, mean, rstd, g_x})))
    return HLQ_ERR_NULL;
  if (!dtype_ok(dtype) || !dtype_ok(param_dtype)) return HLQ_ERR_DTYPE;
  if (!norm_shape_ok(T, C)) return HLQ_ERR_SHAPE;
  if (!all_aligned(esize(dtype), {g_y, h, g_h, g_x}) ||
      !all_aligned(esize(param_dtype), {weight, g_weight, g_bias}) ||
      !all_aligned(4, {mean, rstd}))
    return HLQ_ERR_ALIGN;
  const hlq_status st = check_workspace(workspace, workspace_bytes,
                                        hlq_layer_norm_backward_workspace_size(T, C, dtype));
  if (st != HLQ_OK) return st;
  const hlq::NormBwd a = {g_y, h, g_h,      mean,   rstd, weight, param_dtype, T, C,
                          hlq::norm_parts(T, C, dtype),
                          g_x, g_weight, g_bias, static_cast<float*>(workspace)};
  HLQ_TRY(hlq::launch_norm_backward(a, dtype, static_cast<hipStream_t>(stream)));
  return HLQ_OK;
}

hlq_status hlq_token_logprob_forward(const void* logits, int dtype, int64_t ld,
                                     const int64_t* targets, int64_t T, int64_t V, double scale,
                                     float* logprob, float* stats, void* stream) {
  if (T && any_null({logits, targets, logprob, stats})) return HLQ_ERR_NULL;
  if (!dtype_ok(dtype)) return HLQ_ERR_DTYPE;
  if (!rows_ok(T, V, ld)) return HLQ_ERR_SHAPE;
  if (!scale_ok(scale)) return HLQ_ERR_VALUE;
  if (!aligned(logits, esize(dtype)) || !aligned(targets, 8) || !all_aligned(4, {logprob, stats}))
    return HLQ_ERR_ALIGN;
  hlq::LogitArgs a = logit_args(logits, dtype, ld, targets, T, V, scale);
  a.logprob = logprob;
  a.stats = stats;
  HLQ_TRY(hlq::launch_logprob(a, dtype, static_cast<hipStream_t>(stream)));
  return HLQ_OK;
}

hlq_status hlq_token_logprob_backward(const float* g_logprob, const void* logits, int dtype,
                                      int64_t ld, const int64_t* targets, const float* stats,
                                      int64_t T, int64_t V, double scale, void* g_x,
                                      int64_t g_ld, void* stream) {
  if (T && any_null({g_logprob, logits, targets, stats, g_x})) return HLQ_ERR_NULL;
  if (!dtype_ok(dtype)) return HLQ_ERR_DTYPE;
  if (!rows_ok(T, V, ld) || !rows_ok(T, V, g_ld)) return HLQ_ERR_SHAPE;
  if (!scale_ok(scale)) return HLQ_ERR_VALUE;
  if (!all_aligned(esize(dtype), {logits, g_x}) || !aligned(targets, 8) ||
      !all_aligned(4, {g_logprob, stats}))
    return HLQ_ERR_ALIGN;
  hlq::LogitArgs a = logit_args(logits, dtype, ld, targets, T, V, scale);
  a.g_logprob = g_logprob;
  a.stats = const_cast<float*>(stats);
  a.g_x = g_x;
  a.g_ld = g_ld;
  HLQ_TRY(hlq::launch_logprob_grad(a, dtype, static_cast<hipStream_t>(stream)));
  return HLQ_OK;
}

size_t hlq_policy_loss_workspace_size(int64_t T) {
  return T > 0 && T < kMax ? (size_t)T * 3 * 8 : 0;
}

hlq_status hlq_policy_loss(const float* logprob, const float* old_logprob,
                           const float* advantage, const float* weight,
                           const float* ref_logprob, int64_t T, double clip_low,
                           double clip_high, double kl_coef, float* sums, float* g_logprob,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (!sums || (T && any_null({logprob, old_logprob, advantage, g_logprob}))) return HLQ_ERR_NULL;
  if (T < 0 || T >= kMax) return HLQ_ERR_SHAPE;
  if (!policy_values_ok(clip_low, clip_high, kl_coef)) return HLQ_ERR_VALUE;
  if (T && (ref_logprob != nullptr) != (kl_coef != 0.0)) return HLQ_ERR_NULL;
  if (!all_aligned(4, {logprob, old_logprob, advantage, weight, ref_logprob, sums, g_logprob}))
    return HLQ_ERR_ALIGN;
  const hlq_status st =
      check_workspace(workspace, workspace_bytes, hlq_policy_loss_workspace_size(T));
  if (st != HLQ_OK) return st;
  const hlq::PolicyArgs p = {logprob,  old_logprob, advantage, weight, ref_logprob, T,
                             clip_low, clip_high,   kl_coef,   sums,   g_logprob,
                             static_cast<double*>(workspace)};
  HLQ_TRY(hlq::launch_policy(p, static_cast<hipStream_t>(stream)));
  return HLQ_OK;
}

hlq_status hlq_policy_loss_logits(const void* logits, int dtype, int64_t ld,
                                  const int64_t* targets, const float* old_logprob,
                                  const float* advantage, const float* weight,
                                  const float* ref_logprob, int64_t T, int64_t V, double scale,
                                  double clip_low, double clip_high, double kl_coef,
                                  float* sums, float* logprob, void* g_x, int64_t g_ld,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  if (!sums || (T && any_null({logits, targets, old_logprob, advantage, logprob, g_x})))
    return HLQ_ERR_NULL;
  if (!dtype_ok(dtype)) return HLQ_ERR_DTYPE;
  if (!rows_ok(T, V, ld) || !rows_ok(T, V, g_ld)) return HLQ_ERR_SHAPE;
  if (!scale_ok(scale) || !policy_values_ok(clip_low, clip_high, kl_coef)) return HLQ_ERR_VALUE;
  if (T && (ref_logprob != nullptr) != (kl_coef != 0.0)) return HLQ_ERR_NULL;
  if (!all_aligned(esize(dtype), {logits, g_x}) || !aligned(targets, 8) ||
      !all_aligned(4, {old_logprob, advantage, weight, ref_logprob, sums, logprob}))
    return HLQ_ERR_ALIGN;
  const hlq_status st =
      check_workspace(workspace, workspace_bytes, hlq_policy_loss_workspace_size(T));
  if (st != HLQ_OK) return st;
  hlq::LogitArgs a = logit_args(logits, dtype, ld, targets, T, V, scale);
  a.logprob = logprob;
  a.g_x = g_x;
  a.g_ld = g_ld;
  const hlq::PolicyArgs p = {nullptr,  old_logprob, advantage, weight, ref_logprob, T,
                             clip_low, clip_high,   kl_coef,   sums,   nullptr,
                             static_cast<double*>(workspace)};
  HLQ_TRY(hlq::launch_policy_logits(a, p, dtype, static_cast<hipStream_t>(stream)));
  return HLQ_OK;
}

size_t hlq_preference_loss_workspace_size(int64_t P) {
  return P > 0 && P < kMax / 2 ? (size_t)P * 8 : 0;
}

hlq_status hlq_preference_loss(const float* logprob, const float* ref_logprob,
                               const float* weight, const int64_t* start, int64_t P, int64_t T,
                               double beta, double label_smoothing, int reduction, float* loss,
                               float* margin, float* g_logprob, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (any_null({start, loss, margin}) || (T && any_null({logprob, g_logprob})))
    return HLQ_ERR_NULL;
  if (P < 1 || P >= (int64_t(1) << 24) || T < 0 || T >= kMax) return HLQ_ERR_SHAPE;
  if (!positive(beta) || !not_negative(label_smoothing) || label_smoothing > 1.0)
    return HLQ_ERR_VALUE;
  if (reduction != HLQ_SUM && reduction != HLQ_MEAN) return HLQ_ERR_MODE;
  if (!aligned(start, 8) ||
      !all_aligned(4, {logprob, ref_logprob, weight, loss, margin, g_logprob}))
    return HLQ_ERR_ALIGN;
  const hlq_status st =
      check_workspace(workspace, workspace_bytes, hlq_preference_loss_workspace_size(P));
  if (st != HLQ_OK) return st;
  const hlq::PrefArgs p = {logprob, ref_logprob, weight, start, P, T, beta, label_smoothing,
                           reduction == HLQ_MEAN, loss, margin, g_logprob,
                           static_cast<double*>(workspace), 0};
  HLQ_TRY(hlq::launch_preference(p, static_cast<hipStream_t>(stream)));
  return HLQ_OK;
}

}  // extern "C"

namespace {

// Workgroups of a list: one per chunk up to CLIP_GROUPS.
unsigned clip_groups(uint32_t chunks) {
  return chunks < hlq::CLIP_GROUPS ? chunks : hlq::CLIP_GROUPS;
}

// Walks the tensors in lists that fit a kernel's arguments, calling f on each.
// Empty tensors are left out.
template <typename F>
hlq_status for_lists(const void* const* grads, void* const* outs, const int64_t* sizes,
                     const int* dtypes, int64_t count, F f) {
  hlq::ClipList l;
  l.count = 0;
  l.chunks = 0;
  l.in_place = 1;
  for (int64_t i = 0; i < count; ++i) {
    const size_t es = esize(dtypes[i]);
    for (int64_t at = 0; at < sizes[i]; at += hlq::CLIP_MAX_SIZE) {
      const int64_t left = sizes[i] - at;
      const int64_t n = left < hlq::CLIP_MAX_SIZE ? left : hlq::CLIP_MAX_SIZE;
      const int k = l.count;
      l.grad[k] = grads ? static_cast<const char*>(grads[i]) + at * es : nullptr;
      l.out[k] = outs ? static_cast<char*>(outs[i]) + at * es : const_cast<void*>(l.grad[k]);
      if (l.out[k] != l.grad[k]) l.in_place = 0;
      l.size[k] = (uint32_t)n | (dtypes[i] == HLQ_BF16 ? 0x80000000u : 0u);
      l.first[k] = l.chunks;
      l.chunks += (uint32_t)((n * es + hlq::CLIP_BYTES - 1) / hlq::CLIP_BYTES);
      if (++l.count == hlq::CLIP_LIST) {
        const hlq_status st = f(l);
        if (st != HLQ_OK) return st;
        l.count = 0;
        l.chunks = 0;
        l.in_place = 1;
      }
    }
  }
  return l.count ? f(l) : HLQ_OK;
}

bool clip_sizes_ok(const int64_t* sizes, int64_t count) {
  if (count < 0 || count >= (int64_t(1) << 24)) return false;
  for (int64_t i = 0; i < count; ++i)
    if (sizes[i] < 0 || sizes[i] >= (int64_t(1) << 40)) return false;
  return true;
}

}  // namespace

extern "C" {

size_t hlq_clip_grad_norm_workspace_size(const int64_t* sizes, int64_t count) {
  if ((count > 0 && !sizes) || !clip_sizes_ok(sizes, count)) return 0;
  // one partial per workgroup, CLIP_GROUPS at most per list of CLIP_LIST
  int64_t entries = 0;
  for (int64_t i = 0; i < count; ++i)
    entries += (sizes[i] + hlq::CLIP_MAX_SIZE - 1) / hlq::CLIP_MAX_SIZE;
  return (size_t)((entries + hlq::CLIP_LIST - 1) / hlq::CLIP_LIST) * hlq::CLIP_GROUPS * 8;
}

hlq_status hlq_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* sizes,
                              const int* dtypes, int64_t count, double max_norm, int norm_kind,
                              double* norm, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (!norm || (count > 0 && any_null({grads, sizes, dtypes}))) return HLQ_ERR_NULL;
  if (!clip_sizes_ok(sizes, count)) return HLQ_ERR_SHAPE;
  if (norm_kind != HLQ_NORM_L2 && norm_kind != HLQ_NORM_INF) return HLQ_ERR_MODE;
  if (!(max_norm >= 0.0)) return HLQ_ERR_VALUE;
  int64_t bytes = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (!dtype_ok(dtypes[i])) return HLQ_ERR_DTYPE;
    if (sizes[i] && (!grads[i] || (outs && !outs[i]))) return HLQ_ERR_NULL;
    if (!aligned(grads[i], esize(dtypes[i])) || (outs && !aligned(outs[i], esize(dtypes[i]))))
      return HLQ_ERR_ALIGN;
    bytes += sizes[i] * (int64_t)esize(dtypes[i]);
  }
  if (!aligned(norm, 8)) return HLQ_ERR_ALIGN;
  const hlq_status st = check_workspace(workspace, workspace_bytes,
                                        hlq_clip_grad_norm_workspace_size(sizes, count));
  if (st != HLQ_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool large = bytes > kStreamBytes;
  double* part = static_cast<double*>(workspace);
  int64_t parts = 0;
  hlq_status r = for_lists(grads, outs, sizes, dtypes, count, [&](const hlq::ClipList& l) {
    HLQ_TRY(hlq::launch_clip_norm(l, norm_kind, part + parts, clip_groups(l.chunks), large, s));
    parts += clip_groups(l.chunks);
    return HLQ_OK;
  });
  if (r != HLQ_OK) return r;
  bool first = true;
  r = for_lists(grads, outs, sizes, dtypes, count, [&](const hlq::ClipList& l) {
    HLQ_TRY(hlq::launch_clip_scale(l, norm_kind, part, parts, max_norm, first ? norm : nullptr,
                                   clip_groups(l.chunks), large, s));
    first = false;
    return HLQ_OK;
  });
  if (r != HLQ_OK || !first) return r;
  hlq::ClipList none = {};  // no elements: the norm is 0
  HLQ_TRY(hlq::launch_clip_scale(none, norm_kind, part, 0, max_norm, norm, 1, false, s));
  return HLQ_OK;
}

}  // extern "C"
