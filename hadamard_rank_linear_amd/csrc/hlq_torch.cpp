// Native half of the Python binding of the training step's operators: checks
// of tensors, allocation of outputs and workspaces, the current stream and the
// call of the C ABI, in one step per operator.
//
// These operators are called on single tokens, short sequences and long lists
// of small tensors, where the work on the GPU takes 5 to 10 us.  The same steps
// written in Python (with ctypes, as the linear layer's entry points are) took
// the host 17 to 23 us per call and 185 us for the clipping of 146 tensors,
// longer than the kernels run; here they take 4 to 6 and 12 us, kernel launches
// included.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/StreamGuard.h>
#include <c10/hip/HIPStream.h>
#include <dlfcn.h>
#include <limits.h>
#include <stdarg.h>
#include <stdio.h>

#include <optional>
#include <string>
#include <vector>

#include "../../include/hlq.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

PyObject* g_check = nullptr;  // hlq._check(name, status): raises HLQError

#define HLQ_FUNCTIONS(F)                                                                  \
  F(hlq_layer_norm_forward) F(hlq_layer_norm_backward_workspace_size)                     \
  F(hlq_layer_norm_backward) F(hlq_token_logprob_forward) F(hlq_token_logprob_backward)   \
  F(hlq_policy_loss_workspace_size) F(hlq_policy_loss) F(hlq_policy_loss_logits)          \
  F(hlq_preference_loss_workspace_size) F(hlq_preference_loss)                            \
  F(hlq_clip_grad_norm_workspace_size) F(hlq_clip_grad_norm)

// The C ABI of the library that the Python binding has loaded.
struct Library {
#define F(name) decltype(&::name) name;
  HLQ_FUNCTIONS(F)
#undef F
} lib;

// ------------------------------------------------------------ checks

std::string format(const char* f, va_list v) {
  char buf[512];
  vsnprintf(buf, sizeof buf, f, v);
  return buf;
}
[[noreturn]] void type_error(const char* f, ...) {
  va_list v;
  va_start(v, f);
  const std::string s = format(f, v);
  va_end(v);
  PyErr_SetString(PyExc_TypeError, s.c_str());
  throw python_error();
}
[[noreturn]] void value_error(const char* f, ...) {
  va_list v;
  va_start(v, f);
  const std::string s = format(f, v);
  va_end(v);
  PyErr_SetString(PyExc_ValueError, s.c_str());
  throw python_error();
}

std::string text(IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + (v.size() == 1 ? ",)" : ")");
}

std::string type_name(ScalarType t) {
  std::string s = at::toString(t);
  if (s == "Float") return "torch.float32";
  if (s == "BFloat16") return "torch.bfloat16";
  if (s == "Long") return "torch.int64";
  if (s == "Byte") return "torch.uint8";
  return s;
}

// An argument that has to be a tensor.
const Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o))
    type_error("%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// An argument that may be None.
const Tensor* maybe(const char* name, PyObject* o) {
  return o == Py_None ? nullptr : &tensor(name, o);
}

void expect(const char* name, const Tensor& t, ScalarType type, IntArrayRef shape) {
  if (t.scalar_type() != type)
    type_error("%s must be %s, got %s", name, type_name(type).c_str(),
                           type_name(t.scalar_type()).c_str());
  if (t.sizes() != shape)
    value_error("%s must have shape %s, got %s", name, text(shape).c_str(),
                            text(t.sizes()).c_str());
}

void on_gpu(const Tensor& t) {
  if (!t.is_cuda()) value_error("tensors must live on the GPU");
}

// On the GPU of `like`, contiguous unless the caller checks the layout itself.
void same_gpu(const Tensor& like, std::initializer_list<const Tensor*> ts) {
  on_gpu(like);
  for (const Tensor* t : ts) {
    if (!t) continue;
    on_gpu(*t);
    if (t->device() != like.device())
      value_error("tensors on different devices: %s and %s",
                              like.device().str().c_str(), t->device().str().c_str());
    if (!t->is_contiguous()) value_error("tensors must be contiguous");
  }
}

int code(const Tensor& t) {
  if (t.scalar_type() == ScalarType::Float) return HLQ_F32;
  if (t.scalar_type() == ScalarType::BFloat16) return HLQ_BF16;
  type_error("unsupported dtype %s; use float32 or bfloat16",
                         type_name(t.scalar_type()).c_str());
}

double number(const char* name, PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error("%s must be a number, got %s", name, Py_TYPE(o)->tp_name);
  }
  return v;
}

int integer(const char* name, PyObject* o) {
  int over = 0;
  const long v = PyLong_AsLongAndOverflow(o, &over);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error("%s must be an integer, got %s", name, Py_TYPE(o)->tp_name);
  }
  if (over || v < INT_MIN || v > INT_MAX) value_error("%s is out of range", name);
  return (int)v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}

// ------------------------------------------------------------ calls

template <typename P = void>
P* ptr(const Tensor* t) {
  return t ? static_cast<P*>(t->data_ptr()) : nullptr;
}
template <typename P = void>
P* ptr(const Tensor& t) {
  return static_cast<P*>(t.data_ptr());
}

// A new contiguous tensor on the GPU of `like`, from torch's allocator without
// the way through the dispatcher.
Tensor make(const at::Device& device, ScalarType type, IntArrayRef shape) {
  return at::detail::empty_cuda(shape, type, device, std::nullopt);
}
Tensor make(const Tensor& like, ScalarType type, IntArrayRef shape) {
  return make(like.device(), type, shape);
}

// The stream of an argument that has to be a torch.cuda.Stream of `device`.
c10::Stream stream_of(PyObject* o, const at::Device& device) {
  if (!THPStream_Check(o))
    type_error("stream must be a torch.cuda.Stream, got %s", Py_TYPE(o)->tp_name);
  const THPStream* s = reinterpret_cast<THPStream*>(o);
  const c10::Stream stream =
      c10::Stream::unpack3(s->stream_id, static_cast<c10::DeviceIndex>(s->device_index),
                           static_cast<c10::DeviceType>(s->device_type));
  if (stream.device() != device)
    value_error("the stream is on %s, the tensors on %s", stream.device().str().c_str(),
                device.str().c_str());
  return stream;
}

// The GPU of a call is current while it lasts, and so is its stream: the given
// torch.cuda.Stream or the one that was current (None).  Outputs and workspaces
// then come from the pool of the stream that writes them; a block of the caller's
// stream could be one that it has just freed and still has work in flight for.
struct Launch {
  c10::DeviceGuard guard;
  c10::OptionalStreamGuard on_given;
  bool other = false;  // the given stream is not the caller's
  void* stream;
  Launch(const Tensor& like, PyObject* o) : Launch(like.device(), o) {}
  Launch(const at::Device& device, PyObject* o) : guard(device) {
    if (o != Py_None) {
      on_given.reset_stream(stream_of(o, device));
      other = *on_given.original_stream() != *on_given.current_stream();
    }
    stream = c10::hip::getCurrentHIPStream(device.index()).stream();
  }
  // Tensors of the caller that the call reads or writes: if the caller drops
  // them, their memory stays theirs until the given stream has passed the call.
  void use(const Tensor& t) const {
    if (other) t.record_stream(*on_given.current_stream());
  }
  void use(std::initializer_list<const Tensor*> ts) const {
    for (const Tensor* t : ts)
      if (t) use(*t);
  }
  // New tensors that the call returns: if dropped, theirs until the caller's stream
  // has done with them.
  void give(std::initializer_list<const Tensor*> ts) const {
    if (!other) return;
    for (const Tensor* t : ts)
      if (t) t->record_stream(*on_given.original_stream());
  }
};

void check(const char* name, hlq_status status) {
  if (status == HLQ_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "si", name, (int)status);
  Py_XDECREF(r);
  throw python_error();
}

// Tensors of the caller that the call has written: autograd's version counter
// tells a backward pass that what it saved is not there any more, as torch's own
// in-place operations do (tensors made in inference mode have none).
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(std::initializer_list<const Tensor*> ts) {
  for (const Tensor* t : ts)
    if (t) written(*t);
}

Tensor workspace(const Tensor* given, size_t need, const Tensor& like) {
  if (!given) return make(like, ScalarType::Byte, {(int64_t)std::max<size_t>(need, 256)});
  if (given->scalar_type() != ScalarType::Byte || given->dim() != 1)
    type_error("workspace must be a 1-D uint8 tensor");
  same_gpu(like, {given});
  return *given;
}

PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}
PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

template <typename... Ts>
PyObject* tuple(Ts... items) {
  PyObject* t = PyTuple_New(sizeof...(items));
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(t, i++, items), ...);
  return t;
}

void count(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) type_error("expected %zd arguments, got %zd", want, got);
}

// ------------------------------------------------------------ layer norm

void check_params(const Tensor& weight, const Tensor* bias, int64_t C) {
  expect("weight", weight, weight.scalar_type(), {C});
  if (bias) expect("bias", *bias, weight.scalar_type(), {C});
}

// (x, weight, bias, eps, residual, y, h, stream) -> (y, h, mean, rstd)
PyObject* layer_norm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  const Tensor& x = tensor("x", a[0]);
  const Tensor& w = tensor("weight", a[1]);
  const Tensor* b = maybe("bias", a[2]);
  const double eps = number("eps", a[3]);
  const Tensor* residual = maybe("residual", a[4]);
  const Tensor* y_in = maybe("y", a[5]);
  const Tensor* h_in = maybe("h", a[6]);
  if (!x.dim()) value_error("x must have at least one dimension");
  const int64_t C = x.size(-1), T = C ? x.numel() / C : 0;
  check_params(w, b, C);
  if (residual) expect("residual", *residual, x.scalar_type(), x.sizes());
  if (h_in && !residual)
    value_error("h is an output of the residual addition: no residual was given");
  if (h_in) expect("h", *h_in, x.scalar_type(), x.sizes());
  if (y_in) expect("y", *y_in, x.scalar_type(), x.sizes());
  same_gpu(x, {&x, residual, &w, b, y_in, h_in});
  const Launch on(x, a[7]);
  on.use({&x, residual, &w, b, y_in, h_in});
  const Tensor y = y_in ? *y_in : make(x, x.scalar_type(), x.sizes());
  std::optional<Tensor> h;
  if (residual) h = h_in ? *h_in : make(x, x.scalar_type(), x.sizes());
  const IntArrayRef rows = x.sizes().slice(0, x.dim() - 1);
  const Tensor mean = make(x, ScalarType::Float, rows), rstd = make(x, ScalarType::Float, rows);
  check("hlq_layer_norm_forward",
        lib.hlq_layer_norm_forward(ptr(x), ptr(residual), code(x), ptr(w), ptr(b), code(w), T, C,
                                   eps, ptr(y), h ? ptr(*h) : nullptr, ptr<float>(mean),
                                   ptr<float>(rstd), on.stream));
  written({y_in, h_in});
  on.give({&y, h ? &*h : nullptr, &mean, &rstd});
  return tuple(wrap(y), wrap(h ? *h : x), wrap(mean), wrap(rstd));
  END_HANDLE_TH_ERRORS
}

// (g_y, h, mean, rstd, weight, g_h, with_bias, g_x, workspace, stream)
//   -> (g_x, g_weight, g_bias)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const Tensor& g_y = tensor("g_y", a[0]);
  const Tensor& h = tensor("h", a[1]);
  const Tensor& mean = tensor("mean", a[2]);
  const Tensor& rstd = tensor("rstd", a[3]);
  const Tensor& w = tensor("weight", a[4]);
  const Tensor* g_h = maybe("g_h", a[5]);
  const bool with_bias = truth(a[6]);
  const Tensor* g_x_in = maybe("g_x", a[7]);
  const Tensor* ws_in = maybe("workspace", a[8]);
  if (!h.dim()) value_error("h must have at least one dimension");
  const int64_t C = h.size(-1), T = C ? h.numel() / C : 0;
  check_params(w, nullptr, C);
  const IntArrayRef rows = h.sizes().slice(0, h.dim() - 1);
  expect("g_y", g_y, h.scalar_type(), h.sizes());
  expect("mean", mean, ScalarType::Float, rows);
  expect("rstd", rstd, ScalarType::Float, rows);
  if (g_h) expect("g_h", *g_h, h.scalar_type(), h.sizes());
  if (g_x_in) expect("g_x", *g_x_in, h.scalar_type(), h.sizes());
  same_gpu(h, {&h, &g_y, &mean, &rstd, &w, g_h, g_x_in});
  const Launch on(h, a[9]);
  on.use({&h, &g_y, &mean, &rstd, &w, g_h, g_x_in, ws_in});
  const Tensor g_x = g_x_in ? *g_x_in : make(h, h.scalar_type(), h.sizes());
  const Tensor g_w = make(h, w.scalar_type(), {C});
  std::optional<Tensor> g_b;
  if (with_bias) g_b = make(h, w.scalar_type(), {C});
  const Tensor ws =
      workspace(ws_in, lib.hlq_layer_norm_backward_workspace_size(T, C, code(h)), h);
  check("hlq_layer_norm_backward",
        lib.hlq_layer_norm_backward(ptr(g_y), ptr(h), ptr(g_h), code(h), ptr<float>(mean),
                                    ptr<float>(rstd), ptr(w), code(w), T, C, ptr(g_x), ptr(g_w),
                                    g_b ? ptr(*g_b) : nullptr, ptr(ws), ws.numel(), on.stream));
  written({g_x_in});
  on.give({&g_x, &g_w, g_b ? &*g_b : nullptr});
  return tuple(wrap(g_x), wrap(g_w), g_b ? wrap(*g_b) : none());
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------ logits

// A matrix whose rows are packed, at any pitch (a slice of a padded
// vocabulary); returns the pitch.
int64_t pitch(const char* name, const Tensor& t) {
  if (t.dim() != 2)
    value_error("%s must be a 2-D tensor, got %s", name, text(t.sizes()).c_str());
  on_gpu(t);
  const int64_t T = t.size(0), V = t.size(1), ld = T > 1 ? t.stride(0) : V;
  if ((V > 1 && t.stride(1) != 1) || ld < V)
    value_error(
        "%s: the elements of a row must be contiguous and rows not overlap", name);
  return ld;
}

void same_device(const Tensor& like, const Tensor& t) {
  if (t.device() != like.device())
    value_error("tensors on different devices: %s and %s",
                            like.device().str().c_str(), t.device().str().c_str());
}

// (logits, targets, scale, stream) -> (logprob, stats)
PyObject* token_logprob_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 4);
  const Tensor& x = tensor("logits", a[0]);
  const Tensor& t = tensor("targets", a[1]);
  const double scale = number("scale", a[2]);
  const int64_t ld = pitch("logits", x), T = x.size(0);
  expect("targets", t, ScalarType::Long, {T});
  same_gpu(x, {&t});
  const Launch on(x, a[3]);
  on.use({&x, &t});
  const Tensor lp = make(x, ScalarType::Float, {T}), stats = make(x, ScalarType::Float, {T, 2});
  check("hlq_token_logprob_forward",
        lib.hlq_token_logprob_forward(ptr(x), code(x), ld, ptr<int64_t>(t), T, x.size(1), scale,
                                      ptr<float>(lp), ptr<float>(stats), on.stream));
  on.give({&lp, &stats});
  return tuple(wrap(lp), wrap(stats));
  END_HANDLE_TH_ERRORS
}

// (g_logprob, logits, targets, stats, scale, g_x, stream) -> g_x
PyObject* token_logprob_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 7);
  const Tensor& g = tensor("g_logprob", a[0]);
  const Tensor& x = tensor("logits", a[1]);
  const Tensor& t = tensor("targets", a[2]);
  const Tensor& stats = tensor("stats", a[3]);
  const double scale = number("scale", a[4]);
  const Tensor* g_x_in = maybe("g_x", a[5]);
  const int64_t ld = pitch("logits", x), T = x.size(0), V = x.size(1);
  expect("targets", t, ScalarType::Long, {T});
  expect("g_logprob", g, ScalarType::Float, {T});
  expect("stats", stats, ScalarType::Float, {T, 2});
  same_gpu(x, {&t, &g, &stats});
  if (g_x_in) expect("g_x", *g_x_in, x.scalar_type(), x.sizes());
  const Launch on(x, a[6]);
  on.use({&g, &x, &t, &stats, g_x_in});
  const Tensor g_x = g_x_in ? *g_x_in : make(x, x.scalar_type(), {T, V});
  const int64_t g_ld = pitch("g_x", g_x);
  same_device(x, g_x);
  check("hlq_token_logprob_backward",
        lib.hlq_token_logprob_backward(ptr<float>(g), ptr(x), code(x), ld, ptr<int64_t>(t),
                                       ptr<float>(stats), T, V, scale, ptr(g_x), g_ld,
                                       on.stream));
  written({g_x_in});
  on.give({&g_x});
  return wrap(g_x);
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------ losses

struct PolicyInputs {
  const Tensor *old, *advantage, *weight, *ref;
  PolicyInputs(PyObject* const* a)
      : old(&tensor("old_logprob", a[0])), advantage(&tensor("advantage", a[1])),
        weight(maybe("weight", a[2])), ref(maybe("ref_logprob", a[3])) {}
  void check(const Tensor& like, int64_t T) const {
    expect("old_logprob", *old, ScalarType::Float, {T});
    expect("advantage", *advantage, ScalarType::Float, {T});
    if (weight) expect("weight", *weight, ScalarType::Float, {T});
    if (ref) expect("ref_logprob", *ref, ScalarType::Float, {T});
    same_gpu(like, {old, advantage, weight, ref});
  }
};

// (logprob, old, advantage, weight, ref, clip_low, clip_high, kl_coef, workspace, stream)
//   -> (sums, g_logprob)
PyObject* policy_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  const Tensor& lp = tensor("logprob", a[0]);
  const PolicyInputs in(a + 1);
  const double lo = number("clip_low", a[5]), hi = number("clip_high", a[6]);
  const double kl = number("kl_coef", a[7]);
  const Tensor* ws_in = maybe("workspace", a[8]);
  const int64_t T = lp.numel();
  expect("logprob", lp, ScalarType::Float, {T});
  in.check(lp, T);
  same_gpu(lp, {&lp});
  const Launch on(lp, a[9]);
  on.use({&lp, in.old, in.advantage, in.weight, in.ref, ws_in});
  const Tensor sums = make(lp, ScalarType::Float, {3}), g = make(lp, ScalarType::Float, {T});
  const Tensor ws = workspace(ws_in, lib.hlq_policy_loss_workspace_size(T), lp);
  check("hlq_policy_loss",
        lib.hlq_policy_loss(ptr<float>(lp), ptr<float>(in.old), ptr<float>(in.advantage),
                            ptr<float>(in.weight), ptr<float>(in.ref), T, lo, hi, kl,
                            ptr<float>(sums), ptr<float>(g), ptr(ws), ws.numel(), on.stream));
  on.give({&sums, &g});
  return tuple(wrap(sums), wrap(g));
  END_HANDLE_TH_ERRORS
}

// (logits, targets, old, advantage, weight, ref, scale, clip_low, clip_high, kl_coef, g_x,
//  workspace, stream) -> (sums, logprob, g_x)
PyObject* policy_loss_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 13);
  const Tensor& x = tensor("logits", a[0]);
  const Tensor& t = tensor("targets", a[1]);
  const PolicyInputs in(a + 2);
  const double scale = number("scale", a[6]);
  const double lo = number("clip_low", a[7]), hi = number("clip_high", a[8]);
  const double kl = number("kl_coef", a[9]);
  const Tensor* g_x_in = maybe("g_x", a[10]);
  const Tensor* ws_in = maybe("workspace", a[11]);
  const int64_t ld = pitch("logits", x), T = x.size(0), V = x.size(1);
  expect("targets", t, ScalarType::Long, {T});
  in.check(x, T);
  same_gpu(x, {&t});
  if (g_x_in) expect("g_x", *g_x_in, x.scalar_type(), x.sizes());
  const Launch on(x, a[12]);
  on.use({&x, &t, in.old, in.advantage, in.weight, in.ref, g_x_in, ws_in});
  const Tensor g_x = g_x_in ? *g_x_in : make(x, x.scalar_type(), {T, V});
  const int64_t g_ld = pitch("g_x", g_x);
  same_device(x, g_x);
  const Tensor sums = make(x, ScalarType::Float, {3}), lp = make(x, ScalarType::Float, {T});
  const Tensor ws = workspace(ws_in, lib.hlq_policy_loss_workspace_size(T), x);
  check("hlq_policy_loss_logits",
        lib.hlq_policy_loss_logits(ptr(x), code(x), ld, ptr<int64_t>(t), ptr<float>(in.old),
                                   ptr<float>(in.advantage), ptr<float>(in.weight),
                                   ptr<float>(in.ref), T, V, scale, lo, hi, kl, ptr<float>(sums),
                                   ptr<float>(lp), ptr(g_x), g_ld, ptr(ws), ws.numel(),
                                   on.stream));
  written({g_x_in});
  on.give({&sums, &lp, &g_x});
  return tuple(wrap(sums), wrap(lp), wrap(g_x));
  END_HANDLE_TH_ERRORS
}

// (logprob, start, beta, ref, weight, label_smoothing, reduction, workspace, stream)
//   -> (loss, margin, g_logprob)
PyObject* preference_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  const Tensor& lp = tensor("logprob", a[0]);
  const Tensor& start = tensor("start", a[1]);
  const double beta = number("beta", a[2]);
  const Tensor* ref = maybe("ref_logprob", a[3]);
  const Tensor* w = maybe("weight", a[4]);
  const double e = number("label_smoothing", a[5]);
  const int reduction = integer("reduction", a[6]);
  const Tensor* ws_in = maybe("workspace", a[7]);
  const int64_t T = lp.numel();
  expect("logprob", lp, ScalarType::Float, {T});
  if (ref) expect("ref_logprob", *ref, ScalarType::Float, {T});
  if (w) expect("weight", *w, ScalarType::Float, {T});
  if (start.scalar_type() != ScalarType::Long || start.dim() != 1 || start.numel() % 2 != 1)
    value_error("start must be an int64 tensor of 2P + 1 bounds");
  const int64_t P = start.numel() / 2;
  same_gpu(lp, {&lp, ref, w, &start});
  const Launch on(lp, a[8]);
  on.use({&lp, ref, w, &start, ws_in});
  const Tensor loss = make(lp, ScalarType::Float, {1}), margin = make(lp, ScalarType::Float, {P});
  const Tensor g = make(lp, ScalarType::Float, {T});
  const Tensor ws = workspace(ws_in, lib.hlq_preference_loss_workspace_size(P), lp);
  check("hlq_preference_loss",
        lib.hlq_preference_loss(ptr<float>(lp), ptr<float>(ref), ptr<float>(w),
                                ptr<int64_t>(start), P, T, beta, e, reduction,
                                ptr<float>(loss), ptr<float>(margin), ptr<float>(g), ptr(ws),
                                ws.numel(), on.stream));
  on.give({&loss, &margin, &g});
  return tuple(wrap(loss), wrap(margin), wrap(g));
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------ clipping

// A list or tuple of the items of o, released at the end of the call.
struct Items {
  PyObject* seq;
  explicit Items(PyObject* o) : seq(PySequence_Fast(o, "expected a list of tensors")) {
    if (!seq) throw python_error();
  }
  ~Items() { Py_XDECREF(seq); }
  Items(const Items&) = delete;
  Items& operator=(const Items&) = delete;
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

// (grads, max_norm, norm_kind, out, workspace, stream, device) -> norm
PyObject* clip_grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 7);
  const Items grads(a[0]);
  const double max_norm = number("max_norm", a[1]);
  const int kind = integer("norm_kind", a[2]);
  const bool in_place = a[3] == Py_None;
  const Items outs(in_place ? grads.seq : a[3]);
  const Tensor* ws_in = maybe("workspace", a[4]);
  const Py_ssize_t N = grads.size();
  if (outs.size() != N)
    value_error("%zd gradients and %zd outputs", N, outs.size());
  std::vector<const void*> src(N);
  std::vector<void*> dst(N);
  std::vector<int64_t> sizes(N);
  std::vector<int> types(N);
  const at::Device device = N ? tensor("grads", grads[0]).device()
                              : at::Device(at::kCUDA, (c10::DeviceIndex)integer("device", a[6]));
  for (Py_ssize_t i = 0; i < N; ++i) {
    const Tensor& g = tensor("grads", grads[i]);
    if (!g.is_cuda() || g.device() != device)
      value_error("gradient %zd is on %s, expected one GPU for all", i,
                              g.device().str().c_str());
    if (!g.is_non_overlapping_and_dense())
      value_error("gradient %zd is not dense", i);
    src[i] = g.data_ptr();
    sizes[i] = g.numel();
    types[i] = code(g);
    if (!in_place) {
      const Tensor& o = tensor("out", outs[i]);
      if (o.scalar_type() != g.scalar_type() || o.device() != device || o.sizes() != g.sizes() ||
          o.strides() != g.strides())
        value_error("output %zd must match its gradient's type, shape and strides", i);
      dst[i] = o.data_ptr();
    }
  }
  const Launch on(device, a[5]);
  for (Py_ssize_t i = 0; i < N && on.other; ++i) {
    on.use(THPVariable_Unpack(grads[i]));
    if (!in_place) on.use(THPVariable_Unpack(outs[i]));
  }
  on.use({ws_in});
  const Tensor norm = make(device, ScalarType::Double, {1});
  const Tensor ws =
      workspace(ws_in, lib.hlq_clip_grad_norm_workspace_size(sizes.data(), N), norm);
  check("hlq_clip_grad_norm",
        lib.hlq_clip_grad_norm(src.data(), in_place ? nullptr : dst.data(), sizes.data(),
                               types.data(), N, max_norm, kind, ptr<double>(norm), ptr(ws),
                               ws.numel(), on.stream));
  for (Py_ssize_t i = 0; i < N; ++i) written(THPVariable_Unpack((in_place ? grads : outs)[i]));
  on.give({&norm});
  return wrap(norm);
  END_HANDLE_TH_ERRORS
}

// (handle of the loaded library, hlq._check)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 2);
  void* handle = PyLong_AsVoidPtr(a[0]);
  if (PyErr_Occurred()) throw python_error();
#define F(name)                                                                        \
  lib.name = reinterpret_cast<decltype(lib.name)>(dlsym(handle, #name));               \
  if (!lib.name) value_error("the library does not export %s", #name);
  HLQ_FUNCTIONS(F)
#undef F
  Py_INCREF(a[1]);
  Py_XDECREF(g_check);
  g_check = a[1];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define HLQ_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {HLQ_METHOD(bind),
                         HLQ_METHOD(layer_norm_forward),
                         HLQ_METHOD(layer_norm_backward),
                         HLQ_METHOD(token_logprob_forward),
                         HLQ_METHOD(token_logprob_backward),
                         HLQ_METHOD(policy_loss),
                         HLQ_METHOD(policy_loss_logits),
                         HLQ_METHOD(preference_loss),
                         HLQ_METHOD(clip_grad_norm),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hlq_torch", nullptr, -1, methods,
                      nullptr,               nullptr,      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hlq_torch() { return PyModule_Create(&module); }
