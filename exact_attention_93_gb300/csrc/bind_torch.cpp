// bind_torch.cpp -- the Python entry to include/fattn_cache.h and
// include/fattn_decoder.h: checks torch tensors, allocates the results and calls the
// C ABI of libfattn.so.
//
// These calls are made for every layer and token while generating, when the
// kernels take a few microseconds: the same marshalling written in Python over
// ctypes cost 15 to 30 us a call on the host of a GB300.  Arguments are
// positional; rotary.py, kvcache.py and attention.py hold the public signatures
// and their documentation.  Each function returns its tensors, or the
// fa_status of a refused call as an int.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/Context.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/record_function.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <climits>
#include <cstring>
#include <exception>
#include <optional>
#include <string>
#include <vector>

#include "fattn_decoder.h"

namespace {

// Raised as the Python exception of the given type.  (A std::exception, so that autograd's
// own threads hand it on as well.)
struct Refuse : std::exception {
  Refuse(PyObject* t, const char* w) : type(t), text(w) {}
  const char* what() const noexcept override { return text; }
  PyObject* type;
  const char* text;
};

[[noreturn]] void refuse(const char* what) { throw Refuse{PyExc_ValueError, what}; }

void need(bool ok, const char* what) {
  if (!ok) refuse(what);
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Refuse{PyExc_TypeError, what};
  return THPVariable_Unpack(o);
}

// None gives an undefined tensor.
at::Tensor maybe(PyObject* o, const char* what) {
  return o == Py_None ? at::Tensor() : tensor(o, what);
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

int elem(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return FA_ELEM_BF16;
    case at::kHalf: return FA_ELEM_FP16;
    case at::kFloat: return FA_ELEM_FP32;
    case at::kFloat8_e4m3fn: return FA_ELEM_E4M3;
    default: throw Refuse{PyExc_TypeError, "unsupported dtype"};
  }
}

// Makes the tensors' device the current one for a call, if it is not already.
class Device {
 public:
  explicit Device(std::initializer_list<const at::Tensor*> ts) {
    const c10::Device d = (*ts.begin())->device();
    for (const at::Tensor* t : ts)
      need(!t->defined() || (t->is_cuda() && t->device() == d),
           "libfattn takes CUDA tensors of one device only");
    index_ = d.index();
    if (c10::cuda::current_device() != index_) guard_.emplace(d);
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(index_).stream(); }

 private:
  c10::DeviceIndex index_;
  std::optional<c10::cuda::CUDAGuard> guard_;
};

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

PyObject* pair(at::Tensor a, at::Tensor b) {
  THPObjectPtr x(wrap(std::move(a))), y(wrap(std::move(b)));
  return PyTuple_Pack(2, x.get(), y.get());
}

PyObject* status(fa_status s) { return PyLong_FromLong(static_cast<long>(s)); }

// Whether anyone behind torch's dispatcher wants a part in an allocation: deterministic
// algorithms, which fill what is not initialised, dispatch modes and transforms, or the profiler.
bool dispatched() {
  const at::Context& context = at::globalContext();
  return (context.deterministicAlgorithms() && context.deterministicFillUninitializedMemory()) ||
         !(c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set).empty() ||
         at::getStepCallbacksUnlessEmpty(at::RecordScope::FUNCTION).has_value();
}

// An uninitialised tensor on x's device.  (What at::empty comes to behind its dispatcher,
// which costs a third of the 1.8 us that an allocation takes through it.)
at::Tensor make(const at::Tensor& x, at::IntArrayRef sizes, at::ScalarType type) {
  if (dispatched()) return at::empty(sizes, at::TensorOptions().dtype(type).device(x.device()));
  return at::Tensor(at::detail::empty_cuda(sizes, type, x.device(), std::nullopt));
}

at::Tensor like(const at::Tensor& x) { return make(x, x.sizes(), x.scalar_type()); }

// Forward-mode differentiation gives a tensor a tangent whether or not it needs a
// gradient; none of these calls makes one for its results.
void no_tangent(const at::Tensor& t) {
  TORCH_CHECK_NOT_IMPLEMENTED(
      !t.defined() || !c10::AutogradState::get_tls_state().get_fw_grad_mode() ||
          !t._fw_grad(/*level=*/0).defined(),
      "forward-mode differentiation is not supported: the tangent would be lost");
}

void no_grad(const at::Tensor& t, const char* what) {
  no_tangent(t);
  need(!(t.defined() && t.requires_grad() && c10::GradMode::is_enabled()), what);
}

// What torch's own in-place operations do: autograd then notices that a tensor it
// saved has changed.
void written(const at::Tensor& t) {
  if (t.defined()) t.unsafeGetTensorImpl()->bump_version();
}

fa_rotary_operand rotary_operand(const at::Tensor& x, const at::Tensor& y) {
  const auto xs = x.strides(), ys = y.strides();
  need(xs.back() == 1 && ys.back() == 1, "the head dimension D must be contiguous");
  fa_rotary_operand o;
  o.x = x.const_data_ptr();
  o.y = y.data_ptr();
  if (x.dim() == 4) {
    o.heads = static_cast<int>(x.size(2));
    o.xs = fa_strides{xs[0], xs[2], xs[1]};
    o.ys = fa_strides{ys[0], ys[2], ys[1]};
  } else {
    o.heads = static_cast<int>(x.size(1));
    o.xs = fa_strides{0, xs[1], xs[0]};
    o.ys = fa_strides{0, ys[1], ys[0]};
  }
  return o;
}

// How a rotation is done, apart from the tensors turned.
struct Rotation {
  at::Tensor freq, pos;  // pos may be undefined
  double magnitude;
  bool interleaved, inverse;
  std::string axis;  // of each pair; empty: one axis, and pos without a dimension for it
  int axes = 1;

  // Of (b, n) of x's tokens.
  fa_positions positions() const {
    fa_positions p{nullptr, 0, axes, 0, 0, reinterpret_cast<const unsigned char*>(axis.data())};
    if (!pos.defined() || pos.numel() == 0) return p;  // (no tokens: no address either)
    const int64_t lead = axis.empty() ? 0 : 1;
    p.positions = pos.const_data_ptr();
    p.bits = pos.scalar_type() == at::kInt ? 32 : 64;
    p.axis_stride = lead ? pos.stride(0) : 0;
    p.batch_stride = pos.dim() == lead + 2 ? pos.stride(lead) : 0;
    return p;
  }
  // (as one entry: each costs some 0.3 us each way)
  void save(torch::autograd::AutogradContext* ctx) const {
    ctx->saved_data["rotation"] = std::vector<double>{
        magnitude, static_cast<double>(interleaved), static_cast<double>(inverse),
        static_cast<double>(axes)};
    if (!axis.empty()) ctx->saved_data["axis"] = axis;
  }
  static Rotation saved(torch::autograd::AutogradContext* ctx, const at::Tensor& freq,
                        const at::Tensor& pos) {
    const auto v = ctx->saved_data["rotation"].toDoubleVector();
    const auto axis = ctx->saved_data.find("axis");
    return Rotation{freq,
                    pos,
                    v[0],
                    v[1] != 0.0,
                    v[2] != 0.0,
                    axis == ctx->saved_data.end() ? std::string() : axis->second.toStringRef(),
                    static_cast<int>(v[3])};
  }
};

// sections (None, or how many pairs each axis gets) and their order as the axis of
// each of `pairs` pairs.
void read_sections(PyObject* sections, PyObject* order, int64_t pairs, Rotation& r) {
  const char* name = PyUnicode_Check(order) ? PyUnicode_AsUTF8(order) : nullptr;
  const bool turns = name && !std::strcmp(name, "turns");
  need(turns || (name && !std::strcmp(name, "blocks")),
       "section_order must be \"blocks\" or \"turns\"");
  if (sections == Py_None) return;
  THPObjectPtr items(PySequence_Fast(sections, "sections must be a sequence of integers"));
  if (!items) throw python_error();
  const Py_ssize_t axes = PySequence_Fast_GET_SIZE(items.get());
  need(axes >= 1 && axes <= 8, "sections must name 1 to 8 axes");
  int64_t left[8], all = 0;
  for (Py_ssize_t i = 0; i < axes; ++i) {
    left[i] = integer(PySequence_Fast_GET_ITEM(items.get(), i));
    need(left[i] >= 0 && left[i] <= pairs, "sections must add up to the pairs of inv_freq");
    all += left[i];
  }
  need(all == pairs && pairs > 0, "sections must add up to the pairs of inv_freq");
  r.axes = static_cast<int>(axes);
  while (static_cast<int64_t>(r.axis.size()) < pairs)
    for (Py_ssize_t i = 0; i < axes; ++i) {  // a round: all of an axis, or one of each
      const int64_t n = turns ? std::min<int64_t>(left[i], 1) : left[i];
      r.axis.append(static_cast<size_t>(n), static_cast<char>(i));
      left[i] -= n;
    }
}

// Turns x into y, and x2 (when defined) into y2.
fa_status turn(const at::Tensor& x, const at::Tensor& y, const at::Tensor& x2,
               const at::Tensor& y2, const Rotation& r, const Device& device) {
  const int64_t dim = x.dim(), B = dim == 4 ? x.size(0) : 1, N = x.size(dim - 3);
  need(B <= INT_MAX && N <= INT_MAX, "tensors too large");
  const fa_rotary_operand a = rotary_operand(x, y);
  fa_rotary_operand b;
  if (x2.defined()) b = rotary_operand(x2, y2);
  const fa_positions pos = r.positions();
  return fa_rotary_axes(&a, x2.defined() ? &b : nullptr, static_cast<int>(B), static_cast<int>(N),
                        static_cast<int>(x.size(dim - 1)), static_cast<int>(2 * r.freq.size(0)),
                        r.freq.const_data_ptr<double>(), &pos, static_cast<float>(r.magnitude),
                        r.interleaved, r.inverse, static_cast<fa_elem>(elem(x.scalar_type())),
                        device.stream());
}

// What the C ABI refuses inside autograd.
void check(fa_status st, const char* what = "fa_rotary") {
  TORCH_CHECK(st == FA_OK, what, " failed: ", fa_status_string(st), " (", static_cast<int>(st),
              ")");
}

// The incoming gradient as the kernels need it: D contiguous, 16-byte aligned
// rows.  Anything else is copied once (a contiguous one too, where it begins at an
// odd address: contiguous() would return it as it is).
at::Tensor grad_operand(const at::Tensor& g) {
  if (!g.defined()) return g;
  bool ok = g.stride(-1) == 1 && reinterpret_cast<uintptr_t>(g.const_data_ptr()) % 16 == 0;
  for (int64_t i = 0; i + 1 < g.dim(); ++i) ok = ok && g.stride(i) % 8 == 0;
  return ok ? g : g.clone(at::MemoryFormat::Contiguous);
}

// A rotation's gradient is the rotation back, with the same magnitude; it is
// linear, so its own gradient is a rotation again.  kTensors: one or two tensors
// turned (autograd takes no undefined ones).
template <int kTensors>
struct RotaryFunction : torch::autograd::Function<RotaryFunction<kTensors>> {
  static torch::autograd::variable_list run(torch::autograd::AutogradContext* ctx,
                                            const at::Tensor& q, const at::Tensor& k,
                                            const Rotation& r) {
    ctx->set_materialize_grads(false);
    ctx->save_for_backward({r.freq, r.pos});
    r.save(ctx);
    return rotated(q, k, r);
  }
  static torch::autograd::variable_list forward(torch::autograd::AutogradContext* ctx,
                                                const at::Tensor& q, const Rotation& r) {
    return run(ctx, q, at::Tensor(), r);
  }
  static torch::autograd::variable_list forward(torch::autograd::AutogradContext* ctx,
                                                const at::Tensor& q, const at::Tensor& k,
                                                const Rotation& r) {
    return run(ctx, q, k, r);
  }
  static torch::autograd::variable_list rotated(const at::Tensor& q, const at::Tensor& k,
                                                const Rotation& r) {
    const Device device({&q, &k, &r.freq, &r.pos});
    const at::Tensor yq = like(q), yk = k.defined() ? like(k) : k;
    check(turn(q, yq, k, yk, r, device));
    if (!k.defined()) return {yq};
    return {yq, yk};
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads);
};

template <int kTensors>
torch::autograd::variable_list RotaryFunction<kTensors>::backward(
    torch::autograd::AutogradContext* ctx, torch::autograd::variable_list grads) {
  const auto saved = ctx->get_saved_variables();
  Rotation r = Rotation::saved(ctx, saved[0], saved[1]);
  r.inverse = !r.inverse;
  std::vector<at::Tensor> have;
  for (const at::Tensor& g : grads)
    if (g.defined()) have.push_back(grad_operand(g));
  torch::autograd::variable_list out(kTensors + 1), got;
  if (have.empty()) return out;
  for (const at::Tensor& g : have) no_tangent(g);
  if (c10::GradMode::is_enabled())
    got = have.size() == 1 ? RotaryFunction<1>::apply(have[0], r)
                           : RotaryFunction<2>::apply(have[0], have[1], r);
  else
    got = rotated(have[0], have.size() == 1 ? at::Tensor() : have[1], r);
  for (size_t i = 0, n = 0; i < grads.size(); ++i)
    if (grads[i].defined()) out[i] = got[n++];
  return out;
}

// Checks q, k (may be undefined) and how they are turned, the latter from the
// arguments inv_freq, positions, magnitude, interleaved, sections and section_order.
Rotation rotation(const at::Tensor& q, const at::Tensor& k, PyObject* freq, PyObject* positions,
                  PyObject* magnitude, PyObject* interleaved, PyObject* sections,
                  PyObject* order) {
  Rotation r{tensor(freq, "inv_freq must be a tensor"),
             maybe(positions, "positions must be a tensor or None"), number(magnitude),
             truth(interleaved), false, {}, 1};
  const int64_t dim = q.dim();
  need(dim == 3 || dim == 4,
       "expected (batch, seqlen, nheads, headdim) or packed (total, nheads, headdim) tensors");
  if (k.defined())
    need(k.dim() == dim && k.size(0) == q.size(0) && (dim == 3 || k.size(1) == q.size(1)) &&
             k.size(dim - 1) == q.size(dim - 1) && k.scalar_type() == q.scalar_type(),
         "q and k must agree in type and in every dimension but the heads");
  need(r.freq.scalar_type() == at::kDouble && r.freq.dim() == 1 && r.freq.is_contiguous(),
       "inv_freq must be a contiguous float64 (rotary_dim / 2) tensor");
  read_sections(sections, order, r.freq.size(0), r);
  const int64_t B = dim == 4 ? q.size(0) : 1, N = q.size(dim - 3), lead = r.axis.empty() ? 0 : 1;
  need(!lead || r.pos.defined(), "sections need positions");
  if (r.pos.defined()) {
    if (r.pos.scalar_type() != at::kInt && r.pos.scalar_type() != at::kLong)
      throw Refuse{PyExc_TypeError, "positions must be int32 or int64"};
    const int64_t rest = r.pos.dim() - lead;
    const bool fits = (rest == 1 && r.pos.size(lead) == N) ||
                      (dim == 4 && rest == 2 && r.pos.size(lead) == B && r.pos.size(lead + 1) == N);
    if (lead)
      need(fits && r.pos.size(0) == r.axes,
           "with sections, positions must have shape (axes, seqlen) or (axes, batch, seqlen)");
    else
      need(fits, "positions must have shape (seqlen,) or (batch, seqlen)");
  }
  need(!r.freq.requires_grad(), "inv_freq gets no gradient: detach it");
  if (r.pos.defined() && N > 1 && r.pos.stride(-1) != 1) r.pos = r.pos.contiguous();
  return r;
}

bool wants_grad(const at::Tensor& t) { return t.defined() && t.requires_grad(); }

void apart(const at::Tensor& q, const at::Tensor& k) {
  need(!k.defined() || k.numel() == 0 || k.const_data_ptr() != q.const_data_ptr(),
       "q and k would be written over each other");
}

// rotary(q, k, inv_freq, positions, magnitude, interleaved, inplace, sections, order)
PyObject* rotary(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q must be a tensor");
  const at::Tensor k = maybe(a[1], "k must be a tensor or None");
  const Rotation r = rotation(q, k, a[2], a[3], a[4], a[5], a[7], a[8]);
  const bool inplace = truth(a[6]);
  for (const at::Tensor* t : {&q, &k, &r.freq}) no_tangent(*t);
  const Device device({&q, &k, &r.freq, &r.pos});
  if (c10::GradMode::is_enabled() && (wants_grad(q) || wants_grad(k))) {
    need(!inplace, "inplace=True would overwrite tensors that need a gradient");
    auto y = k.defined() ? RotaryFunction<2>::apply(q, k, r) : RotaryFunction<1>::apply(q, r);
    return k.defined() ? pair(std::move(y[0]), std::move(y[1])) : wrap(std::move(y[0]));
  }
  const at::Tensor yq = inplace ? q : like(q), yk = !k.defined() || inplace ? k : like(k);
  if (inplace) {
    apart(q, k);
    written(q);
    written(k);
  }
  const fa_status st = turn(q, yq, k, yk, r, device);
  if (st != FA_OK) return status(st);
  return k.defined() ? pair(yq, yk) : wrap(yq);
}

// Norm and rotation of one or two tensors.  Undefined tensors stand for what is absent;
// autograd takes none, and gets empty ones instead.
struct Norm {
  Rotation r;
  double eps;
  bool grad_wq, grad_wk;  // weights that need a gradient
};

at::Tensor present(const at::Tensor& t, const at::Tensor& like) {
  return t.defined() ? t : make(like, {0}, like.scalar_type());
}

at::Tensor absent(const at::Tensor& t) { return t.dim() == 1 && t.size(0) == 0 ? at::Tensor() : t; }

fa_elem weight_elem(const at::Tensor& x, const at::Tensor& wq, const at::Tensor& wk) {
  const at::Tensor& w = wq.defined() ? wq : wk;
  return static_cast<fa_elem>(elem((w.defined() ? w : x).scalar_type()));
}

const void* address(const at::Tensor& t) { return t.defined() ? t.const_data_ptr() : nullptr; }

// A weight as the library takes it, on 8 bytes: a view into a buffer of many parameters,
// which may lie anywhere, is copied.
at::Tensor weight_operand(const at::Tensor& w) {
  const bool ok = reinterpret_cast<uintptr_t>(address(w)) % 8 == 0;
  return ok ? w : w.clone();
}

fa_status normed(const at::Tensor& q, const at::Tensor& yq, const at::Tensor& k,
                 const at::Tensor& yk, const at::Tensor& weight_q, const at::Tensor& weight_k,
                 const Norm& n, const Device& device) {
  const at::Tensor wq = weight_operand(weight_q), wk = weight_operand(weight_k);
  const int64_t dim = q.dim(), B = dim == 4 ? q.size(0) : 1, N = q.size(dim - 3);
  need(B <= INT_MAX && N <= INT_MAX, "tensors too large");
  const fa_rotary_operand a = rotary_operand(q, yq);
  fa_rotary_operand b;
  if (k.defined()) b = rotary_operand(k, yk);
  const fa_positions pos = n.r.positions();
  return fa_qk_norm_rotary(&a, k.defined() ? &b : nullptr, address(wq), address(wk),
                           weight_elem(q, wq, wk), static_cast<float>(n.eps), static_cast<int>(B),
                           static_cast<int>(N), static_cast<int>(q.size(dim - 1)),
                           static_cast<int>(2 * n.r.freq.size(0)),
                           n.r.freq.const_data_ptr<double>(), &pos,
                           static_cast<float>(n.r.magnitude), n.r.interleaved,
                           static_cast<fa_elem>(elem(q.scalar_type())), device.stream());
}

// The gradients of x and of its weight (undefined where not wanted), for one or two
// tensors x with the gradients g of their results.
struct NormOperand {
  at::Tensor x, g, w, dx, dw;
};

void norm_gradients(std::vector<NormOperand>& ops, const Norm& n) {
  const at::Tensor none;
  const bool two = ops.size() > 1;
  NormOperand &a = ops[0], &b = ops[two ? 1 : 0];
  const Device device({&a.x, &a.g, &a.w, two ? &b.x : &none, two ? &b.g : &none,
                       two ? &b.w : &none, &n.r.freq, &n.r.pos});
  fa_rotary_operand o[2];
  fa_strides gs[2] = {};
  for (size_t i = 0; i < ops.size(); ++i) {
    ops[i].g = grad_operand(ops[i].g);
    ops[i].w = weight_operand(ops[i].w);
    ops[i].dx = like(ops[i].x);
    o[i] = rotary_operand(ops[i].x, ops[i].dx);
    gs[i] = rotary_operand(ops[i].g, ops[i].dx).xs;
  }
  const at::Tensor& x = a.x;
  const int64_t dim = x.dim(), B = dim == 4 ? x.size(0) : 1, N = x.size(dim - 3), D = x.size(dim - 1);
  size_t bytes = 0;
  check(fa_qk_norm_rotary_bwd_workspace_size(static_cast<int>(D), &bytes), "fa_qk_norm_rotary_bwd");
  const at::Tensor ws = make(x, {static_cast<int64_t>(bytes)}, at::kByte);
  const fa_positions pos = n.r.positions();
  check(fa_qk_norm_rotary_bwd(
            &o[0], two ? &o[1] : nullptr, a.g.const_data_ptr(), gs[0],
            two ? b.g.const_data_ptr() : nullptr, gs[1], address(a.w),
            two ? address(b.w) : nullptr, a.dw.defined() ? a.dw.data_ptr() : nullptr,
            two && b.dw.defined() ? b.dw.data_ptr() : nullptr,
            weight_elem(x, a.w, two ? b.w : none), static_cast<float>(n.eps), static_cast<int>(B),
            static_cast<int>(N), static_cast<int>(D), static_cast<int>(2 * n.r.freq.size(0)),
            n.r.freq.const_data_ptr<double>(), &pos, static_cast<float>(n.r.magnitude),
            n.r.interleaved, static_cast<fa_elem>(elem(x.scalar_type())), ws.data_ptr(), bytes,
            device.stream()),
        "fa_qk_norm_rotary_bwd");
}

// (dq, dk, dq_weight, dk_weight), undefined where there is nothing.
torch::autograd::variable_list norm_backward(const at::Tensor& gq, const at::Tensor& gk,
                                             const at::Tensor& q, const at::Tensor& k,
                                             const at::Tensor& wq, const at::Tensor& wk,
                                             const Norm& n) {
  std::vector<NormOperand> ops;
  if (gq.defined()) ops.push_back({q, gq, wq, {}, n.grad_wq ? like(wq) : at::Tensor()});
  if (gk.defined()) ops.push_back({k, gk, wk, {}, n.grad_wk ? like(wk) : at::Tensor()});
  torch::autograd::variable_list out(4);
  if (ops.empty()) return out;
  norm_gradients(ops, n);
  size_t i = 0;
  if (gq.defined()) {
    out[0] = ops[i].dx;
    out[2] = ops[i++].dw;
  }
  if (gk.defined()) {
    out[1] = ops[i].dx;
    out[3] = ops[i].dw;
  }
  return out;
}

// The gradients as a function of their own, which has none: differentiating twice is
// an error instead of a wrong result.
struct NormGradient : torch::autograd::Function<NormGradient> {
  static torch::autograd::variable_list forward(torch::autograd::AutogradContext*,
                                                const at::Tensor& gq, const at::Tensor& gk,
                                                const at::Tensor& q, const at::Tensor& k,
                                                const at::Tensor& wq, const at::Tensor& wk,
                                                const Norm& n) {
    auto out = norm_backward(absent(gq), absent(gk), q, absent(k), absent(wq), absent(wk), n);
    for (at::Tensor& t : out) t = present(t, q);
    return out;
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext*,
                                                 torch::autograd::variable_list) {
    TORCH_CHECK_NOT_IMPLEMENTED(false,
                                "qk_norm_rotary_func is differentiable once: its gradients have "
                                "none of their own");
  }
};

struct NormFunction : torch::autograd::Function<NormFunction> {
  static torch::autograd::variable_list forward(torch::autograd::AutogradContext* ctx,
                                                const at::Tensor& q, const at::Tensor& k,
                                                const at::Tensor& wq, const at::Tensor& wk,
                                                const Norm& n) {
    ctx->set_materialize_grads(false);
    ctx->save_for_backward({n.r.freq, n.r.pos, q, k, wq, wk});
    n.r.save(ctx);
    ctx->saved_data["norm"] = std::vector<double>{n.eps, static_cast<double>(n.grad_wq),
                                                  static_cast<double>(n.grad_wk)};
    const at::Tensor k2 = absent(k), w1 = absent(wq), w2 = absent(wk);
    const Device device({&q, &k2, &w1, &w2, &n.r.freq, &n.r.pos});
    const at::Tensor yq = like(q), yk = k2.defined() ? like(k2) : k2;
    check(normed(q, yq, k2, yk, w1, w2, n, device), "fa_qk_norm_rotary");
    if (!k2.defined()) return {yq};
    return {yq, yk};
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    const auto saved = ctx->get_saved_variables();
    const auto v = ctx->saved_data["norm"].toDoubleVector();
    const Norm n{Rotation::saved(ctx, saved[0], saved[1]), v[0], v[1] != 0.0, v[2] != 0.0};
    const at::Tensor gq = grads[0], gk = grads.size() > 1 ? grads[1] : at::Tensor();
    const at::Tensor &q = saved[2], &k = saved[3], &wq = saved[4], &wk = saved[5];
    for (const at::Tensor& g : {gq, gk}) no_tangent(g);
    torch::autograd::variable_list out(5);
    if (!gq.defined() && !gk.defined()) return out;
    auto got = c10::GradMode::is_enabled()
                   ? NormGradient::apply(present(gq, q), present(gk, q), q, k, wq, wk, n)
                   : norm_backward(gq, gk, q, absent(k), absent(wq), absent(wk), n);
    for (size_t i = 0; i < got.size(); ++i)
      if (got[i].defined()) out[i] = absent(got[i]);
    return out;
  }
};

// norm_rotary(q, k, q_weight, k_weight, inv_freq, positions, eps, magnitude, interleaved,
//             inplace, sections, order)
PyObject* norm_rotary(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q must be a tensor");
  const at::Tensor k = maybe(a[1], "k must be a tensor or None"),
                   wq = maybe(a[2], "q_weight must be a tensor or None"),
                   wk = maybe(a[3], "k_weight must be a tensor or None");
  Norm n{rotation(q, k, a[4], a[5], a[7], a[8], a[10], a[11]), number(a[6]), wants_grad(wq),
         wants_grad(wk)};
  const bool inplace = truth(a[9]);
  need(k.defined() || !wk.defined(), "k_weight belongs to k");
  for (const at::Tensor* w : {&wq, &wk})
    if (w->defined())
      need(w->dim() == 1 && w->size(0) == q.size(-1) && w->is_contiguous() &&
               (w->scalar_type() == q.scalar_type() || w->scalar_type() == at::kFloat),
           "weights must be contiguous (headdim,) tensors of q's type or float32");
  need(!wq.defined() || !wk.defined() || wq.scalar_type() == wk.scalar_type(),
       "q_weight and k_weight must be of one type");
  for (const at::Tensor* t : {&q, &k, &wq, &wk, static_cast<const at::Tensor*>(&n.r.freq)})
    no_tangent(*t);
  const Device device({&q, &k, &wq, &wk, &n.r.freq, &n.r.pos});
  if (c10::GradMode::is_enabled() &&
      (wants_grad(q) || wants_grad(k) || wants_grad(wq) || wants_grad(wk))) {
    need(!inplace, "inplace=True would overwrite what the gradients need");
    auto y = NormFunction::apply(q, present(k, q), present(wq, q), present(wk, q), n);
    return k.defined() ? pair(std::move(y[0]), std::move(y[1])) : wrap(std::move(y[0]));
  }
  const at::Tensor yq = inplace ? q : like(q), yk = !k.defined() || inplace ? k : like(k);
  if (inplace) {
    apart(q, k);
    written(q);
    written(k);
  }
  const fa_status st = normed(q, yq, k, yk, wq, wk, n, device);
  if (st != FA_OK) return status(st);
  return k.defined() ? pair(yq, yk) : wrap(yq);
}

fa_kv_pages kv_pages(const at::Tensor& k, const at::Tensor& v, const at::Tensor& ke,
                     const at::Tensor& ve) {
  need(k.dim() == 4 && v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type(),
       "k_pages and v_pages must be (pages, page_size, heads, D) tensors of one shape and type");
  const auto ks = k.strides(), vs = v.strides();
  need(ks[3] == 1 && vs[3] == 1, "the head dimension D must be contiguous");
  fa_kv_pages c{};
  c.type = elem(k.scalar_type());
  if (c.type == FA_ELEM_E4M3) {
    for (const at::Tensor* e : {&ke, &ve})
      need(e->defined() && e->scalar_type() == at::kByte && e->dim() == 3 &&
               e->size(0) == k.size(0) && e->size(1) == k.size(2) && e->size(2) == k.size(1) &&
               e->is_contiguous(),
           "an e4m3 cache needs k_exp and v_exp: contiguous uint8 (pages, heads, page_size) "
           "tensors");
    c.k_exp = static_cast<unsigned char*>(ke.data_ptr());
    c.v_exp = static_cast<unsigned char*>(ve.data_ptr());
  } else {
    need(!ke.defined() && !ve.defined(), "k_exp and v_exp belong to an e4m3 cache");
  }
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.k_page = ks[0];
  c.k_token = ks[1];
  c.k_head = ks[2];
  c.v_page = vs[0];
  c.v_token = vs[1];
  c.v_head = vs[2];
  need(k.size(0) <= INT_MAX && k.size(2) <= INT_MAX, "the cache is too large");
  c.pages = static_cast<int>(k.size(0));
  c.page_size = static_cast<int>(std::min<int64_t>(k.size(1), INT_MAX));
  c.heads = static_cast<int>(k.size(2));
  c.head_dim = static_cast<int>(std::min<int64_t>(k.size(3), INT_MAX));
  return c;
}

fa_ragged ragged(const at::Tensor& table, const at::Tensor& cu, const at::Tensor& lens,
                 int64_t total) {
  need(table.dim() == 2 && table.scalar_type() == at::kInt &&
           (table.size(1) <= 1 || table.stride(1) == 1),
       "block_table must be an int32 (batch, max_pages) tensor with contiguous rows");
  const int64_t batch = table.size(0), pages = table.size(1);
  need(cu.scalar_type() == at::kInt && cu.dim() == 1 && cu.size(0) == batch + 1 &&
           cu.is_contiguous(),
       "cu_seqlens must be a contiguous int32 (batch + 1) tensor");
  if (lens.defined())
    need(lens.scalar_type() == at::kInt && lens.dim() == 1 && lens.size(0) == batch &&
             lens.is_contiguous(),
         "sequence lengths and starts must be contiguous int32 (batch) tensors");
  need(batch <= INT_MAX && pages <= INT_MAX && total >= 0 && total <= INT_MAX,
       "the batch is too large");
  fa_ragged r{};
  r.block_table = table.const_data_ptr<int>();
  r.table_stride = batch > 1 ? table.stride(0) : std::max(pages, table.stride(0));
  r.max_pages = static_cast<int>(pages);
  r.cu_seqlens = cu.const_data_ptr<int>();
  r.seqlens = lens.defined() ? lens.const_data_ptr<int>() : nullptr;
  r.batch = static_cast<int>(batch);
  r.total = static_cast<int>(total);
  return r;
}

void check_rows(const at::Tensor& k, const at::Tensor& v, const at::Tensor& pages) {
  need(k.dim() == 3 && v.sizes() == k.sizes() && pages.dim() == 4 && k.size(1) == pages.size(2) &&
           k.size(2) == pages.size(3) && k.scalar_type() == v.scalar_type() && k.stride(2) == 1 &&
           v.stride(2) == 1,
       "k and v must be packed (total, nheads, headdim) tensors of the cache's heads, of one type "
       "and with the head dimension contiguous");
}

// append(k, v, k_pages, v_pages, block_table, cu_seqlens, seqlens, k_exp, v_exp)
PyObject* append(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0], "k must be a tensor"), &v = tensor(a[1], "v must be a tensor"),
                   &kp = tensor(a[2], "k_pages must be a tensor"),
                   &vp = tensor(a[3], "v_pages must be a tensor"),
                   &table = tensor(a[4], "block_table must be a tensor"),
                   &cu = tensor(a[5], "cu_seqlens must be a tensor"),
                   &lens = tensor(a[6], "seqlens must be a tensor");
  const at::Tensor ke = maybe(a[7], "k_exp must be a tensor or None"),
                   ve = maybe(a[8], "v_exp must be a tensor or None");
  for (const at::Tensor* t : {&k, &v, &kp, &vp})
    no_grad(*t, "the cache keeps no gradients: call under torch.no_grad()");
  check_rows(k, v, kp);
  const fa_kv_pages c = kv_pages(kp, vp, ke, ve);
  const fa_ragged r = ragged(table, cu, lens, k.size(0));
  const Device device({&k, &v, &kp, &vp, &table, &cu, &lens, &ke, &ve});
  for (const at::Tensor* t : {&kp, &vp, &ke, &ve}) written(*t);
  const fa_status st = fa_cache_append(&c, &r, k.const_data_ptr(), k.stride(0), k.stride(1),
                                       v.const_data_ptr(), v.stride(0), v.stride(1),
                                       static_cast<fa_elem>(elem(k.scalar_type())),
                                       device.stream());
  if (st != FA_OK) return status(st);
  Py_RETURN_NONE;
}

// read(k_pages, v_pages, block_table, cu_seqlens, total, starts, k_exp, v_exp, fa_elem or -1,
//      out_k, out_v)
PyObject* read(PyObject* const* a) {
  const at::Tensor &kp = tensor(a[0], "k_pages must be a tensor"),
                   &vp = tensor(a[1], "v_pages must be a tensor"),
                   &table = tensor(a[2], "block_table must be a tensor"),
                   &cu = tensor(a[3], "cu_seqlens must be a tensor");
  const int64_t total = integer(a[4]);
  const at::Tensor starts = maybe(a[5], "starts must be a tensor or None"),
                   ke = maybe(a[6], "k_exp must be a tensor or None"),
                   ve = maybe(a[7], "v_exp must be a tensor or None");
  for (const at::Tensor* t : {&kp, &vp})
    no_grad(*t, "the cache keeps no gradients: call under torch.no_grad()");
  const fa_kv_pages c = kv_pages(kp, vp, ke, ve);
  const fa_ragged r = ragged(table, cu, starts, total);
  const int asked = static_cast<int>(integer(a[8]));
  const int out_elem = asked >= 0 ? asked : c.type == FA_ELEM_E4M3 ? FA_ELEM_BF16 : c.type;
  if (out_elem != FA_ELEM_BF16 && out_elem != FA_ELEM_FP16)
    throw Refuse{PyExc_TypeError, "unsupported dtype; use bfloat16 or float16"};
  at::Tensor k = maybe(a[9], "out must be a pair of tensors"),
             v = maybe(a[10], "out must be a pair of tensors");
  if (k.defined() || v.defined()) {
    need(k.defined() && v.defined(), "out must be a pair of tensors");
    check_rows(k, v, kp);
    no_grad(k, "out must not need a gradient");
    no_grad(v, "out must not need a gradient");
    need(k.size(0) == total && elem(k.scalar_type()) == out_elem,
         "out must hold `total` rows of dtype");
  }
  const Device device({&kp, &vp, &table, &cu, &starts, &ke, &ve, &k, &v});
  if (k.defined()) {
    written(k);
    written(v);
  } else {
    const at::ScalarType type = out_elem == FA_ELEM_BF16 ? at::kBFloat16 : at::kHalf;
    k = make(kp, {total, kp.size(2), kp.size(3)}, type);
    v = make(kp, {total, kp.size(2), kp.size(3)}, type);
  }
  const fa_status st =
      fa_cache_read(&c, &r, r.seqlens, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
                    v.stride(0), v.stride(1), static_cast<fa_elem>(out_elem), device.stream());
  if (st != FA_OK) return status(st);
  return pair(k, v);
}

const int* int32s(const at::Tensor& t, int64_t n, const char* what) {
  need(t.scalar_type() == at::kInt && t.dim() == 1 && t.size(0) == n && t.is_contiguous(), what);
  return t.const_data_ptr<int>();
}

void check_table(const at::Tensor& table, const at::Tensor& free_pages) {
  need(table.dim() == 2 && table.scalar_type() == at::kInt &&
           (table.size(1) <= 1 || table.stride(1) == 1) && table.size(0) <= INT_MAX &&
           table.size(1) <= INT_MAX &&
           (table.size(0) <= 1 || table.stride(0) >= table.size(1)),
       "block_table must be an int32 (batch, max_pages) tensor with contiguous rows");
  need(free_pages.dim() == 1 && free_pages.scalar_type() == at::kInt &&
           free_pages.is_contiguous() && free_pages.size(0) <= INT_MAX,
       "free_pages must be a contiguous int32 tensor");
}

// Several one-dimensional results in one buffer, 16-byte aligned each.
class Parts {
 public:
  size_t take(int64_t bytes) {
    const size_t at = bytes_;
    bytes_ += (static_cast<size_t>(bytes) + 15) / 16 * 16;
    return at;
  }
  void allocate(const at::Tensor& like) {
    buffer_ = make(like, {static_cast<int64_t>(bytes_)}, at::kByte);
  }
  at::Tensor tensor(size_t at, int64_t n, at::ScalarType type) const {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(buffer_.storage()),
                                                     buffer_.key_set(),
                                                     c10::scalarTypeToTypeMeta(type));
    impl->set_storage_offset(static_cast<int64_t>(at / c10::elementSize(type)));
    impl->set_sizes_contiguous({n});
    return at::Tensor(std::move(impl));
  }

 private:
  at::Tensor buffer_;
  size_t bytes_ = 0;
};

constexpr const char* kBatchInts =
    "new_tokens, seqlens and keep_pages must be contiguous int32 (batch,) tensors";
constexpr const char* kOneInt = "free_count must be an int32 (1,) tensor";

int size_of_page(PyObject* o) {
  const long long v = integer(o);
  need(v >= 16 && v <= 256 && (v & (v - 1)) == 0, "page_size must be 16, 32, 64, 128 or 256");
  return static_cast<int>(v);
}

// reserve(new_tokens, seqlens, block_table, free_pages, free_count, page_size, total, inplace)
PyObject* reserve(PyObject* const* a) {
  const at::Tensor &fresh = tensor(a[0], "new_tokens must be a tensor"),
                   &lens = tensor(a[1], "seqlens must be a tensor"),
                   &table = tensor(a[2], "block_table must be a tensor"),
                   &pages = tensor(a[3], "free_pages must be a tensor"),
                   &count = tensor(a[4], "free_count must be a tensor");
  check_table(table, pages);
  const int64_t batch = table.size(0);
  fa_reserve r{};
  r.new_tokens = int32s(fresh, batch, kBatchInts);
  r.seqlens = int32s(lens, batch, kBatchInts);
  r.free_count = int32s(count, 1, kOneInt);
  r.page_size = size_of_page(a[5]);
  const long long total = integer(a[6]);
  need(total >= 0 && total <= INT_MAX, "total must not be negative");
  const bool inplace = truth(a[7]);
  const Device device({&fresh, &lens, &table, &pages, &count});
  // One allocation for all results: each costs about as much as the kernel takes.
  Parts parts;
  const size_t at_slots = parts.take(8 * total), at_positions = parts.take(4 * total),
               at_cu = parts.take(4 * (batch + 1)), at_lens = parts.take(4 * batch),
               at_count = parts.take(4), at_missing = parts.take(4);
  parts.allocate(fresh);
  const at::Tensor cu = parts.tensor(at_cu, batch + 1, at::kInt),
                   positions = parts.tensor(at_positions, total, at::kInt),
                   slots = parts.tensor(at_slots, total, at::kLong),
                   missing = parts.tensor(at_missing, 1, at::kInt),
                   lens_out = inplace ? lens : parts.tensor(at_lens, batch, at::kInt),
                   count_out = inplace ? count : parts.tensor(at_count, 1, at::kInt);
  r.block_table = table.data_ptr<int>();
  r.table_stride = batch > 1 ? table.stride(0) : std::max(table.size(1), table.stride(0));
  r.max_pages = static_cast<int>(table.size(1));
  r.free_pages = pages.const_data_ptr<int>();
  r.capacity = static_cast<int>(pages.size(0));
  r.batch = static_cast<int>(batch);
  r.total = static_cast<int>(total);
  r.cu_seqlens = cu.data_ptr<int>();
  r.seqlens_out = lens_out.data_ptr<int>();
  r.positions = positions.data_ptr<int>();
  r.slots = reinterpret_cast<long long*>(slots.data_ptr<int64_t>());
  r.free_count_out = count_out.data_ptr<int>();
  r.missing = missing.data_ptr<int>();
  written(table);
  if (inplace) {
    written(lens);
    written(count);
  }
  const fa_status st = fa_cache_reserve(&r, device.stream());
  if (st != FA_OK) return status(st);
  THPObjectPtr out(PyTuple_New(6));
  if (!out) throw python_error();
  Py_ssize_t i = 0;
  for (const at::Tensor* t : {&cu, &lens_out, &positions, &slots, &count_out, &missing})
    PyTuple_SET_ITEM(out.get(), i++, wrap(*t));
  return out.release();
}

// release(done, seqlens, block_table, free_pages, free_count, page_size, keep_pages)
PyObject* release(PyObject* const* a) {
  const at::Tensor &done = tensor(a[0], "done must be a tensor"),
                   &lens = tensor(a[1], "seqlens must be a tensor"),
                   &table = tensor(a[2], "block_table must be a tensor"),
                   &pages = tensor(a[3], "free_pages must be a tensor"),
                   &count = tensor(a[4], "free_count must be a tensor");
  const at::Tensor keep = maybe(a[6], "keep_pages must be a tensor or None");
  check_table(table, pages);
  const int64_t batch = table.size(0);
  need((done.scalar_type() == at::kBool || done.scalar_type() == at::kByte) && done.dim() == 1 &&
           done.size(0) == batch && done.is_contiguous(),
       "done must be a contiguous bool or uint8 (batch,) tensor");
  int32s(lens, batch, kBatchInts);
  int32s(count, 1, kOneInt);
  const int* kept = keep.defined() ? int32s(keep, batch, kBatchInts) : nullptr;
  const int page_size = size_of_page(a[5]);
  const Device device({&done, &lens, &table, &pages, &count, &keep});
  for (const at::Tensor* t : {&lens, &pages, &count}) written(*t);
  const fa_status st = fa_cache_release(
      static_cast<const unsigned char*>(done.const_data_ptr()), lens.data_ptr<int>(), kept,
      table.const_data_ptr<int>(),
      batch > 1 ? table.stride(0) : std::max(table.size(1), table.stride(0)),
      static_cast<int>(table.size(1)), pages.data_ptr<int>(), static_cast<int>(pages.size(0)),
      count.data_ptr<int>(), static_cast<int>(batch), page_size, device.stream());
  if (st != FA_OK) return status(st);
  Py_RETURN_NONE;
}

// write(k, v, k_pages, v_pages, slots, k_exp, v_exp)
PyObject* write(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0], "k must be a tensor"), &v = tensor(a[1], "v must be a tensor"),
                   &kp = tensor(a[2], "k_pages must be a tensor"),
                   &vp = tensor(a[3], "v_pages must be a tensor"),
                   &slots = tensor(a[4], "slots must be a tensor");
  const at::Tensor ke = maybe(a[5], "k_exp must be a tensor or None"),
                   ve = maybe(a[6], "v_exp must be a tensor or None");
  for (const at::Tensor* t : {&k, &v, &kp, &vp})
    no_grad(*t, "the cache keeps no gradients: call under torch.no_grad()");
  check_rows(k, v, kp);
  need(slots.scalar_type() == at::kLong && slots.dim() == 1 && slots.size(0) == k.size(0) &&
           slots.is_contiguous() && k.size(0) <= INT_MAX,
       "slots must be a contiguous int64 (total,) tensor");
  const fa_kv_pages c = kv_pages(kp, vp, ke, ve);
  const Device device({&k, &v, &kp, &vp, &slots, &ke, &ve});
  for (const at::Tensor* t : {&kp, &vp, &ke, &ve}) written(*t);
  const fa_status st = fa_cache_write(
      &c, reinterpret_cast<const long long*>(slots.const_data_ptr<int64_t>()),
      static_cast<int>(k.size(0)), k.const_data_ptr(), k.stride(0), k.stride(1), v.const_data_ptr(),
      v.stride(0), v.stride(1), static_cast<fa_elem>(elem(k.scalar_type())), device.stream());
  if (st != FA_OK) return status(st);
  Py_RETURN_NONE;
}

// paged(q, k_pages, v_pages, block_table, cu_seqlens, seqlens, scale, causal, window_left,
//       window_right, alibi_slopes, k_exp, v_exp, cu_groups, shared_pages)
PyObject* paged(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q must be a tensor"),
                   &kp = tensor(a[1], "k_pages must be a tensor"),
                   &vp = tensor(a[2], "v_pages must be a tensor"),
                   &table = tensor(a[3], "block_table must be a tensor"),
                   &cu = tensor(a[4], "cu_seqlens must be a tensor"),
                   &lens = tensor(a[5], "seqlens must be a tensor");
  const at::Tensor slopes = maybe(a[10], "alibi_slopes must be a tensor or None"),
                   ke = maybe(a[11], "k_exp must be a tensor or None"),
                   ve = maybe(a[12], "v_exp must be a tensor or None"),
                   cu_groups = maybe(a[13], "cu_groups must be a tensor or None"),
                   shared = maybe(a[14], "shared_pages must be a tensor or None");
  for (const at::Tensor* t : {&q, &kp, &vp, &slopes})
    no_grad(*t, "attention over a cache has no backward: call under torch.no_grad()");
  const fa_kv_pages c = kv_pages(kp, vp, ke, ve);
  need(q.dim() == 3 && q.stride(2) == 1 && q.size(2) == c.head_dim,
       "q must be a packed (total, nheads, headdim) tensor of the cache's headdim, which must be "
       "contiguous");
  const int64_t total = q.size(0), heads = q.size(1);
  need(c.heads > 0 && heads % c.heads == 0 && heads <= INT_MAX,
       "nheads must be a multiple of the cache's heads");
  const fa_ragged r = ragged(table, cu, lens, total);
  fa_options opt{};
  opt.window_left = static_cast<int>(std::min<long long>(integer(a[8]), INT_MAX));
  opt.window_right = static_cast<int>(std::min<long long>(integer(a[9]), INT_MAX));
  if (slopes.defined()) {
    need(slopes.scalar_type() == at::kFloat && slopes.is_contiguous() &&
             ((slopes.dim() == 1 && slopes.size(0) == heads) ||
              (slopes.dim() == 2 && slopes.size(0) == r.batch && slopes.size(1) == heads)),
         "alibi_slopes must be a contiguous float32 (nheads,) or (batch, nheads) tensor");
    opt.alibi_slopes = slopes.const_data_ptr<float>();
    opt.alibi_per_batch = slopes.dim() == 2;
  }
  const bool grouped = cu_groups.defined();
  const bool causal = truth(a[7]);
  need(grouped == shared.defined(), "cu_groups and shared_pages go together");
  int groups = 0;
  if (grouped) {
    need(causal && opt.window_left == -1 && opt.window_right == -1 && !slopes.defined(),
         "cu_groups are for causal attention without window and alibi_slopes");
    need(shared.dim() == 1 && shared.size(0) <= r.batch,
         "there must be at most as many groups as sequences");
    groups = static_cast<int>(shared.size(0));
    int32s(shared, groups, "shared_pages must be a contiguous int32 (groups,) tensor");
    int32s(cu_groups, groups + 1, "cu_groups must be a contiguous int32 (groups + 1,) tensor");
  }
  const Device device({&q, &kp, &vp, &table, &cu, &lens, &slopes, &ke, &ve, &cu_groups, &shared});
  const int D = c.head_dim, H = static_cast<int>(heads);
  const long long max_keys = static_cast<long long>(r.max_pages) * c.page_size;
  size_t bytes = 0;
  fa_status st =
      grouped ? fa_fwd_paged_shared_workspace_size(r.batch, r.total, H, c.heads, D, max_keys,
                                                   groups, &bytes)
              : fa_fwd_paged_workspace_size(r.batch, r.total, H, c.heads, D, max_keys, &bytes);
  if (st != FA_OK) return status(st);
  const at::Tensor o = like(q);
  const at::Tensor lse = make(q, {heads, total}, at::kFloat);
  at::Tensor ws;
  if (bytes)
    ws = make(q, {static_cast<int64_t>(bytes)}, at::kByte);
  const float scale = static_cast<float>(number(a[6]));
  const fa_elem type = static_cast<fa_elem>(elem(q.scalar_type()));
  void* const room = bytes ? ws.data_ptr() : nullptr;
  if (grouped)
    st = fa_fwd_paged_shared(q.const_data_ptr(), q.stride(0), q.stride(1), o.data_ptr(),
                             o.stride(0), o.stride(1), lse.data_ptr<float>(), &c, &r,
                             cu_groups.const_data_ptr<int>(), shared.const_data_ptr<int>(), groups,
                             H, scale, type, room, bytes, device.stream());
  else
    st = fa_fwd_paged(q.const_data_ptr(), q.stride(0), q.stride(1), o.data_ptr(), o.stride(0),
                      o.stride(1), lse.data_ptr<float>(), &c, &r, H, &opt, scale, causal, type,
                      room, bytes, device.stream());
  if (st != FA_OK) return status(st);
  return pair(o, lse);
}

// Turns what a function above throws into a Python exception.
template <PyObject* (*kFn)(PyObject* const*), Py_ssize_t kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != kArgs) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return kFn(args);
  } catch (const Refuse& r) {
    PyErr_SetString(r.type, r.text);
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*kFn)(PyObject* const*), Py_ssize_t kArgs>
PyMethodDef method(const char* name) {
  return PyMethodDef{name,
                     reinterpret_cast<PyCFunction>(
                         reinterpret_cast<void (*)()>(&entry<kFn, kArgs>)),
                     METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<rotary, 9>("rotary"),   method<norm_rotary, 12>("norm_rotary"),
                         method<append, 9>("append"),   method<write, 7>("write"),
                         method<read, 11>("read"),      method<reserve, 8>("reserve"),
                         method<release, 7>("release"), method<paged, 15>("paged"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind_torch", nullptr, -1, methods,
                      nullptr,               nullptr,       nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind_torch(void) { return PyModule_Create(&module); }
