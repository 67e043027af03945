// bind_torch.cpp -- the Python entry to include/fattn_cache.h: checks torch
// tensors, allocates the results and calls the C ABI of libfattn.so.
//
// These calls are made for every layer and token while generating, when the
// kernels take a few microseconds: the same marshalling written in Python over
// ctypes cost 15 to 30 us a call on the host of a GB300.  Arguments are
// positional; rotary.py, kvcache.py and attention.py hold the public signatures
// and their documentation.  Each function returns its tensors, or the
// fa_status of a refused call as an int.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <climits>
#include <optional>
#include <vector>

#include "fattn_cache.h"

namespace {

// Raised as the Python exception of the given type.
struct Refuse {
  PyObject* type;
  const char* what;
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

at::Tensor like(const at::Tensor& x) { return at::empty(x.sizes(), x.options().requires_grad(false)); }

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
};

// Turns x into y, and x2 (when defined) into y2.
fa_status turn(const at::Tensor& x, const at::Tensor& y, const at::Tensor& x2,
               const at::Tensor& y2, const Rotation& r, const Device& device) {
  const int64_t dim = x.dim(), B = dim == 4 ? x.size(0) : 1, N = x.size(dim - 3);
  need(B <= INT_MAX && N <= INT_MAX, "tensors too large");
  const fa_rotary_operand a = rotary_operand(x, y);
  fa_rotary_operand b;
  if (x2.defined()) b = rotary_operand(x2, y2);
  const bool pos = r.pos.defined() && r.pos.numel() > 0;  // (no tokens: no address either)
  return fa_rotary(&a, x2.defined() ? &b : nullptr, static_cast<int>(B), static_cast<int>(N),
                   static_cast<int>(x.size(dim - 1)), static_cast<int>(2 * r.freq.size(0)),
                   r.freq.const_data_ptr<double>(), pos ? r.pos.const_data_ptr() : nullptr,
                   !pos ? 0 : r.pos.scalar_type() == at::kInt ? 32 : 64,
                   pos && r.pos.dim() == 2 ? r.pos.stride(0) : 0,
                   static_cast<float>(r.magnitude), r.interleaved, r.inverse,
                   static_cast<fa_elem>(elem(x.scalar_type())), device.stream());
}

// What the C ABI refuses inside autograd.
void check(fa_status st) {
  TORCH_CHECK(st == FA_OK, "fa_rotary failed: ", fa_status_string(st), " (", static_cast<int>(st),
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
    ctx->saved_data["magnitude"] = r.magnitude;
    ctx->saved_data["interleaved"] = r.interleaved;
    ctx->saved_data["inverse"] = r.inverse;
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
  const Rotation r{saved[0], saved[1], ctx->saved_data["magnitude"].toDouble(),
                   ctx->saved_data["interleaved"].toBool(),
                   !ctx->saved_data["inverse"].toBool()};
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

// rotary(q, k, inv_freq, positions, magnitude, interleaved, inplace)
PyObject* rotary(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q must be a tensor");
  const at::Tensor k = maybe(a[1], "k must be a tensor or None");
  Rotation r{tensor(a[2], "inv_freq must be a tensor"),
             maybe(a[3], "positions must be a tensor or None"), number(a[4]), truth(a[5]), false};
  const bool inplace = truth(a[6]);
  const int64_t dim = q.dim();
  need(dim == 3 || dim == 4,
       "expected (batch, seqlen, nheads, headdim) or packed (total, nheads, headdim) tensors");
  if (k.defined())
    need(k.dim() == dim && k.size(0) == q.size(0) && (dim == 3 || k.size(1) == q.size(1)) &&
             k.size(dim - 1) == q.size(dim - 1) && k.scalar_type() == q.scalar_type(),
         "q and k must agree in type and in every dimension but the heads");
  need(r.freq.scalar_type() == at::kDouble && r.freq.dim() == 1 && r.freq.is_contiguous(),
       "inv_freq must be a contiguous float64 (rotary_dim / 2) tensor");
  const int64_t B = dim == 4 ? q.size(0) : 1, N = q.size(dim - 3);
  if (r.pos.defined()) {
    if (r.pos.scalar_type() != at::kInt && r.pos.scalar_type() != at::kLong)
      throw Refuse{PyExc_TypeError, "positions must be int32 or int64"};
    need((r.pos.dim() == 1 && r.pos.size(0) == N) ||
             (dim == 4 && r.pos.dim() == 2 && r.pos.size(0) == B && r.pos.size(1) == N),
         "positions must have shape (seqlen,) or (batch, seqlen)");
  }
  need(!r.freq.requires_grad(), "inv_freq gets no gradient: detach it");
  for (const at::Tensor* t : {&q, &k, static_cast<const at::Tensor*>(&r.freq)}) no_tangent(*t);
  const Device device({&q, &k, &r.freq, &r.pos});
  if (r.pos.defined() && N > 1 && r.pos.stride(-1) != 1) r.pos = r.pos.contiguous();
  const bool grad =
      c10::GradMode::is_enabled() && (q.requires_grad() || (k.defined() && k.requires_grad()));
  if (grad) {
    need(!inplace, "inplace=True would overwrite tensors that need a gradient");
    auto y = k.defined() ? RotaryFunction<2>::apply(q, k, r) : RotaryFunction<1>::apply(q, r);
    return k.defined() ? pair(std::move(y[0]), std::move(y[1])) : wrap(std::move(y[0]));
  }
  const at::Tensor yq = inplace ? q : like(q), yk = !k.defined() || inplace ? k : like(k);
  if (inplace) {
    need(!k.defined() || k.numel() == 0 || k.const_data_ptr() != q.const_data_ptr(),
         "q and k would be written over each other");
    written(q);
    written(k);
  }
  const fa_status st = turn(q, yq, k, yk, r, device);
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
    const auto opt = kp.options().requires_grad(false).dtype(out_elem == FA_ELEM_BF16 ? at::kBFloat16
                                                                                    : at::kHalf);
    k = at::empty({total, kp.size(2), kp.size(3)}, opt);
    v = at::empty({total, kp.size(2), kp.size(3)}, opt);
  }
  const fa_status st =
      fa_cache_read(&c, &r, r.seqlens, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
                    v.stride(0), v.stride(1), static_cast<fa_elem>(out_elem), device.stream());
  if (st != FA_OK) return status(st);
  return pair(k, v);
}

// paged(q, k_pages, v_pages, block_table, cu_seqlens, seqlens, scale, causal, window_left,
//       window_right, alibi_slopes, k_exp, v_exp)
PyObject* paged(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q must be a tensor"),
                   &kp = tensor(a[1], "k_pages must be a tensor"),
                   &vp = tensor(a[2], "v_pages must be a tensor"),
                   &table = tensor(a[3], "block_table must be a tensor"),
                   &cu = tensor(a[4], "cu_seqlens must be a tensor"),
                   &lens = tensor(a[5], "seqlens must be a tensor");
  const at::Tensor slopes = maybe(a[10], "alibi_slopes must be a tensor or None"),
                   ke = maybe(a[11], "k_exp must be a tensor or None"),
                   ve = maybe(a[12], "v_exp must be a tensor or None");
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
  const Device device({&q, &kp, &vp, &table, &cu, &lens, &slopes, &ke, &ve});
  const int D = c.head_dim, H = static_cast<int>(heads);
  size_t bytes = 0;
  fa_status st = fa_fwd_paged_workspace_size(r.batch, r.total, H, c.heads, D,
                                             static_cast<long long>(r.max_pages) * c.page_size,
                                             &bytes);
  if (st != FA_OK) return status(st);
  const at::Tensor o = like(q);
  const at::Tensor lse = at::empty({heads, total}, q.options().requires_grad(false).dtype(at::kFloat));
  at::Tensor ws;
  if (bytes)
    ws = at::empty({static_cast<int64_t>(bytes)},
                   q.options().requires_grad(false).dtype(at::kByte));
  st = fa_fwd_paged(q.const_data_ptr(), q.stride(0), q.stride(1), o.data_ptr(), o.stride(0),
                    o.stride(1), lse.data_ptr<float>(), &c, &r, H, &opt,
                    static_cast<float>(number(a[6])), truth(a[7]),
                    static_cast<fa_elem>(elem(q.scalar_type())), bytes ? ws.data_ptr() : nullptr,
                    bytes, device.stream());
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
    PyErr_SetString(r.type, r.what);
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

PyMethodDef methods[] = {method<rotary, 7>("rotary"), method<append, 9>("append"),
                         method<read, 11>("read"), method<paged, 13>("paged"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind_torch", nullptr, -1, methods,
                      nullptr,               nullptr,       nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind_torch(void) { return PyModule_Create(&module); }
