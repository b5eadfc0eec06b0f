// Native calls of the dense operators for ordinary arguments.  A decode step makes many of
// these calls and each runs for a few microseconds, less than the interpreter takes to check
// and marshal one.  Every function here checks what the Python wrapper checks (api.py) and
// allocates the outputs; whatever is not ordinary (a tensor subclass, rows apart, buffers
// given, a wrong argument) it leaves alone by returning None, and the wrapper, which names
// what is wrong, goes on.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mbq.h"

namespace {

constexpr auto kF8 = at::kFloat8_e4m3fn;

const at::Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// On the device and contiguous, of this many dimensions.
bool plain(const at::Tensor* t, int64_t device, int64_t dims) {
  return t && t->dim() == dims && t->is_cuda() && t->get_device() == device && t->is_contiguous();
}
bool is_float(at::ScalarType t) { return t == at::kFloat || t == at::kBFloat16; }
mbq_dtype code(at::ScalarType t) { return t == at::kFloat ? MBQ_F32 : t == at::kBFloat16 ? MBQ_BF16 : MBQ_E4M3; }

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& like) {
  return at::empty(sizes, like.options().dtype(type));
}

// An optional float32 [k] vector: its address, or nullptr for None; ok says whether it is one of the two.
const float* vector(PyObject* o, int64_t k, int64_t device, bool& ok) {
  if (o == Py_None) return nullptr;
  const at::Tensor* t = tensor(o);
  if (!plain(t, device, 1) || t->size(0) != k || t->scalar_type() != at::kFloat) {
    ok = false;
    return nullptr;
  }
  return static_cast<const float*>(t->data_ptr());
}

// An output type: None for `missing`; anything but float32 and bfloat16 is not ordinary.
bool out_type(PyObject* o, at::ScalarType missing, at::ScalarType& type) {
  type = o == Py_None ? missing : THPDtype_Check(o) ? reinterpret_cast<THPDtype*>(o)->scalar_type : at::kByte;
  return is_float(type);
}

// (desc address, blob, x, scale, act or -1, out_dtype, device, stream) -> y
PyObject* fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) return PyErr_Format(PyExc_TypeError, "fp8 takes 8 arguments");
  const auto* d = static_cast<const mbq_fp8_desc*>(PyLong_AsVoidPtr(a[0]));
  const int64_t device = PyLong_AsLongLong(a[6]);
  const long act = PyLong_AsLong(a[4]);
  void* stream = PyLong_AsVoidPtr(a[7]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor *blob = tensor(a[1]), *x = tensor(a[2]);
  if (!plain(x, device, 2) || !plain(blob, device, 1)) Py_RETURN_NONE;
  const int64_t t = x->size(0);
  const at::ScalarType xt = x->scalar_type();
  if (x->size(1) != d->k || (d->gated != 0) != (act >= 0) || t > (1 << 21) || blob->scalar_type() != at::kByte ||
      uint64_t(blob->numel()) < d->total_bytes)
    Py_RETURN_NONE;
  const float* scale = nullptr;
  if (xt == kF8) {
    const at::Tensor* s = tensor(a[3]);
    if (!plain(s, device, 2) || s->scalar_type() != at::kFloat || s->size(0) != d->k_blocks || s->size(1) != t) Py_RETURN_NONE;
    scale = static_cast<const float*>(s->data_ptr());
  } else if (!is_float(xt) || a[3] != Py_None) {
    Py_RETURN_NONE;
  }
  at::ScalarType yt;
  size_t need = 0;
  if (!out_type(a[5], xt == kF8 ? at::kBFloat16 : xt, yt) ||
      mbq_fp8_linear_workspace(d, int32_t(t), code(xt), &need) != MBQ_OK)
    Py_RETURN_NONE;
  at::AutoDispatchBelowADInplaceOrView guard;
  const at::Tensor y = empty({t, d->n}, yt, *x);
  at::Tensor ws;
  if (need) ws = empty({int64_t(need)}, at::kByte, *x);
  void* wp = need ? ws.data_ptr() : nullptr;
  const auto s = static_cast<hipStream_t>(stream);
  const mbq_status st =
      act < 0 ? mbq_fp8_linear(d, blob->data_ptr(), int32_t(t), x->data_ptr(), code(xt), d->k, scale, y.data_ptr(), code(yt), wp, need, s)
              : mbq_fp8_gated(d, blob->data_ptr(), int32_t(t), x->data_ptr(), code(xt), d->k, scale, mbq_act(act), y.data_ptr(),
                              code(yt), wp, need, s);
  if (st != MBQ_OK) Py_RETURN_NONE;
  return THPVariable_Wrap(y);
}

// (x, device, stream) -> (codes, scale)
PyObject* fp8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3) return PyErr_Format(PyExc_TypeError, "fp8_quantize takes 3 arguments");
  const int64_t device = PyLong_AsLongLong(a[1]);
  void* stream = PyLong_AsVoidPtr(a[2]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor* x = tensor(a[0]);
  if (!plain(x, device, 2) || !is_float(x->scalar_type()) || x->size(0) > (1 << 21) || x->size(1) > (1 << 24)) Py_RETURN_NONE;
  const int64_t t = x->size(0), k = x->size(1);
  at::AutoDispatchBelowADInplaceOrView guard;
  const at::Tensor q = empty({t, k}, kF8, *x), s = empty({(k + 127) / 128, t}, at::kFloat, *x);
  if (mbq_fp8_quantize(int32_t(t), int32_t(k), x->data_ptr(), code(x->scalar_type()), k, q.data_ptr(), k,
                       static_cast<float*>(s.data_ptr()), static_cast<hipStream_t>(stream)) != MBQ_OK)
    Py_RETURN_NONE;
  return Py_BuildValue("(NN)", THPVariable_Wrap(q), THPVariable_Wrap(s));
}

// (x, residual, pre, post, gate, residual_scale, gate_scale, eps, kind, pre_bias, post_bias, quantized, out_dtype,
//  device, stream) -> (y, h) or (y, codes, scale)
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 15) return PyErr_Format(PyExc_TypeError, "block_norm takes 15 arguments");
  const float residual_scale = float(PyFloat_AsDouble(a[5])), gate_scale = float(PyFloat_AsDouble(a[6]));
  const float eps = float(PyFloat_AsDouble(a[7]));
  const int64_t device = PyLong_AsLongLong(a[13]);
  void* stream = PyLong_AsVoidPtr(a[14]);
  const long kind = PyLong_AsLong(a[8]);
  const int quantized = PyObject_IsTrue(a[11]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor* x = tensor(a[0]);
  if (!plain(x, device, 2) || !is_float(x->scalar_type()) || x->size(0) > (1 << 21) || x->size(1) > (1 << 24)) Py_RETURN_NONE;
  const int64_t t = x->size(0), k = x->size(1);
  mbq_block_norm_args g = {};
  at::ScalarType rt = x->scalar_type(), ht;
  if (a[1] != Py_None) {
    const at::Tensor* r = tensor(a[1]);
    if (!plain(r, device, 2) || !is_float(r->scalar_type()) || r->size(0) != t || r->size(1) != k) Py_RETURN_NONE;
    rt = r->scalar_type();
    g.residual = r->data_ptr();
  }
  bool ok = true;
  g.pre_weight = vector(a[2], k, device, ok);
  g.post_weight = vector(a[3], k, device, ok);
  g.pre_bias = vector(a[9], k, device, ok);
  g.post_bias = vector(a[10], k, device, ok);
  if (!ok) Py_RETURN_NONE;
  if (a[4] != Py_None) {
    const at::Tensor* v = tensor(a[4]);
    if (v && v->dim() == 2) {
      if (!plain(v, device, 2) || v->scalar_type() != x->scalar_type() || v->size(0) != t || v->size(1) != k) Py_RETURN_NONE;
      g.gate_kind = MBQ_GATE_FULL;
    } else {
      if (!plain(v, device, 1) || v->scalar_type() != at::kFloat || (v->size(0) != k && v->size(0) != t)) Py_RETURN_NONE;
      g.gate_kind = v->size(0) == k ? MBQ_GATE_CHANNEL : MBQ_GATE_TOKEN;
    }
    g.gate = v->data_ptr();
  }
  if (!out_type(a[12], x->scalar_type(), ht)) Py_RETURN_NONE;
  if (quantized) ht = kF8;
  at::AutoDispatchBelowADInplaceOrView guard;
  const at::Tensor y = empty({t, k}, rt, *x), h = empty({t, k}, ht, *x);
  at::Tensor s;
  if (quantized) {
    s = empty({(k + 127) / 128, t}, at::kFloat, *x);
    g.scale = static_cast<float*>(s.data_ptr());
  }
  g.t = int32_t(t);
  g.k = int32_t(k);
  g.kind = int32_t(kind);
  g.x_dtype = code(x->scalar_type());
  g.r_dtype = code(rt);
  g.h_dtype = code(ht);
  g.post = a[3] != Py_None;
  g.x = x->data_ptr();
  g.y = y.data_ptr();
  g.h = h.data_ptr();
  g.ldx = g.ldr = g.ldy = g.ldh = k;
  g.residual_scale = residual_scale;
  g.gate_scale = gate_scale;
  g.eps = eps;
  if (mbq_block_norm(&g, static_cast<hipStream_t>(stream)) != MBQ_OK) Py_RETURN_NONE;
  if (quantized) return Py_BuildValue("(NNN)", THPVariable_Wrap(y), THPVariable_Wrap(h), THPVariable_Wrap(s));
  return Py_BuildValue("(NN)", THPVariable_Wrap(y), THPVariable_Wrap(h));
}

// (logits, targets, top, inv_temperature, device, stream) -> (logprob, entropy, rank, top_ids or None, top_logprobs or None)
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return PyErr_Format(PyExc_TypeError, "token_logprobs takes 6 arguments");
  const long top = PyLong_AsLong(a[2]);
  const float inv_temperature = float(PyFloat_AsDouble(a[3]));
  const int64_t device = PyLong_AsLongLong(a[4]);
  void* stream = PyLong_AsVoidPtr(a[5]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor *x = tensor(a[0]), *targets = tensor(a[1]);
  if (!plain(x, device, 2) || !is_float(x->scalar_type()) || !plain(targets, device, 1)) Py_RETURN_NONE;
  const int64_t t = x->size(0), v = x->size(1);
  const at::ScalarType tt = targets->scalar_type();
  if (targets->size(0) != t || (tt != at::kInt && tt != at::kLong) || t > (1 << 21) || v > (1 << 28) || top < 0 ||
      top > MBQ_MAX_TOP || top > v)
    Py_RETURN_NONE;
  size_t need = 0;
  if (mbq_token_logprobs_workspace(int32_t(t), int32_t(v), int32_t(top), &need) != MBQ_OK) Py_RETURN_NONE;
  at::AutoDispatchBelowADInplaceOrView guard;
  const at::Tensor logprob = empty({t}, at::kFloat, *x), entropy = empty({t}, at::kFloat, *x), rank = empty({t}, at::kInt, *x);
  at::Tensor ids, best, ws;
  if (top) {
    ids = empty({t, top}, at::kInt, *x);
    best = empty({t, top}, at::kFloat, *x);
  }
  if (need) ws = empty({int64_t(need)}, at::kByte, *x);
  if (mbq_token_logprobs(int32_t(t), int32_t(v), x->data_ptr(), code(x->scalar_type()), v, targets->data_ptr(),
                         tt == at::kInt ? 32 : 64, inv_temperature, int32_t(top), static_cast<float*>(logprob.data_ptr()),
                         static_cast<float*>(entropy.data_ptr()), static_cast<int32_t*>(rank.data_ptr()),
                         top ? static_cast<int32_t*>(ids.data_ptr()) : nullptr,
                         top ? static_cast<float*>(best.data_ptr()) : nullptr, need ? ws.data_ptr() : nullptr, need,
                         static_cast<hipStream_t>(stream)) != MBQ_OK)
    Py_RETURN_NONE;
  if (!top)
    return Py_BuildValue("(NNNOO)", THPVariable_Wrap(logprob), THPVariable_Wrap(entropy), THPVariable_Wrap(rank), Py_None, Py_None);
  return Py_BuildValue("(NNNNN)", THPVariable_Wrap(logprob), THPVariable_Wrap(entropy), THPVariable_Wrap(rank),
                       THPVariable_Wrap(ids), THPVariable_Wrap(best));
}

// No C++ exception (an allocation that fails, above all) crosses into the interpreter.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;  // the wrapper meets the same failure and reports it
  }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<fp8>("fp8"), method<fp8_quantize>("fp8_quantize"), method<block_norm>("block_norm"),
                         method<token_logprobs>("token_logprobs"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
