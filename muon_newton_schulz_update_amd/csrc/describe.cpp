// Python extension `_describe`: packs lists of torch tensors into arrays of
// muon_matrix for the C ABI. Argument marshalling only, the same checks as the
// binding's Python code, natively: from Python each tensor costs about 0.6 us
// (shape, stride, type, device and pointer are a call each), which for the few
// dozen tensors of an optimizer's list is several times the GPU's work. The norms,
// whose GPU work is a few us, are called from here as a whole, through the address
// of the C entry point.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/Functions.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../include/libmuon.h"

namespace {

// Fills one descriptor; false with a Python error set.
bool describe(const at::Tensor& t, const char* what, long device, muon_matrix* m) {
  const auto type = t.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) {
    PyErr_Format(PyExc_TypeError, "%s: dtype %s is not float32 or bfloat16", what, c10::toString(type));
    return false;
  }
  if (t.layout() != at::kStrided) {
    PyErr_Format(PyExc_ValueError, "%s: expected a dense tensor", what);
    return false;
  }
  if (t.is_neg()) {
    PyErr_Format(PyExc_ValueError, "%s: a negated view holds its values with the other sign", what);
    return false;
  }
  if (t._fw_grad(0).defined()) {
    // (the kernels see the values alone: the result would have no tangent)
    PyErr_Format(PyExc_ValueError, "%s: a forward-mode tangent cannot be carried through", what);
    return false;
  }
  m->dtype = type == at::kBFloat16 ? MUON_BF16 : MUON_F32;
  if (t.dim() == 2) {
    m->rows = t.size(0);
    m->cols = t.size(1);
    if (m->cols > 1 && m->rows > 0 && t.stride(1) != 1) {
      PyErr_Format(PyExc_ValueError, "%s: columns must be contiguous (stride(1) == 1)", what);
      return false;
    }
    m->ld = m->rows > 1 ? t.stride(0) : m->cols;
  } else {
    if (!t.is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s: a tensor that is not a matrix must be contiguous", what);
      return false;
    }
    m->rows = 1;
    m->cols = t.numel();
    m->ld = m->cols;
  }
  const bool any = m->rows > 0 && m->cols > 0;
  if (any && (!t.is_cuda() || t.get_device() != device)) {
    PyErr_Format(PyExc_ValueError, "%s: expected a tensor on GPU %ld, got one on %s", what, device,
                 t.device().str().c_str());
    return false;
  }
  m->ptr = any ? t.data_ptr() : nullptr;
  return true;
}

// The same of rows: the last dimension's, all the others together.
bool describe_rows(const at::Tensor& t, const char* what, long device, muon_matrix* m) {
  if (!describe(t, what, device, m)) return false;
  if (t.dim() <= 2) return true;
  const int64_t cols = t.size(-1);
  m->rows = cols ? t.numel() / cols : 0;
  m->cols = m->ld = cols;
  return true;
}

const at::Tensor* tensor_of(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: expected a tensor, got %s", what, Py_TYPE(o)->tp_name);
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}

// pack(tensors, what, device, like=None, like_what="") -> bytes: one muon_matrix
// a tensor. With `like`, a list of as many tensors of the same shapes, entries
// may be None (an empty descriptor).
PyObject* pack(PyObject*, PyObject* args) {
  PyObject *tensors, *like = Py_None;
  const char *what, *like_what = "";
  long device;
  if (!PyArg_ParseTuple(args, "Osl|Os", &tensors, &what, &device, &like, &like_what)) return nullptr;
  PyObject* list = PySequence_Fast(tensors, "expected a sequence of tensors");
  if (!list) return nullptr;
  PyObject* likes = nullptr;
  if (like != Py_None && !(likes = PySequence_Fast(like, "expected a sequence of tensors"))) {
    Py_DECREF(list);
    return nullptr;
  }
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(list);
  PyObject* out = nullptr;
  bool ok = true;
  if (likes && PySequence_Fast_GET_SIZE(likes) != n) {
    PyErr_Format(PyExc_ValueError, "%s and %s differ in length", like_what, what);
    ok = false;
  }
  // (never empty: an empty list still has an address)
  if (ok) out = PyBytes_FromStringAndSize(nullptr, (n ? n : 1) * (Py_ssize_t)sizeof(muon_matrix));
  ok = ok && out;
  if (ok) {
    muon_matrix* m = (muon_matrix*)PyBytes_AS_STRING(out);
    memset(m, 0, (size_t)(n ? n : 1) * sizeof(muon_matrix));
    try {
      for (Py_ssize_t i = 0; ok && i < n; ++i) {
        PyObject* o = PySequence_Fast_GET_ITEM(list, i);
        if (o == Py_None && likes) continue;
        const at::Tensor* t = tensor_of(o, what);
        ok = t && describe(*t, what, device, m + i);
        if (!ok || !likes) continue;
        const at::Tensor* u = tensor_of(PySequence_Fast_GET_ITEM(likes, i), like_what);
        ok = u != nullptr;
        if (ok && t->sizes() != u->sizes()) {
          PyErr_Format(PyExc_ValueError, "%s[%zd] and %s[%zd] differ in shape", like_what, i, what, i);
          ok = false;
        }
      }
    } catch (const std::exception& e) {
      PyErr_SetString(PyExc_RuntimeError, e.what());
      ok = false;
    }
  }
  Py_DECREF(list);
  Py_XDECREF(likes);
  if (!ok) {
    Py_XDECREF(out);
    return nullptr;
  }
  return out;
}

// pack_rows(tensors, names, device) -> (bytes, their address): one muon_matrix a
// tensor, whose columns are its last dimension and whose rows all the others
// together; None is an empty descriptor. The address holds while the bytes do.
PyObject* pack_rows(PyObject*, PyObject* args) {
  PyObject *tensors, *names;
  long device;
  if (!PyArg_ParseTuple(args, "O!O!l", &PyTuple_Type, &tensors, &PyTuple_Type, &names, &device)) return nullptr;
  const Py_ssize_t n = PyTuple_GET_SIZE(tensors);
  if (PyTuple_GET_SIZE(names) != n) {
    PyErr_SetString(PyExc_ValueError, "tensors and names differ in length");
    return nullptr;
  }
  PyObject* out = PyBytes_FromStringAndSize(nullptr, (n ? n : 1) * (Py_ssize_t)sizeof(muon_matrix));
  if (!out) return nullptr;
  muon_matrix* m = (muon_matrix*)PyBytes_AS_STRING(out);
  memset(m, 0, (size_t)(n ? n : 1) * sizeof(muon_matrix));
  bool ok = true;
  try {
    for (Py_ssize_t i = 0; ok && i < n; ++i) {
      PyObject* o = PyTuple_GET_ITEM(tensors, i);
      if (o == Py_None) continue;
      const char* what = PyUnicode_AsUTF8(PyTuple_GET_ITEM(names, i));
      const at::Tensor* t = what ? tensor_of(o, what) : nullptr;
      ok = t && describe_rows(*t, what, device, m + i);
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    ok = false;
  }
  PyObject* both = ok ? Py_BuildValue("(Nn)", out, (Py_ssize_t)m) : nullptr;
  if (!both && !ok) Py_DECREF(out);
  return both;
}

// device_of(tensors) -> index of the first tensor on a GPU, or -1
PyObject* device_of(PyObject*, PyObject* arg) {
  PyObject* list = PySequence_Fast(arg, "expected a sequence of tensors");
  if (!list) return nullptr;
  long device = -1;
  for (Py_ssize_t i = 0; device < 0 && i < PySequence_Fast_GET_SIZE(list); ++i) {
    PyObject* o = PySequence_Fast_GET_ITEM(list, i);
    if (THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda()) device = THPVariable_Unpack(o).get_device();
  }
  Py_DECREF(list);
  return PyLong_FromLong(device);
}

// leaf_elsewhere(tensors) -> whether what adds to the gradient of one of them, a leaf,
// is there already and runs on another stream than the current one of its device
PyObject* leaf_elsewhere(PyObject*, PyObject* arg) {
  PyObject* list = PySequence_Fast(arg, "expected a sequence of tensors");
  if (!list) return nullptr;
  bool found = false, ok = true;
  try {
    for (Py_ssize_t i = 0; !found && i < PySequence_Fast_GET_SIZE(list); ++i) {
      PyObject* o = PySequence_Fast_GET_ITEM(list, i);
      if (!THPVariable_Check(o)) continue;
      const at::Tensor& t = THPVariable_Unpack(o);
      if (!t.is_cuda() || !t.requires_grad() || t.grad_fn()) continue;
      const auto node = torch::autograd::impl::try_get_grad_accumulator(t);
      const auto stream = node ? node->stream() : std::nullopt;
      found = stream && *stream != c10::impl::VirtualGuardImpl(at::kCUDA).getStream(t.device());
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    ok = false;
  }
  Py_DECREF(list);
  return ok ? PyBool_FromLong(found) : nullptr;
}

// empty(device, shape_of=None, type_of=None) -> a contiguous tensor on the GPU:
// the shape of one tensor (None: a scalar), the type of another (None: float32)
PyObject* empty(PyObject*, PyObject* args) {
  PyObject *shape_of = Py_None, *type_of = Py_None;
  long device;
  if (!PyArg_ParseTuple(args, "l|OO", &device, &shape_of, &type_of)) return nullptr;
  const at::Tensor *shape = nullptr, *type = nullptr;
  if (shape_of != Py_None && !(shape = tensor_of(shape_of, "shape_of"))) return nullptr;
  if (type_of != Py_None && !(type = tensor_of(type_of, "type_of"))) return nullptr;
  try {
    const auto options = at::TensorOptions()
                             .dtype(type ? type->scalar_type() : at::kFloat)
                             .device(at::kCUDA, (c10::DeviceIndex)device);
    return THPVariable_Wrap(at::empty(shape ? shape->sizes() : at::IntArrayRef(), options));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// ---------------------------------------------------------------------------
// The norms around a block (norms.py): shapes, results, descriptors and the call.
// ---------------------------------------------------------------------------
constexpr int kNormInputs = 6;
const char* const kNormNames[kNormInputs] = {"x", "y", "post_gain", "gate", "scale", "pre_gain"};
const char* const kNormGrads[kNormInputs] = {"dx", "dy", "dpost_gain", "dgate", "dscale", "dpre_gain"};

struct NormCall {
  const at::Tensor* t[kNormInputs] = {};
  muon_matrix m[kNormInputs];
  muon_norm_params params;
  const muon_matrix* at(int i) const { return t[i] ? m + i : nullptr; }
};

bool same_shape(const at::Tensor& t, const char* what, const at::Tensor& x) {
  if (t.sizes() == x.sizes()) return true;
  PyErr_Format(PyExc_ValueError, "%s of shape %s beside x of %s", what, c10::str(t.sizes()).c_str(), c10::str(x.sizes()).c_str());
  return false;
}

bool norm_inputs(PyObject* inputs, long device, int post_norm, int pre_norm, double eps, NormCall& c) {
  if (PyTuple_GET_SIZE(inputs) != kNormInputs) {
    PyErr_SetString(PyExc_ValueError, "expected six inputs");
    return false;
  }
  for (int i = 0; i < kNormInputs; ++i) {
    PyObject* o = PyTuple_GET_ITEM(inputs, i);
    if (i && o == Py_None) continue;
    if (!(c.t[i] = tensor_of(o, kNormNames[i]))) return false;
  }
  if (c.t[1] && !same_shape(*c.t[1], "y", *c.t[0])) return false;
  // (rows alone would take a gate whose leading dimensions are y's in another order)
  const at::Tensor* gate = c.t[3];
  if (gate && gate->dim() > 1 && gate->numel() != gate->size(-1) && !same_shape(*gate, "gate", *c.t[0])) return false;
  for (int i = 0; i < kNormInputs; ++i)
    if (c.t[i] && !describe_rows(*c.t[i], kNormNames[i], device, c.m + i)) return false;
  c.params = muon_norm_params{c.at(2), c.at(5), c.at(3), c.at(4), post_norm, pre_norm, (float)eps};
  return true;
}

at::Tensor like(const at::Tensor& t, at::ScalarType type, long device) {
  return at::empty(t.sizes(), at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)device));
}

// residual_norm(entry, handle, device, inputs, post_norm, pre_norm, eps, dtype) -> (status, out or None, hidden or None)
PyObject* residual_norm_of(PyObject*, PyObject* args) {
  unsigned long long entry, handle;
  long device;
  PyObject *inputs, *dtype;
  int post_norm, pre_norm;
  double eps;
  if (!PyArg_ParseTuple(args, "KKlO!ppdO", &entry, &handle, &device, &PyTuple_Type, &inputs, &post_norm, &pre_norm, &eps, &dtype))
    return nullptr;
  if (dtype != Py_None && !THPDtype_Check(dtype)) {
    PyErr_Format(PyExc_TypeError, "dtype: expected a torch.dtype or None, got %s", Py_TYPE(dtype)->tp_name);
    return nullptr;
  }
  try {
    NormCall c;
    if (!norm_inputs(inputs, device, post_norm, pre_norm, eps, c)) return nullptr;
    at::Tensor out, hidden;
    muon_matrix m[2];
    if (c.t[1]) out = like(*c.t[0], c.t[0]->scalar_type(), device);
    if (pre_norm)
      hidden = like(*c.t[0], THPDtype_Check(dtype) ? ((THPDtype*)dtype)->scalar_type : (c.t[1] ? c.t[1] : c.t[0])->scalar_type(), device);
    if (out.defined() && !describe_rows(out, "out", device, m)) return nullptr;
    if (hidden.defined() && !describe_rows(hidden, "hidden", device, m + 1)) return nullptr;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = ((decltype(&residual_norm))entry)((muon_handle*)handle, c.m, c.at(1), &c.params, out.defined() ? m : nullptr,
                                                hidden.defined() ? m + 1 : nullptr);
    Py_END_ALLOW_THREADS
    return Py_BuildValue("(iNN)", status, THPVariable_Wrap(out), THPVariable_Wrap(hidden));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// residual_norm_grad(entry, handle, device, inputs, dout, dhidden, wanted, post_norm, pre_norm, eps) ->
// (status, the six inputs' gradients or None)
PyObject* residual_norm_grad_of(PyObject*, PyObject* args) {
  unsigned long long entry, handle;
  long device;
  PyObject *inputs, *into[2], *wanted;
  int post_norm, pre_norm;
  double eps;
  if (!PyArg_ParseTuple(args, "KKlO!OOO!ppd", &entry, &handle, &device, &PyTuple_Type, &inputs, &into[0], &into[1], &PyTuple_Type,
                        &wanted, &post_norm, &pre_norm, &eps))
    return nullptr;
  if (PyTuple_GET_SIZE(wanted) != kNormInputs) {
    PyErr_SetString(PyExc_ValueError, "expected six answers");
    return nullptr;
  }
  PyObject* grads = nullptr;
  try {
    NormCall c;
    const char* const names[2] = {"dout", "dhidden"};
    const at::Tensor* in[2] = {};
    muon_matrix m[2], of[kNormInputs];
    const muon_matrix* to[kNormInputs] = {};
    if (!norm_inputs(inputs, device, post_norm, pre_norm, eps, c)) return nullptr;
    for (int i = 0; i < 2; ++i) {
      if (into[i] == Py_None) continue;
      if (!(in[i] = tensor_of(into[i], names[i])) || !same_shape(*in[i], names[i], *c.t[0]) ||
          !describe_rows(*in[i], names[i], device, m + i))
        return nullptr;
    }
    grads = PyTuple_New(kNormInputs);
    if (!grads) return nullptr;
    for (int i = 0; i < kNormInputs; ++i) {
      at::Tensor g;
      const int want = c.t[i] ? PyObject_IsTrue(PyTuple_GET_ITEM(wanted, i)) : 0;
      if (want < 0) goto fail;
      if (want) {
        g = like(*c.t[i], c.t[i]->scalar_type(), device);
        if (!describe_rows(g, kNormGrads[i], device, of + i)) goto fail;
        to[i] = of + i;
      }
      PyObject* wrapped = THPVariable_Wrap(std::move(g));
      if (!wrapped) goto fail;
      PyTuple_SET_ITEM(grads, i, wrapped);
    }
    {
      const muon_norm_grads g{to[0], to[1], to[2], to[3], to[4], to[5]};
      int status;
      Py_BEGIN_ALLOW_THREADS
      status = ((decltype(&residual_norm_grad))entry)((muon_handle*)handle, c.m, c.at(1), &c.params, in[0] ? m : nullptr,
                                                       in[1] ? m + 1 : nullptr, &g);
      Py_END_ALLOW_THREADS
      return Py_BuildValue("(iN)", status, grads);
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
fail:
  Py_XDECREF(grads);
  return nullptr;
}

PyMethodDef methods[] = {
    {"empty", empty, METH_VARARGS, "A tensor on the GPU with the shape and type of others."},
    {"pack", pack, METH_VARARGS, "Descriptors of a list of tensors, as bytes."},
    {"pack_rows", pack_rows, METH_VARARGS, "Descriptors of tensors as rows, as bytes, and their address."},
    {"residual_norm", residual_norm_of, METH_VARARGS, "Results of residual_norm, after its status."},
    {"residual_norm_grad", residual_norm_grad_of, METH_VARARGS, "Gradients of residual_norm_grad, after its status."},
    {"leaf_elsewhere", leaf_elsewhere, METH_O, "Whether a leaf's gradient is added on another stream than the current one."},
    {"device_of", device_of, METH_O, "Index of the first tensor on a GPU, or -1."},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_describe", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__describe(void) { return PyModule_Create(&module); }
