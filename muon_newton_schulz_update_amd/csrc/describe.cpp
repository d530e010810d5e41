// Python extension `_describe`: packs lists of torch tensors into arrays of
// muon_matrix for the C ABI. Argument marshalling only, the same checks as the
// binding's Python code, natively: from Python each tensor costs about 0.6 us
// (shape, stride, type, device and pointer are a call each), which for the few
// dozen tensors of an optimizer's list is several times the GPU's work.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/Functions.h>
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

PyMethodDef methods[] = {
    {"empty", empty, METH_VARARGS, "A tensor on the GPU with the shape and type of others."},
    {"pack", pack, METH_VARARGS, "Descriptors of a list of tensors, as bytes."},
    {"device_of", device_of, METH_O, "Index of the first tensor on a GPU, or -1."},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_describe", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__describe(void) { return PyModule_Create(&module); }
