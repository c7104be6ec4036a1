// ssm_tensors.cpp -- the host's part of the calls that take a list of tensors
// (ssm_grad_norm, ssm_grad_clip): a module that walks the list once and leaves
// what the C ABI wants of it, the addresses, sizes and types, in host arrays.
// A pass in Python for each of them, and for contiguity and device, cost 0.2 us
// a tensor and list, more than the kernels over hundreds of small tensors.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <exception>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ssm_scan.h"

namespace {

struct Ref {
  PyObject *p;
  explicit Ref(PyObject *q) : p(q) {}
  ~Ref() { Py_XDECREF(p); }
  Ref(const Ref &) = delete;
  Ref &operator=(const Ref &) = delete;
};

// What a list holds: something that the calls do not take, tensors of which
// some are not contiguous, contiguous tensors.
enum { kOther = 0, kStrided = 1, kDense = 2 };

// tensors(list or tuple, device index) -> (addresses, sizes, types, kind); the
// first three are bytes that hold uint64, int64 and int32 (ssm_dtype) elements,
// empty where the kind is kOther.
PyObject *tensors(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
  if (nargs != 2) {
    PyErr_SetString(PyExc_TypeError, "tensors(list, device index)");
    return nullptr;
  }
  const long device = PyLong_AsLong(args[1]);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  // a copy of its own: a tensor whose sizes are Python code could change the list
  const Ref list(PySequence_Tuple(args[0]));
  if (!list.p) return nullptr;
  const Py_ssize_t n = PyTuple_GET_SIZE(list.p);
  const Ref at(PyBytes_FromStringAndSize(nullptr, n * 8));
  const Ref sizes(PyBytes_FromStringAndSize(nullptr, n * 8));
  const Ref types(PyBytes_FromStringAndSize(nullptr, n * 4));
  if (!at.p || !sizes.p || !types.p) return nullptr;
  // the characters of a bytes object follow 32 bytes of an allocation
  uint64_t *const a = reinterpret_cast<uint64_t *>(PyBytes_AS_STRING(at.p));
  int64_t *const s = reinterpret_cast<int64_t *>(PyBytes_AS_STRING(sizes.p));
  int32_t *const d = reinterpret_cast<int32_t *>(PyBytes_AS_STRING(types.p));
  bool dense = true;
  try {
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject *const o = PyTuple_GET_ITEM(list.p, i);
      if (!THPVariable_Check(o)) return Py_BuildValue("yyyi", "", "", "", kOther);
      const at::Tensor &t = THPVariable_Unpack(o);
      const at::ScalarType type = t.scalar_type();
      if ((type != at::kFloat && type != at::kBFloat16) || t.layout() != at::kStrided ||
          t.get_device() != device)
        return Py_BuildValue("yyyi", "", "", "", kOther);
      a[i] = reinterpret_cast<uint64_t>(t.data_ptr());
      s[i] = t.numel();
      d[i] = type == at::kFloat ? SSM_DTYPE_F32 : SSM_DTYPE_BF16;
      dense = dense && t.is_contiguous();
    }
  } catch (const std::exception &e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  return Py_BuildValue("OOOi", at.p, sizes.p, types.p, dense ? kDense : kStrided);
}

PyMethodDef methods[] = {
    {"tensors", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tensors)),
     METH_FASTCALL,
     "tensors(list, device index): addresses, sizes and types of its tensors as bytes, and 2 if "
     "all are contiguous, 1 if some are not, 0 if the list holds something else than float32 and "
     "bfloat16 tensors of that device."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ssmtensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ssmtensors() { return PyModule_Create(&module); }
