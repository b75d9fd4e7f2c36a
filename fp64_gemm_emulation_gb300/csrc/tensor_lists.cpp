// tensor_lists.cpp -- what the C ABI wants to know of a list of torch tensors, gathered in one call.
//
// A Python module (_tensor_lists) for the binding alone: an entry point over hundreds of tensors needs five facts of each,
// and five attribute calls a tensor cost more than its kernels (600 tensors: a call of 360 us; with 7 us here, 50).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <vector>

namespace {

// OZ_BF16, OZ_F16, OZ_F32; 0 for any other type.
int code_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return 1;
    case at::kHalf: return 2;
    case at::kFloat: return 3;
    default: return 0;
  }
}

struct Gathered {
  std::vector<int32_t> codes;
  std::vector<int64_t> pointers, counts;
};

// False with a Python error set.  device: the index that all must have, or -1 before the first.
bool gather(PyObject* list, int64_t* device, Gathered* out) {
  const Py_ssize_t n = PyList_GET_SIZE(list);
  out->codes.reserve(n);
  out->pointers.reserve(n);
  out->counts.reserve(n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* item = PyList_GET_ITEM(list, i);
    if (!THPVariable_Check(item)) {
      PyErr_SetString(PyExc_TypeError, "gradients and outputs must be tensors");
      return false;
    }
    const at::Tensor& t = THPVariable_Unpack(item);
    if (!t.is_cuda() || t.layout() != at::kStrided || !t.is_contiguous() || (*device >= 0 && t.get_device() != *device)) {
      PyErr_SetString(PyExc_ValueError, "gradients and outputs must be contiguous CUDA tensors on one device");
      return false;
    }
    *device = t.get_device();
    const int code = code_of(t);
    if (!code) {
      PyErr_SetString(PyExc_TypeError, "dtype must be bfloat16, float16 or float32");
      return false;
    }
    out->codes.push_back(code);
    out->pointers.push_back(reinterpret_cast<int64_t>(t.data_ptr()));
    out->counts.push_back(t.numel());
  }
  return true;
}

template <class T>
PyObject* bytes_of(const std::vector<T>& v) {
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(v.data()), static_cast<Py_ssize_t>(v.size() * sizeof(T)));
}

// pairs(grads, outs) -> (device index, codes int32, pointers, output pointers, counts: int64 each, as bytes)
PyObject* pairs(PyObject*, PyObject* args) {
  PyObject *grads, *outs;
  if (!PyArg_ParseTuple(args, "O!O!", &PyList_Type, &grads, &PyList_Type, &outs)) return nullptr;
  try {
    int64_t device = -1;
    Gathered g, o;
    if (!gather(grads, &device, &g)) return nullptr;
    if (outs != grads) {
      if (!gather(outs, &device, &o)) return nullptr;
      if (o.codes != g.codes || o.counts != g.counts) {
        PyErr_SetString(PyExc_ValueError, "outputs must have their gradients' dtypes and numbers of elements");
        return nullptr;
      }
    }
    return Py_BuildValue("LNNNN", static_cast<long long>(device), bytes_of(g.codes), bytes_of(g.pointers),
                         bytes_of(outs == grads ? g.pointers : o.pointers), bytes_of(g.counts));
  } catch (const std::exception& e) {  // (a tensor without memory of its own)
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {{"pairs", pairs, METH_VARARGS, "What clipping needs of its gradients and outputs (lists of tensors)."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_lists", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_lists() { return PyModule_Create(&module); }
