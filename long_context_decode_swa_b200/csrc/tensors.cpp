// tensors.cpp -- the tensor checks of binding.py in one native call (a CPython extension, _tensors).
//
// A call of the library passes up to 20 tensors, and checking one in Python (type, dtype, shape, device,
// contiguity, address) takes 0.4 us: 5 to 7 us of a call whose kernels may take 10. Here it takes
// 0.09 us a tensor. Nothing is computed and no GPU is touched.
#include <ATen/core/grad_mode.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

namespace {

std::string text(PyObject* o) {  // str(o), for messages
  PyObject* s = PyObject_Str(o);
  const char* c = s != nullptr ? PyUnicode_AsUTF8(s) : nullptr;
  std::string r = c != nullptr ? c : "?";
  if (c == nullptr) PyErr_Clear();
  Py_XDECREF(s);
  return r;
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

bool refuse(PyObject* type, PyObject* name, const std::string& why) {
  PyErr_SetString(type, (text(name) + ": " + why).c_str());
  return false;
}

// Whether t is a (with `dense`: contiguous, else: not part of a gradient that is being recorded) tensor of this dtype and
// shape on CUDA device `index`; sets the Python error if not.
bool check(PyObject* t, PyObject* name, PyObject* dtype, PyObject* shape, long index, bool dense) {
  if (!THPVariable_Check(t)) return refuse(PyExc_TypeError, name, "expected a torch.Tensor");
  if (!THPDtype_Check(dtype) || !PyTuple_Check(shape))
    return refuse(PyExc_TypeError, name, "a spec is (tensor, name, torch dtype, shape tuple)");
  const at::Tensor& x = THPVariable_Unpack(t);
  if (x.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type)
    return refuse(PyExc_TypeError, name, "expected " + text(dtype) + ", got another dtype: " + c10::toString(x.scalar_type()));
  if (x.layout() != at::kStrided) return refuse(PyExc_ValueError, name, "must be a dense (strided) tensor");
  if (!x.is_cuda() || x.get_device() != index)
    return refuse(PyExc_ValueError, name, "expected a tensor on cuda:" + std::to_string(index) + ", got " + x.device().str());
  const at::IntArrayRef s = x.sizes();
  bool same = (Py_ssize_t)s.size() == PyTuple_GET_SIZE(shape);
  for (size_t d = 0; same && d < s.size(); ++d) {
    const long long want = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, d));
    if (want == -1 && PyErr_Occurred()) return false;
    same = s[d] == want;
  }
  if (!same) return refuse(PyExc_ValueError, name, "expected shape " + text(shape) + ", got " + text(s));
  if (dense && !x.is_contiguous()) return refuse(PyExc_ValueError, name, "must be contiguous");
  if (!dense && x.requires_grad() && at::GradMode::is_enabled())
    return refuse(PyExc_ValueError, name, "requires a gradient, and the call records none (call it from an autograd.Function "
                  "or under torch.no_grad())");
  return true;
}

PyObject* strides_of(const at::Tensor& x) {
  PyObject* t = PyTuple_New(x.dim());
  for (int64_t d = 0; t != nullptr && d < x.dim(); ++d) {
    PyObject* v = PyLong_FromLongLong(x.stride(d));
    if (v == nullptr) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, d, v);
  }
  return t;
}

// The results of the specs: addresses, or with !dense an (address, strides) pair each.
PyObject* each(PyObject* const* args, Py_ssize_t n, bool dense) {
  if (n < 1) {
    PyErr_SetString(PyExc_TypeError, "expected (index, spec, ..)");
    return nullptr;
  }
  const long index = PyLong_AsLong(args[0]);
  if (index == -1 && PyErr_Occurred()) return nullptr;
  PyObject* out = PyTuple_New(n - 1);
  if (out == nullptr) return nullptr;
  try {
    for (Py_ssize_t i = 1; i < n; ++i) {
      PyObject* spec = args[i];
      if (!PyTuple_Check(spec) || PyTuple_GET_SIZE(spec) < 4) {
        PyErr_SetString(PyExc_TypeError, "a spec is (tensor, name, torch dtype, shape tuple)");
        Py_DECREF(out);
        return nullptr;
      }
      PyObject* t = PyTuple_GET_ITEM(spec, 0);
      PyObject* result = nullptr;
      if (t == Py_None && PyTuple_GET_SIZE(spec) > 4) {
        result = Py_NewRef(Py_None);
      } else if (check(t, PyTuple_GET_ITEM(spec, 1), PyTuple_GET_ITEM(spec, 2), PyTuple_GET_ITEM(spec, 3), index, dense)) {
        const at::Tensor& x = THPVariable_Unpack(t);
        result = PyLong_FromUnsignedLongLong(reinterpret_cast<unsigned long long>(x.const_data_ptr()));
        if (result != nullptr && !dense) {
          PyObject* strides = strides_of(x);
          PyObject* pair = strides != nullptr ? PyTuple_Pack(2, result, strides) : nullptr;
          Py_DECREF(result);
          Py_XDECREF(strides);
          result = pair;
        }
      }
      if (result == nullptr) {
        Py_DECREF(out);
        return nullptr;
      }
      PyTuple_SET_ITEM(out, i - 1, result);
    }
  } catch (const std::exception& e) {  // e.g. a tensor without storage
    Py_DECREF(out);
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  return out;
}

PyObject* addresses(PyObject*, PyObject* const* args, Py_ssize_t n) { return each(args, n, true); }
PyObject* strided(PyObject*, PyObject* const* args, Py_ssize_t n) { return each(args, n, false); }

PyMethodDef methods[] = {
    {"addresses", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(addresses)), METH_FASTCALL,
     "addresses(index, (tensor, name, dtype, shape[, optional]), ..) -> data pointers of contiguous tensors on CUDA "
     "device index; an optional tensor may be None"},
    {"strided", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(strided)), METH_FASTCALL,
     "strided(index, spec, ..) -> (data pointer, strides) of tensors that need not be contiguous; none may require a "
     "gradient that autograd would record"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
