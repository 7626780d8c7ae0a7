// Checks and unpacks a list of torch tensors in one call, for the entry points
// that take many tensors: in Python five attributes of each of the six lists'
// tensors cost 1.6 us a tensor, 240 us for the gains of a 36-layer model, where
// the step's kernels take 21. And makes the several small outputs of a call, which
// cost a call of torch.empty each otherwise.
#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <algorithm>
#include <cstdint>
#include <vector>

namespace {

// pack(tensors, sizes, block) -> (pointers, sizes, dtype name, device index)
//   tensors: a list or tuple of dense tensors of one dtype on one device
//   sizes: None, or bytes of int64: tensor i must hold ceil(sizes[i] / block) elements
// pointers and sizes: bytes of uint64 and int64. None instead of the tuple if the tensors are not as described.
PyObject* pack(PyObject*, PyObject* args) {
  PyObject *list, *sizes;
  long long block;
  if (!PyArg_ParseTuple(args, "OOL", &list, &sizes, &block)) return nullptr;
  PyObject* fast = PySequence_Fast(list, "a list of tensors is wanted");
  if (!fast) return nullptr;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast);
  const int64_t* want = nullptr;
  bool good = n > 0;
  if (sizes != Py_None) {
    if (!PyBytes_Check(sizes) || PyBytes_GET_SIZE(sizes) != (Py_ssize_t)(n * sizeof(int64_t))) good = false;
    else want = reinterpret_cast<const int64_t*>(PyBytes_AS_STRING(sizes));
  }
  PyObject* pointers = PyBytes_FromStringAndSize(nullptr, n * 8);
  PyObject* counts = PyBytes_FromStringAndSize(nullptr, n * 8);
  if (!pointers || !counts) {
    Py_XDECREF(pointers), Py_XDECREF(counts), Py_DECREF(fast);
    return nullptr;
  }
  uint64_t* p = reinterpret_cast<uint64_t*>(PyBytes_AS_STRING(pointers));
  int64_t* c = reinterpret_cast<int64_t*>(PyBytes_AS_STRING(counts));
  at::ScalarType type = at::ScalarType::Undefined;
  at::Device device(at::kCPU);
  try {
    for (Py_ssize_t i = 0; good && i < n; ++i) {
      PyObject* o = PySequence_Fast_GET_ITEM(fast, i);
      if (!THPVariable_Check(o)) {
        good = false;
        break;
      }
      const at::Tensor& t = THPVariable_Unpack(o);
      if (!t.defined() || t.layout() != at::kStrided) {
        good = false;
        break;
      }
      if (i == 0) type = t.scalar_type(), device = t.device();
      c[i] = t.numel();
      good = t.scalar_type() == type && t.device() == device && t.is_contiguous() &&
             (!want || c[i] == (want[i] + block - 1) / block);
      if (good) p[i] = reinterpret_cast<uint64_t>(t.data_ptr());
    }
  } catch (const std::exception&) {  // e.g. a tensor without storage
    good = false;
  }
  Py_DECREF(fast);
  if (!good) {
    Py_DECREF(pointers), Py_DECREF(counts);
    Py_RETURN_NONE;
  }
  return Py_BuildValue("(NNsi)", pointers, counts, c10::toString(type), device.is_cuda() ? (int)device.index() : -1);
}

// pack_gradients(tensors) -> (pointers, sizes, types, bytes, device index)
//   tensors: a list or tuple of dense tensors on one device, each bf16 (type 0) or float32 (1)
// pointers and sizes as above, types: bytes of int32, bytes: of int64, each tensor's. None instead of the tuple if the tensors are not as described.
PyObject* pack_gradients(PyObject*, PyObject* list) {
  PyObject* fast = PySequence_Fast(list, "a list of tensors is wanted");
  if (!fast) return nullptr;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast);
  PyObject* pointers = PyBytes_FromStringAndSize(nullptr, n * 8);
  PyObject* counts = PyBytes_FromStringAndSize(nullptr, n * 8);
  PyObject* types = PyBytes_FromStringAndSize(nullptr, n * 4);
  PyObject* lengths = PyBytes_FromStringAndSize(nullptr, n * 8);
  if (!pointers || !counts || !types || !lengths) {
    Py_XDECREF(pointers), Py_XDECREF(counts), Py_XDECREF(types), Py_XDECREF(lengths), Py_DECREF(fast);
    return nullptr;
  }
  uint64_t* p = reinterpret_cast<uint64_t*>(PyBytes_AS_STRING(pointers));
  int64_t* c = reinterpret_cast<int64_t*>(PyBytes_AS_STRING(counts));
  int32_t* k = reinterpret_cast<int32_t*>(PyBytes_AS_STRING(types));
  int64_t* b = reinterpret_cast<int64_t*>(PyBytes_AS_STRING(lengths));
  at::Device device(at::kCPU);
  bool good = n > 0;
  try {
    for (Py_ssize_t i = 0; good && i < n; ++i) {
      PyObject* o = PySequence_Fast_GET_ITEM(fast, i);
      good = THPVariable_Check(o);
      if (!good) break;
      const at::Tensor& t = THPVariable_Unpack(o);
      good = t.defined() && t.layout() == at::kStrided;
      if (!good) break;
      if (i == 0) device = t.device();
      const at::ScalarType type = t.scalar_type();
      good = (type == at::kBFloat16 || type == at::kFloat) && t.device() == device && t.is_contiguous();
      if (!good) break;
      c[i] = t.numel();
      k[i] = type == at::kFloat;
      b[i] = c[i] * (type == at::kFloat ? 4 : 2);
      p[i] = reinterpret_cast<uint64_t>(t.data_ptr());
    }
  } catch (const std::exception&) {  // e.g. a tensor without storage
    good = false;
  }
  Py_DECREF(fast);
  if (!good) {
    Py_DECREF(pointers), Py_DECREF(counts), Py_DECREF(types), Py_DECREF(lengths);
    Py_RETURN_NONE;
  }
  return Py_BuildValue("(NNNNi)", pointers, counts, types, lengths, device.is_cuda() ? (int)device.index() : -1);
}

// fresh(like, dtype, shape, dtype, shape, ...) -> tuple of new dense tensors on like's device, their contents
// whatever the memory holds; shape: a tuple of integers, or None for None in the tensor's place
PyObject* fresh(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS  // torch's own exceptions, out of memory among them, as torch.empty raises them
  if (n < 1 || n % 2 == 0 || !THPVariable_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "a tensor, then pairs of a dtype and a shape are wanted");
    return nullptr;
  }
  const at::Device device = THPVariable_Unpack(args[0]).device();
  THPObjectPtr out(PyTuple_New(n / 2));
  if (!out) return nullptr;
  for (Py_ssize_t i = 0; i < n / 2; ++i) {
    PyObject *type = args[1 + 2 * i], *shape = args[2 + 2 * i];
    PyObject* made = Py_None;
    if (shape == Py_None) {
      Py_INCREF(Py_None);
    } else {
      if (!THPDtype_Check(type) || !PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) > 4) {
        PyErr_SetString(PyExc_TypeError, "a dtype and a tuple of up to four integers are wanted");
        return nullptr;
      }
      int64_t sizes[4];
      const Py_ssize_t dims = PyTuple_GET_SIZE(shape);
      for (Py_ssize_t d = 0; d < dims; ++d) {
        sizes[d] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, d));
        if (PyErr_Occurred()) return nullptr;
      }
      made = THPVariable_Wrap(at::empty(at::IntArrayRef(sizes, dims),
                                        at::TensorOptions().dtype(reinterpret_cast<THPDtype*>(type)->scalar_type).device(device)));
      if (!made) return nullptr;
    }
    PyTuple_SET_ITEM(out.get(), i, made);
  }
  return out.release();
  END_HANDLE_TH_ERRORS
}

struct Range {
  uint64_t from, to;
  bool operator<(const Range& other) const { return from < other.from; }
};

// The ranges of a (pointers, counts, bytes of an element) triple that hold anything, in ascending order.
bool ranges_of(PyObject* triple, std::vector<Range>& out) {
  PyObject *pointers, *counts;
  long long size;
  if (!PyArg_ParseTuple(triple, "SSL", &pointers, &counts, &size)) return false;
  if (PyBytes_GET_SIZE(pointers) != PyBytes_GET_SIZE(counts)) {
    PyErr_SetString(PyExc_ValueError, "as many counts as pointers are wanted");
    return false;
  }
  const uint64_t* p = reinterpret_cast<const uint64_t*>(PyBytes_AS_STRING(pointers));
  const int64_t* c = reinterpret_cast<const int64_t*>(PyBytes_AS_STRING(counts));
  const Py_ssize_t n = PyBytes_GET_SIZE(pointers) / 8;
  const size_t first = out.size();
  for (Py_ssize_t i = 0; i < n; ++i)
    if (c[i] > 0) out.push_back({p[i], p[i] + (uint64_t)(c[i] * size)});
  if (!std::is_sorted(out.begin() + first, out.end())) std::sort(out.begin() + first, out.end());
  std::inplace_merge(out.begin(), out.begin() + first, out.end());
  return true;
}

// disjoint(read, written, written, ...) -> whether no written range meets another or a read one; each a tuple
// (pointers, counts, bytes of an element) as pack gives the first two
PyObject* disjoint(PyObject*, PyObject* args) {
  const Py_ssize_t lists = PyTuple_GET_SIZE(args);
  bool yes = true;
  try {
    std::vector<Range> read, written;
    for (Py_ssize_t i = 0; i < lists; ++i) {
      PyObject* t = PyTuple_GET_ITEM(args, i);
      if (!PyTuple_Check(t)) {
        PyErr_SetString(PyExc_TypeError, "tuples of pointers, counts and an element's bytes are wanted");
        return nullptr;
      }
      if (!ranges_of(t, i == 0 ? read : written)) return nullptr;
    }
    for (size_t i = 1; i < written.size(); ++i) yes = yes && written[i - 1].to <= written[i].from;
    size_t w = 0;
    for (const Range& r : read) {  // (written ranges are ascending and apart here, or the answer is no already)
      while (w < written.size() && written[w].to <= r.from) ++w;
      yes = yes && (w == written.size() || r.to <= written[w].from);
    }
  } catch (const std::exception&) {
    return PyErr_NoMemory();
  }
  return PyBool_FromLong(yes);
}

PyMethodDef kMethods[] = {
    {"pack", pack, METH_VARARGS, "Addresses and sizes of a list of dense tensors of one type and device, or None."},
    {"pack_gradients", pack_gradients, METH_O, "Addresses, sizes, types and bytes of a list of dense bf16 and float32 tensors, or None."},
    {"fresh", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(fresh)), METH_FASTCALL, "Several new tensors on a tensor's device."},
    {"disjoint", disjoint, METH_VARARGS, "Whether no written range meets another or a read one."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_rgc_lists", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rgc_lists(void) { return PyModule_Create(&kModule); }
