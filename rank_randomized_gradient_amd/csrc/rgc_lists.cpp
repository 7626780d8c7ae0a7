// Checks and unpacks a list of torch tensors in one call, for the entry points
// that take many tensors: in Python five attributes of each of the six lists'
// tensors cost 1.6 us a tensor, 240 us for the gains of a 36-layer model, where
// the step's kernels take 21.
#include <torch/csrc/autograd/python_variable.h>

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
    {"disjoint", disjoint, METH_VARARGS, "Whether no written range meets another or a read one."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_rgc_lists", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rgc_lists(void) { return PyModule_Create(&kModule); }
