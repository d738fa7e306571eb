// The call path of the operators' binding for sizes it has checked before
// (Python module _opcall, host code only).
//
// ops.py checks a call's tensors in Python and makes the C entry point's
// parameter struct from them. Everything those checks look at is in a call's
// key: the entry point, the plain arguments and every tensor's type, device,
// sizes and strides; no address and no value of a tensor. `remember` keeps the
// struct under that key, and `again` makes the same call for tensors of the same
// key without the checks: reading six tensors from Python took 2.5 us of a
// call's 6.8, reading them here takes 0.4 of 3.9 (the rest is the launch), where
// a decode step's kernel runs for 2 to 4 us. What shapes do not settle (a tensor
// that requires grad while grad mode is on, one with a forward-mode tangent,
// another current device, a view with a pending negation) is looked at in every
// call; `again` returns None for it, and for anything it does not know, and the
// checks speak. What a call writes gets a new version, as from torch's own
// in-place operations: its check of tensors saved for a backward pass relies on it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <string>
#include <unordered_map>

namespace {

constexpr int kMaxTensors = 7;
constexpr Py_ssize_t kMaxParams = 128;
constexpr size_t kMaxPlans = 2048;   // cleared when full

struct Plan {
  alignas(8) char params[kMaxParams];
  int64_t workspace;   // bytes of the last pointer, the call's own
  unsigned written;    // bit i: tensor i is written
};

std::unordered_map<std::string, Plan>& plans() {
  static std::unordered_map<std::string, Plan> map;   // used under the GIL
  return map;
}

struct Call {
  std::string key;
  void* ptr[kMaxTensors];
  int n = 0;
  c10::Device device = c10::kCPU;   // the tensors'

  void add(int64_t v) { key.append(reinterpret_cast<const char*>(&v), sizeof v); }

  // entry, device, plain arguments (a tuple of integers and None) and tensors
  // (or None) of a call; false: not one that this path takes
  bool read(PyObject* entry, int64_t device, PyObject* plain, PyObject* const* tensors, Py_ssize_t count) {
    key.clear();
    n = (int)count;
    if (count > kMaxTensors || !PyTuple_Check(plain)) return false;
    add(reinterpret_cast<intptr_t>(entry_address(entry)));
    add(device);
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(plain); ++i) {
      PyObject* v = PyTuple_GET_ITEM(plain, i);
      if (v == Py_None) {
        add(0);
        add(0);
      } else if (PyLong_Check(v)) {
        const int64_t x = PyLong_AsLongLong(v);
        if (x == -1 && PyErr_Occurred()) return false;
        add(1);
        add(x);
      } else {
        return false;
      }
    }
    const bool grad = c10::GradMode::is_enabled();
    const bool forward = c10::AutogradState::get_tls_state().get_fw_grad_mode();
    for (int i = 0; i < n; ++i) {
      if (tensors[i] == Py_None) {
        ptr[i] = nullptr;
        add(-1);
        continue;
      }
      if (!THPVariable_Check(tensors[i])) return false;
      const at::Tensor& t = THPVariable_Unpack(tensors[i]);
      if (t.layout() != c10::kStrided || t.get_device() != device || t.is_neg() || (grad && t.requires_grad())) return false;
      if (forward && t._fw_grad(0).defined()) return false;   // the only level there is
      const auto sizes = t.sizes();
      const auto strides = t.strides();
      add((int64_t)t.device().type() << 48 | (int64_t)t.scalar_type() << 32 | (int64_t)sizes.size());
      key.append(reinterpret_cast<const char*>(sizes.data()), sizes.size() * sizeof(int64_t));
      key.append(reinterpret_cast<const char*>(strides.data()), strides.size() * sizeof(int64_t));
      ptr[i] = t.data_ptr();
      if (ptr[i] == nullptr && t.numel() > 0) return false;   // a wrapper without memory would count as absent
      this->device = t.device();
    }
    return true;
  }

  static void* entry_address(PyObject* o) { return PyLong_AsVoidPtr(o); }
};

// One for the process: its key's storage is reused, under the GIL
Call& scratch() {
  static Call c;
  return c;
}

int32_t launch(void* entry, const void* p, void* const* a, int n, void* s) {
  using P = const void*;
  switch (n) {
    case 3: return reinterpret_cast<int32_t (*)(P, void*, void*, void*, void*)>(entry)(p, a[0], a[1], a[2], s);
    case 4: return reinterpret_cast<int32_t (*)(P, void*, void*, void*, void*, void*)>(entry)(p, a[0], a[1], a[2], a[3], s);
    case 5:
      return reinterpret_cast<int32_t (*)(P, void*, void*, void*, void*, void*, void*)>(entry)(p, a[0], a[1], a[2], a[3],
                                                                                               a[4], s);
    case 6:
      return reinterpret_cast<int32_t (*)(P, void*, void*, void*, void*, void*, void*, void*)>(entry)(
          p, a[0], a[1], a[2], a[3], a[4], a[5], s);
    default:
      return reinterpret_cast<int32_t (*)(P, void*, void*, void*, void*, void*, void*, void*, void*)>(entry)(
          p, a[0], a[1], a[2], a[3], a[4], a[5], a[6], s);
  }
}

// read() of Python arguments; 1 read, 0 not one for this path, -1 with an
// error set. What torch throws for tensors without strides or storage counts as
// the second: the checks say what is wrong with them.
int read_call(Call& c, PyObject* entry, PyObject* device, PyObject* plain, PyObject* const* tensors, Py_ssize_t count) {
  const int64_t d = PyLong_AsLongLong(device);
  if (d == -1 && PyErr_Occurred()) return -1;
  bool ok = false;
  try {
    ok = c.read(entry, d, plain, tensors, count);
  } catch (...) {
    ok = false;
  }
  PyErr_Clear();
  return ok ? 1 : 0;
}

// A new version for the tensors of `written` (none is kept of tensors made in
// inference mode). They were read before the call and are still referenced.
void new_versions(unsigned written, PyObject* const* tensors, int n) {
  for (int i = 0; i < n; ++i) {
    if (!(written >> i & 1) || tensors[i] == Py_None) continue;
    const at::Tensor& t = THPVariable_Unpack(tensors[i]);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }
}

// again(entry, device, stream, current, plain, *tensors) -> status, or None;
// False where the call takes a workspace and `current` does not say that the
// stream is the current one: it is allocated for the current stream
PyObject* again(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs < 8) {
    PyErr_SetString(PyExc_TypeError, "again(entry, device, stream, current, plain, *tensors): at least three tensors");
    return nullptr;
  }
  Call& c = scratch();
  const int got = read_call(c, args[0], args[1], args[4], args + 5, nargs - 5);
  if (got < 0) return nullptr;
  if (got == 0) Py_RETURN_NONE;
  const auto it = plans().find(c.key);
  if (it == plans().end()) Py_RETURN_NONE;
  void* const stream = PyLong_AsVoidPtr(args[2]);
  void* const entry = Call::entry_address(args[0]);
  if (PyErr_Occurred()) return nullptr;
  const Plan plan = it->second;   // copies: the GIL is given up during the call
  void* ptr[kMaxTensors];
  const int n = c.n;
  std::memcpy(ptr, c.ptr, sizeof ptr);
  at::Tensor workspace;
  if (plan.workspace > 0) {
    if (args[3] != Py_True) Py_RETURN_FALSE;
    try {
      workspace = at::empty({plan.workspace}, at::TensorOptions().dtype(at::kByte).device(c.device));
    } catch (...) {
      Py_RETURN_NONE;   // the call in Python meets the same and raises it
    }
    ptr[n - 1] = workspace.data_ptr();
  }
  int32_t status;
  Py_BEGIN_ALLOW_THREADS
  status = launch(entry, plan.params, ptr, n, stream);
  Py_END_ALLOW_THREADS
  if (status == 0) new_versions(plan.written, args + 5, n);
  return PyLong_FromLong(status);
}

// remember(params, entry, device, workspace, plain, *tensors, written=0): the
// struct's bytes for calls like this one, the bytes of workspace that they take
// (in the place of the last tensor), and which tensors they write (bit i: tensor i)
PyObject* remember(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* names) {
  const Py_ssize_t named = names ? PyTuple_GET_SIZE(names) : 0;
  if (nargs < 8 || !PyBytes_Check(args[0]) || PyBytes_GET_SIZE(args[0]) > kMaxParams || !PyLong_Check(args[3]) ||
      named > 1 || (named == 1 && PyUnicode_CompareWithASCIIString(PyTuple_GET_ITEM(names, 0), "written") != 0)) {
    PyErr_SetString(PyExc_TypeError, "remember(params, entry, device, workspace, plain, *tensors, written=0): bytes and "
                                     "at least three tensors");
    return nullptr;
  }
  Plan plan{};
  plan.workspace = PyLong_AsLongLong(args[3]);
  if (named) plan.written = (unsigned)PyLong_AsUnsignedLong(args[nargs]);
  if (PyErr_Occurred()) return nullptr;
  Call& c = scratch();
  const int got = read_call(c, args[1], args[2], args[4], args + 5, nargs - 5);
  if (got < 0) return nullptr;
  if (got == 0) Py_RETURN_FALSE;
  if (plans().size() >= kMaxPlans) plans().clear();
  std::memcpy(plan.params, PyBytes_AS_STRING(args[0]), (size_t)PyBytes_GET_SIZE(args[0]));
  try {
    plans()[c.key] = plan;
  } catch (...) {
    Py_RETURN_FALSE;   // no memory for it: the next call is checked again
  }
  Py_RETURN_TRUE;
}

PyMethodDef methods[] = {
    {"again", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(again)), METH_FASTCALL,
     "again(entry, device, stream, current, plain, *tensors): the call of a C entry point for sizes that were "
     "remembered; its status, None for a call that has to be checked, or False for one that takes a workspace on a "
     "stream that is not the current one."},
    {"remember", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(remember)), METH_FASTCALL | METH_KEYWORDS,
     "remember(params, entry, device, workspace, plain, *tensors, written=0): keep a checked call's parameter struct "
     "(bytes); bit i of written: tensor i is written."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_opcall", "Call path of the operators for sizes checked before.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__opcall() { return PyModule_Create(&module); }
