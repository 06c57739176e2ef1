// binding.cpp -- the Python binding's per-step calls in native code: the checks of train.py on tensors
// and lists of tensors, the results' allocation and the call into libcgtp (include/cgtp_train.h), whose
// entry points train.py hands over by address.
//
// A training step of a small model is bound by such marshalling: reading type, size, strides and address
// of one tensor costs about 0.4 us through the interpreter and a few ns here, and a step passes three lists
// of all parameters.
//
// Every function returns its results; the library's status (an int) where that is not CGTP_OK; or
// NotImplemented where an argument does not fit, and train.py then says which.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <vector>

#include "cgtp_train.h"

namespace {

decltype(&cgtp_resnorm_forward) lib_forward = nullptr;
decltype(&cgtp_resnorm_backward) lib_backward = nullptr;
decltype(&cgtp_adamw_step) lib_step = nullptr;
decltype(&cgtp_grad_norm) lib_norm = nullptr;
decltype(&cgtp_adamw_state_values) lib_values = nullptr;

// an argument that train.py has to explain
struct Misfit {};

at::ScalarType type_of(int64_t code) {
  return code == CGTP_F64 ? at::kDouble : code == CGTP_BF16 ? at::kBFloat16 : at::kFloat;
}

int64_t number(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Misfit();
  }
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Misfit();
  }
  return v;
}
void* address(PyObject* o) { return reinterpret_cast<void*>(static_cast<uintptr_t>(number(o))); }

// The device of a plan or optimizer.  Its tables are there, and the library launches on the current device: a call
// needs both to be the same, and every tensor there.
struct Device {
  int64_t index;
  explicit Device(PyObject* o) : index(number(o)) {
    if (c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice().index() != index) throw Misfit();
  }
};

const at::Tensor& tensor(PyObject* o, at::ScalarType type, const Device& device) {
  if (!THPVariable_Check(o)) throw Misfit();
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != device.index || t.scalar_type() != type || t.layout() != at::kStrided) throw Misfit();
  return t;
}

// rows [n, width], or a column range of wider ones
struct Rows {
  void* p = nullptr;
  int64_t ld = 0;
};
Rows rows(PyObject* o, at::ScalarType type, const Device& device, int64_t n, int64_t width) {
  if (o == Py_None) return {};
  const at::Tensor& t = tensor(o, type, device);
  if (t.dim() != 2 || t.size(0) != n || t.size(1) != width || (t.stride(1) != 1 && width > 1 && n > 0)) throw Misfit();
  if (n <= 1) return {t.data_ptr(), 0};
  if (t.stride(0) < width) throw Misfit();
  return {t.data_ptr(), t.stride(0)};
}
void* vector(PyObject* o, at::ScalarType type, const Device& device, int64_t width) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, type, device);
  if (t.dim() != 1 || t.size(0) != width || !t.is_contiguous()) throw Misfit();
  return t.data_ptr();
}

// `like` on its device, or a new tensor there
struct Result {
  PyObject* object;   // a new reference
  void* p = nullptr;
};
Result fresh(c10::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  at::Tensor t = at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
  void* p = t.data_ptr();
  return {THPVariable_Wrap(std::move(t)), p};
}

// new references that go where the call ends early
struct Held {
  std::vector<PyObject*> objects;
  PyObject* keep(PyObject* o) {
    objects.push_back(o);
    return o;
  }
  PyObject* none() {
    Py_INCREF(Py_None);
    return keep(Py_None);
  }
  PyObject* same(PyObject* o) {
    Py_INCREF(o);
    return keep(o);
  }
  PyObject* tuple() {
    PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(objects.size()));
    if (!t) return nullptr;
    for (size_t i = 0; i < objects.size(); ++i) PyTuple_SET_ITEM(t, static_cast<Py_ssize_t>(i), objects[i]);
    objects.clear();
    return t;
  }
  ~Held() {
    for (PyObject* o : objects) Py_XDECREF(o);
  }
};

// field i of a tuple of `size`
PyObject* field(PyObject* t, Py_ssize_t size, Py_ssize_t i) {
  if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != size) throw Misfit();
  return PyTuple_GET_ITEM(t, i);
}

// ResNormPlan._native
struct NormPlan {
  cgtp_resnorm handle;
  at::ScalarType stream, in, out, param;
  int64_t dim, chan;
  bool pre_norm, gated;
  Device device;
  explicit NormPlan(PyObject* t) : device(field(t, 10, 9)) {
    const auto at_ = [&](int i) { return PyTuple_GET_ITEM(t, i); };
    handle = static_cast<cgtp_resnorm>(address(at_(0)));
    stream = type_of(number(at_(1))), in = type_of(number(at_(2))), out = type_of(number(at_(3))), param = type_of(number(at_(4)));
    dim = number(at_(5)), chan = number(at_(6)), pre_norm = number(at_(7)), gated = number(at_(8));
  }
};

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Misfit&) {
    Py_RETURN_NOTIMPLEMENTED;
  } catch (...) {   // torch's allocator: torch.OutOfMemoryError and what else its own calls raise
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

// (plan, h, z, q, post, scale, pre, out, y, stream) -> (out, y)
PyObject* resnorm_forward(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    if (n_args != 10) throw Misfit();
    const NormPlan p(a[0]);
    PyObject* ref = a[1] != Py_None ? a[1] : a[2];
    const at::Tensor& like = tensor(ref, a[1] != Py_None ? p.stream : p.in, p.device);
    if (like.dim() != 2) throw Misfit();
    const int64_t n = like.size(0);
    const Rows h = rows(a[1], p.stream, p.device, n, p.dim), z = rows(a[2], p.in, p.device, n, p.dim), q = rows(a[3], p.in, p.device, n, p.chan);
    const void *post = vector(a[4], p.param, p.device, p.chan), *scale = vector(a[5], p.param, p.device, p.chan), *pre = vector(a[6], p.param, p.device, p.chan);
    Rows out = rows(a[7], p.stream, p.device, n, p.dim), y = rows(a[8], p.out, p.device, n, p.dim);
    Held held;
    if (a[2] == Py_None) {
      held.same(a[1]);
    } else if (a[7] == Py_None) {
      const Result r = fresh({n, p.dim}, p.stream, like);
      held.keep(r.object);
      out = {r.p, 0};
    } else {
      held.same(a[7]);
    }
    if (p.pre_norm && a[8] == Py_None) {
      const Result r = fresh({n, p.dim}, p.out, like);
      held.keep(r.object);
      y = {r.p, 0};
    } else {
      held.same(a[8]);
    }
    const cgtp_status s = lib_forward(p.handle, n, h.p, h.ld, z.p, z.ld, q.p, q.ld, post, scale, pre, out.p, out.ld, y.p, y.ld, address(a[9]));
    return s == CGTP_OK ? held.tuple() : PyLong_FromLong(s);
  });
}

// (plan, gout, gy, x, z, q, post, scale, pre, need_gh, outs, stream) -> (gh, gz, gq, gpost, gscale, gpre)
PyObject* resnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    if (n_args != 12) throw Misfit();
    const NormPlan p(a[0]);
    const at::Tensor& like = tensor(a[1] != Py_None ? a[1] : a[2], a[1] != Py_None ? p.stream : p.in, p.device);
    if (like.dim() != 2) throw Misfit();
    const int64_t n = like.size(0);
    const Rows gout = rows(a[1], p.stream, p.device, n, p.dim), gy = rows(a[2], p.in, p.device, n, p.dim), x = rows(a[3], p.stream, p.device, n, p.dim),
               z = rows(a[4], p.in, p.device, n, p.dim), q = rows(a[5], p.in, p.device, n, p.chan);
    const void* factors[3];
    for (int i = 0; i < 3; ++i) factors[i] = vector(a[6 + i], p.param, p.device, p.chan);
    Held held;
    Rows g[3];      // gh, gz, gq
    void* sums[3];  // gpost, gscale, gpre
    const at::ScalarType types[3] = {p.stream, p.out, p.out};
    const int64_t widths[3] = {p.dim, p.dim, p.chan};
    if (a[10] != Py_None) {
      if (!PyTuple_Check(a[10]) || PyTuple_GET_SIZE(a[10]) != 6) throw Misfit();
      for (int i = 0; i < 3; ++i) g[i] = rows(held.same(PyTuple_GET_ITEM(a[10], i)), types[i], p.device, n, widths[i]);
      for (int i = 0; i < 3; ++i) sums[i] = vector(held.same(PyTuple_GET_ITEM(a[10], 3 + i)), p.param, p.device, p.chan);
    } else {
      const bool wanted[3] = {PyObject_IsTrue(a[9]) == 1, a[4] != Py_None, a[4] != Py_None && p.gated};
      for (int i = 0; i < 3; ++i) {
        if (wanted[i]) {
          const Result r = fresh({n, widths[i]}, types[i], like);
          held.keep(r.object);
          g[i] = {r.p, 0};
        } else {
          held.none();
        }
      }
      for (int i = 0; i < 3; ++i) {
        sums[i] = nullptr;
        if (a[6 + i] != Py_None) {
          const Result r = fresh({p.chan}, p.param, like);
          held.keep(r.object);
          sums[i] = r.p;
        } else {
          held.none();
        }
      }
    }
    const cgtp_status s = lib_backward(p.handle, n, gout.p, gout.ld, gy.p, gy.ld, x.p, x.ld, z.p, z.ld, q.p, q.ld, factors[0], factors[1],
                                       factors[2], g[0].p, g[0].ld, g[1].p, g[1].ld, g[2].p, g[2].ld, sums[0], sums[1], sums[2],
                                       address(a[11]));
    return s == CGTP_OK ? held.tuple() : PyLong_FromLong(s);
  });
}

// AdamW._native
struct Optimizer {
  cgtp_adamw handle;
  at::ScalarType param, grad, state;
  int64_t state_numel, count;
  const int64_t* numel;
  bool eight;
  Device device;
  explicit Optimizer(PyObject* t) : device(field(t, 8, 7)) {
    const auto at_ = [&](int i) { return PyTuple_GET_ITEM(t, i); };
    handle = static_cast<cgtp_adamw>(address(at_(0)));
    param = type_of(number(at_(1))), grad = type_of(number(at_(2)));
    eight = number(at_(3));
    state = eight ? at::kByte : param;
    state_numel = number(at_(4)), count = number(at_(5));
    numel = static_cast<const int64_t*>(address(at_(6)));
  }
};

// addresses of a list of contiguous tensors with the optimizer's sizes; None stays null
void gather(PyObject* list, const Optimizer& o, at::ScalarType type, std::vector<void*>* out, const at::Tensor** first = nullptr) {
  const bool is_list = PyList_Check(list);
  if (!is_list && !PyTuple_Check(list)) throw Misfit();
  if ((is_list ? PyList_GET_SIZE(list) : PyTuple_GET_SIZE(list)) != o.count) throw Misfit();
  out->resize(static_cast<size_t>(o.count));
  for (int64_t i = 0; i < o.count; ++i) {
    PyObject* item = is_list ? PyList_GET_ITEM(list, i) : PyTuple_GET_ITEM(list, i);
    (*out)[i] = nullptr;
    if (item == Py_None) continue;
    const at::Tensor& t = tensor(item, type, o.device);
    if (t.numel() != o.numel[i] || !t.is_contiguous()) throw Misfit();
    (*out)[i] = t.data_ptr();
    if (first && !*first) *first = &t;
  }
}

struct StatePointers {
  void *m, *v, *m_exp, *v_exp;
  StatePointers(const Optimizer& o, PyObject* const* a) {
    if (a[0] == Py_None || a[1] == Py_None || (o.eight && (a[2] == Py_None || a[3] == Py_None))) throw Misfit();
    m = vector(a[0], o.state, o.device, o.state_numel), v = vector(a[1], o.state, o.device, o.state_numel);
    m_exp = o.eight ? vector(a[2], at::kByte, o.device, o.state_numel / 128) : nullptr;
    v_exp = o.eight ? vector(a[3], at::kByte, o.device, o.state_numel / 128) : nullptr;
  }
};

// (opt, params, grads, copies, m, v, m_exp, v_exp, lr, beta1, beta2, eps, weight_decay, step, seed, clip, stream) -> None
PyObject* adamw_step(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    if (n_args != 17) throw Misfit();
    const Optimizer o(a[0]);
    std::vector<void*> p, g, c;
    gather(a[1], o, o.param, &p);
    gather(a[2], o, o.grad, &g);
    if (a[3] != Py_None) gather(a[3], o, at::kBFloat16, &c);
    const StatePointers s(o, a + 4);
    const unsigned long long seed = PyLong_AsUnsignedLongLongMask(a[14]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw Misfit();
    }
    const cgtp_status r = lib_step(o.handle, p.data(), const_cast<const void* const*>(g.data()), a[3] == Py_None ? nullptr : c.data(), s.m,
                                   s.v, s.m_exp, s.v_exp, real(a[8]), real(a[9]), real(a[10]), real(a[11]), real(a[12]), number(a[13]),
                                   seed, vector(a[15], o.param, o.device, 2), address(a[16]));
    if (r != CGTP_OK) return PyLong_FromLong(r);
    Py_RETURN_NONE;
  });
}

// (opt, grads, max_norm, out, stream) -> out
PyObject* grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    if (n_args != 5) throw Misfit();
    const Optimizer o(a[0]);
    std::vector<void*> g;
    const at::Tensor* first = nullptr;
    gather(a[1], o, o.grad, &g, &first);
    Held held;
    void* out;
    PyObject* result;
    if (a[3] == Py_None) {
      if (!first) throw Misfit();
      const Result r = fresh({2}, o.param, *first);
      result = held.keep(r.object);
      out = r.p;
    } else {
      out = vector(a[3], o.param, o.device, 2);
      result = held.same(a[3]);
    }
    const cgtp_status r = lib_norm(o.handle, const_cast<const void* const*>(g.data()), real(a[2]), out, address(a[4]));
    if (r != CGTP_OK) return PyLong_FromLong(r);
    held.objects.clear();
    return result;
  });
}

// (opt, m, v, m_exp, v_exp, stream) -> (m, v)
PyObject* state_values(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    if (n_args != 6) throw Misfit();
    const Optimizer o(a[0]);
    const StatePointers s(o, a + 1);
    const at::Tensor& like = THPVariable_Unpack(a[1]);
    Held held;
    const Result m = fresh({o.state_numel}, at::kFloat, like);
    held.keep(m.object);
    const Result v = fresh({o.state_numel}, at::kFloat, like);
    held.keep(v.object);
    const cgtp_status r = lib_values(o.handle, s.m, s.v, s.m_exp, s.v_exp, static_cast<float*>(m.p), static_cast<float*>(v.p), address(a[5]));
    return r == CGTP_OK ? held.tuple() : PyLong_FromLong(r);
  });
}

// addresses of the library's entry points
PyObject* connect(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded([&]() -> PyObject* {
    if (n_args != 5) throw Misfit();
    lib_forward = reinterpret_cast<decltype(lib_forward)>(address(a[0]));
    lib_backward = reinterpret_cast<decltype(lib_backward)>(address(a[1]));
    lib_step = reinterpret_cast<decltype(lib_step)>(address(a[2]));
    lib_norm = reinterpret_cast<decltype(lib_norm)>(address(a[3]));
    lib_values = reinterpret_cast<decltype(lib_values)>(address(a[4]));
    Py_RETURN_NONE;
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F));
}

PyMethodDef methods[] = {{"connect", fast<connect>(), METH_FASTCALL, nullptr},
                         {"resnorm_forward", fast<resnorm_forward>(), METH_FASTCALL, nullptr},
                         {"resnorm_backward", fast<resnorm_backward>(), METH_FASTCALL, nullptr},
                         {"adamw_step", fast<adamw_step>(), METH_FASTCALL, nullptr},
                         {"grad_norm", fast<grad_norm>(), METH_FASTCALL, nullptr},
                         {"state_values", fast<state_values>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
