// Python entry of the ragged-step calls: checks the tensors and passes their
// addresses, sizes and strides to libmla (include/mla.h).
//
// At decode sizes these kernels take two to four microseconds, and the same
// checks and a ctypes call in Python took 16 to 21 with the launch; here checks
// and launch take 3.2.  Every
// function returns the library's status, or kBadTensor without having called it
// when a tensor's type, device, shape or layout is not the call's; the caller
// (mla.py) then says which one.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>

#include "../../include/mla.h"

namespace {

constexpr long kBadTensor = 1;
constexpr int64_t kAny = -1;
struct Bad {};

// The tensors of one call: all on the device of the first, which has to be the
// current one.
class Args {
 public:
  Args(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
    if (n != want) throw Bad{};
  }
  bool none(int i) const { return a_[i] == Py_None; }
  // Argument i as a tensor of this type and shape (kAny: any size); `packed`:
  // contiguous, else with a contiguous last axis.
  const at::Tensor& tensor(int i, c10::ScalarType type, std::initializer_list<int64_t> shape, bool packed = true) {
    if (!THPVariable_Check(a_[i])) throw Bad{};
    const at::Tensor& t = THPVariable_Unpack(a_[i]);
    if (!t.is_cuda() || t.layout() != c10::kStrided || t.scalar_type() != type || t.dim() != (int64_t)shape.size())
      throw Bad{};
    if (dev_ < 0) {
      dev_ = t.get_device();
      if (dev_ != c10::cuda::current_device()) throw Bad{};
    } else if (t.get_device() != dev_) {
      throw Bad{};
    }
    const int64_t* size = t.sizes().data();
    for (int64_t want : shape) {
      if (want != kAny && want != *size) throw Bad{};
      ++size;
    }
    if (packed ? !t.is_contiguous() : (t.sizes().back() > 1 && t.strides().back() != 1)) throw Bad{};
    return t;
  }
  // The same, or null for None.
  void* maybe(int i, c10::ScalarType type, std::initializer_list<int64_t> shape) {
    return none(i) ? nullptr : tensor(i, type, shape).data_ptr();
  }
  // Any tensor's memory, contiguous.
  const at::Tensor& memory(int i) {
    if (!THPVariable_Check(a_[i])) throw Bad{};
    const at::Tensor& t = THPVariable_Unpack(a_[i]);
    if (!t.is_cuda() || t.layout() != c10::kStrided || t.get_device() != dev_ || !t.is_contiguous()) throw Bad{};
    return t;
  }
  // An address as a number.
  void* address(int i) const { return as_address(a_[i]); }
  int integer(int i) const {
    const long v = PyLong_AsLong(a_[i]);
    if ((v == -1 && PyErr_Occurred()) || v != (int)v) throw Bad{};
    return (int)v;
  }
  float real(int i) const {
    const double v = PyFloat_AsDouble(a_[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Bad{};
    return (float)v;
  }
  mla_dims dims(int i) const {
    Py_buffer b;
    if (PyObject_GetBuffer(a_[i], &b, PyBUF_SIMPLE)) throw Bad{};
    mla_dims d{};
    const bool ok = b.len == (Py_ssize_t)sizeof d;
    if (ok) d = *static_cast<const mla_dims*>(b.buf);
    PyBuffer_Release(&b);
    if (!ok) throw Bad{};
    return d;
  }
  // None: torch's current stream; a raw handle; or an object with one.
  cudaStream_t stream(int i) const {
    if (none(i)) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev_).stream();
    if (PyLong_Check(a_[i])) return static_cast<cudaStream_t>(as_address(a_[i]));
    PyObject* h = PyObject_GetAttrString(a_[i], "cuda_stream");
    if (!h) throw Bad{};
    void* p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!p && PyErr_Occurred()) throw Bad{};  // null is a stream, the legacy one
    return static_cast<cudaStream_t>(p);
  }

 private:
  static void* as_address(PyObject* o) {
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Bad{};
    return p;
  }
  PyObject* const* a_;
  int64_t dev_ = -1;
};

// The stride of an axis; of one with a single entry, any will do.
int64_t step_of(const at::Tensor& t, int axis, int64_t least) {
  return t.size(axis) > 1 ? t.stride(axis) : least;
}
template <class T>
T* ptr(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

c10::ScalarType type_of(const mla_dims& d) { return d.dtype == MLA_BF16 ? at::kBFloat16 : at::kFloat; }
int row_of(const mla_dims& d) { return d.d_c + (d.rope_key_per_head ? d.n_h : 1) * d.d_r; }

// Runs a call without the interpreter lock; anything that is not a status (a
// tensor that does not fit, an object of another kind) becomes kBadTensor.
template <class Call>
PyObject* status(Call call) {
  long s = kBadTensor;
  try {
    s = call();
  } catch (const Bad&) {
    PyErr_Clear();
  } catch (const std::exception&) {
    PyErr_Clear();
  }
  return PyLong_FromLong(s);
}
template <class Launch>
long unlocked(Launch launch) {
  PyThreadState* s = PyEval_SaveThread();
  const long r = launch();
  PyEval_RestoreThread(s);
  return r;
}

PyObject* plan_step(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return status([&]() -> long {
    Args a(args, n, 13);
    const auto i32 = at::kInt;
    const auto& new_len = a.tensor(0, i32, {kAny});
    const int64_t B = new_len.size(0);
    const auto& past = a.tensor(1, i32, {B});
    const auto& free = a.tensor(2, i32, {kAny});
    const auto& table = a.tensor(3, i32, {B, kAny});
    const int num_pages = a.integer(4);
    const auto& q_start = a.tensor(5, i32, {B + 1});
    const auto& kv_len = a.tensor(6, i32, {B});
    const auto& seq = a.tensor(7, i32, {kAny});
    const int64_t rows = seq.size(0);
    const auto& pos = a.tensor(8, i32, {rows});
    const auto& slot = a.tensor(9, at::kLong, {rows});
    const auto& counts = a.tensor(10, i32, {3});
    void* err = a.maybe(11, i32, {1});
    const cudaStream_t st = a.stream(12);
    if (B > INT_MAX || rows > INT_MAX || free.size(0) > INT_MAX || table.size(1) > INT_MAX) throw Bad{};
    return unlocked([&] {
      return mla_plan_step(ptr<int32_t>(new_len), ptr<int32_t>(past), (int)B, ptr<int32_t>(free), (int)free.size(0),
                           ptr<int32_t>(table), (int)table.size(1), num_pages, ptr<int32_t>(q_start),
                           ptr<int32_t>(kv_len), ptr<int32_t>(seq), ptr<int32_t>(pos), ptr<int64_t>(slot), (int)rows,
                           ptr<int32_t>(counts), static_cast<int32_t*>(err), st);
    });
  });
}

PyObject* append_normed(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return status([&]() -> long {
    Args a(args, n, 12);
    const mla_dims d = a.dims(0);
    const auto dt = type_of(d);
    const auto& kv = a.tensor(1, dt, {kAny, row_of(d)}, false);
    const int64_t T = kv.size(0);
    void* kv_gamma = a.maybe(2, dt, {d.d_c});
    const auto& pos = a.tensor(3, at::kInt, {T});
    const auto& slot = a.tensor(4, at::kLong, {T});
    const auto& cache = a.tensor(5, dt, {kAny, d.page_size, row_of(d)});
    const float eps = a.real(6);
    const void* cq = nullptr;
    void* cq_out = nullptr;
    int64_t cs = 0, os = 0;
    if (a.none(7) != a.none(9)) throw Bad{};
    if (!a.none(7)) {
      const auto& x = a.tensor(7, dt, {T, d.d_cq}, false);
      const auto& y = a.tensor(9, dt, {T, d.d_cq}, false);
      cq = x.data_ptr();
      cq_out = y.data_ptr();
      cs = step_of(x, 0, d.d_cq);
      os = step_of(y, 0, d.d_cq);
    }
    void* cq_gamma = a.maybe(8, dt, {d.d_cq});
    void* err = a.maybe(10, at::kInt, {1});
    const cudaStream_t st = a.stream(11);
    if (T > INT_MAX || cache.size(0) > INT_MAX) throw Bad{};
    return unlocked([&] {
      return mla_append_normed(&d, kv.data_ptr(), step_of(kv, 0, row_of(d)), kv_gamma, cq, cs, cq_gamma, cq_out, os, eps,
                               ptr<int32_t>(pos), ptr<int64_t>(slot), cache.data_ptr(), (int)cache.size(0), (int)T,
                               static_cast<int32_t*>(err), st);
    });
  });
}

PyObject* query_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return status([&]() -> long {
    Args a(args, n, 8);
    const mla_dims d = a.dims(0);
    const auto dt = type_of(d);
    const int64_t dq = (int64_t)d.d_h + d.d_r;
    const auto& q = a.tensor(1, dt, {kAny, d.n_h, dq}, false);
    const int64_t T = q.size(0);
    if (d.n_h > 1 && q.stride(1) != dq) throw Bad{};
    void* gamma = a.maybe(2, dt, {d.d_h});
    const auto& pos = a.tensor(3, at::kInt, {T});
    const auto& qc = a.tensor(4, dt, {T, d.n_h, d.d_h}, false);
    const auto& qr = a.tensor(5, dt, {T, d.n_h, d.d_r}, false);
    const float eps = a.real(6);
    const cudaStream_t st = a.stream(7);
    const int64_t ch = step_of(qc, 1, d.d_h), rh = step_of(qr, 1, d.d_r);
    if (T > INT_MAX) throw Bad{};
    return unlocked([&] {
      return mla_query_norm_rope(&d, q.data_ptr(), step_of(q, 0, d.n_h * dq), gamma, eps, ptr<int32_t>(pos),
                                 qc.data_ptr(), step_of(qc, 0, d.n_h * ch), ch, qr.data_ptr(),
                                 step_of(qr, 0, d.n_h * rh), rh, (int)T, st);
    });
  });
}

PyObject* attend_ragged(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return status([&]() -> long {
    Args a(args, n, 10);
    const mla_dims d = a.dims(0);
    const auto dt = type_of(d);
    const int64_t row = (int64_t)d.d_c + d.d_r;
    const auto& q = a.tensor(1, dt, {kAny, d.n_h, row}, false);
    const int64_t T = q.size(0);
    const auto& kv_len = a.tensor(3, at::kInt, {kAny});
    const int64_t B = kv_len.size(0);
    const auto& q_start = a.tensor(2, at::kInt, {B + 1});
    const auto& table = a.tensor(4, at::kInt, {B, kAny});
    const auto& cache = a.tensor(5, dt, {kAny, d.page_size, row});
    const auto& out = a.tensor(6, dt, {T, d.n_h, d.d_c});
    void* lse = a.maybe(7, at::kFloat, {T, d.n_h});
    const auto& ws = a.memory(8);
    const cudaStream_t st = a.stream(9);
    const int64_t hs = step_of(q, 1, row);
    if (T > INT_MAX || B > INT_MAX || cache.size(0) > INT_MAX || table.size(1) > INT_MAX) throw Bad{};
    return unlocked([&] {
      return mla_attend_ragged(&d, q.data_ptr(), step_of(q, 0, d.n_h * hs), hs, ptr<int32_t>(q_start),
                               ptr<int32_t>(kv_len), ptr<int32_t>(table), (int)table.size(1), (int)cache.size(0),
                               cache.data_ptr(), out.data_ptr(), static_cast<float*>(lse), (int)B, (int)T,
                               ws.data_ptr(), ws.nbytes(), st);
    });
  });
}

PyObject* ragged_step(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return status([&]() -> long {
    Args a(args, n, 13);
    const auto* w = static_cast<const mla_weights*>(a.address(0));
    mla_dims d{};
    if (const mla_status s = mla_weights_dims(w, &d)) return s;
    const auto dt = type_of(d);
    const auto i32 = at::kInt;
    const auto& h = a.tensor(2, dt, {kAny, d.d_model});
    const int64_t T = h.size(0);
    a.memory(1);  // the weights' buffer, on the tensors' device
    const auto& kv_len = a.tensor(4, i32, {kAny});
    const int64_t B = kv_len.size(0);
    const auto& q_start = a.tensor(3, i32, {B + 1});
    const auto& seq = a.tensor(5, i32, {T});
    const auto& pos = a.tensor(6, i32, {T});
    const auto& table = a.tensor(7, i32, {B, kAny});
    const int num_pages = a.integer(8);
    const auto& cache = a.tensor(9, dt, {kAny, d.page_size, row_of(d)});
    const auto& out = a.tensor(10, at::kFloat, {T, d.n_h, d.d_v});
    const auto& ws = a.memory(11);
    const cudaStream_t st = a.stream(12);
    if (T > INT_MAX || B > INT_MAX || table.size(1) > INT_MAX || num_pages > cache.size(0)) throw Bad{};
    return unlocked([&] {
      return mla_ragged_step(w, h.data_ptr(), ptr<int32_t>(q_start), ptr<int32_t>(kv_len), ptr<int32_t>(seq),
                             ptr<int32_t>(pos), ptr<int32_t>(table), (int)table.size(1), num_pages, cache.data_ptr(),
                             ptr<float>(out), (int)B, (int)T, ws.data_ptr(), ws.nbytes(), st);
    });
  });
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(plan_step), ENTRY(append_normed), ENTRY(query_norm_rope), ENTRY(attend_ragged),
                         ENTRY(ragged_step), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ragged", "Ragged-step calls of libmla on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ragged(void) { return PyModule_Create(&module); }
