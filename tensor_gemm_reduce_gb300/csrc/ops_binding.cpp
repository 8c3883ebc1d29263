// ops_binding.cpp -- Python entry of the operators that are called every step
// (include/gemm_rs_ops.h): checks the tensors, passes their addresses and the
// current stream to the library, and returns its status code.
//
// Checking and unpacking a call's 4 to 14 tensors took 8 to 11 us in Python,
// several times as long as the smallest operators run; here it takes well
// under 1 us.  Nothing of the operators is computed in this file.
#define PY_SSIZE_T_CLEAN
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdio>
#include <exception>
#include <initializer_list>
#include <string>

#include "../../include/gemm_rs_ops.h"

namespace {

constexpr int64_t kWorld = GEMM_RS_WORLD;

// A refusal: becomes a Python TypeError or ValueError.
struct Refused {
  PyObject* type;
  std::string what;
};
[[noreturn]] void value_error(const std::string& what) { throw Refused{PyExc_ValueError, what}; }
[[noreturn]] void type_error(const std::string& what) { throw Refused{PyExc_TypeError, what}; }

std::string text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}

// The tensors of one call: their buffers must be on the current device, and no
// output may overlap another buffer.
class Call {
 public:
  const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
  }
  void* in(PyObject* o, at::ScalarType type, at::IntArrayRef shape, const char* name) {
    return pointer(o, type, shape, name, false);
  }
  void* out(PyObject* o, at::ScalarType type, at::IntArrayRef shape, const char* name) {
    return pointer(o, type, shape, name, true);
  }
  // Contiguous CUDA memory of any type, at least `need` bytes; `written` as for an output.
  void* buffer(PyObject* o, size_t need, const char* name, bool written) {
    if (o == Py_None) value_error(std::string(name) + " is missing");
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda() || !t.is_contiguous() || t.nbytes() < need)
      value_error(std::string(name) + " must be at least " + std::to_string(need) +
                  " bytes of contiguous CUDA memory");
    return add(t, name, written);
  }
  // The given stream handle, or the current stream's.
  void* stream(PyObject* handle) {
    for (int i = 0; i < n_; ++i)
      for (int j = 0; j < i; ++j)
        if ((span_[i].written || span_[j].written) && span_[i].lo < span_[j].hi && span_[j].lo < span_[i].hi)
          value_error(std::string(span_[i].name) + " shares memory with " + span_[j].name);
    const c10::cuda::CUDAStream s = c10::cuda::getCurrentCUDAStream();
    if (device_ >= 0 && device_ != s.device_index())
      value_error("the tensors are on cuda:" + std::to_string(device_) + ", the current device is cuda:" +
                  std::to_string((int)s.device_index()));
    return handle == Py_None ? static_cast<void*>(s.stream()) : PyLong_AsVoidPtr(handle);
  }

 private:
  struct Span {
    const char *lo, *hi, *name;
    bool written;
  };
  Span span_[16];
  int n_ = 0, device_ = -1;

  void* pointer(PyObject* o, at::ScalarType type, at::IntArrayRef shape, const char* name, bool written) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type)
      type_error(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
      value_error(std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
    if (!t.is_cuda() || !t.is_contiguous()) value_error(std::string(name) + " must be a contiguous CUDA tensor");
    return add(t, name, written);
  }
  void* add(const at::Tensor& t, const char* name, bool written) {
    if (t.numel() == 0) return nullptr;
    if (device_ < 0) device_ = t.device().index();
    if (t.device().index() != device_) value_error(std::string(name) + " is on another device");
    void* p = t.data_ptr();
    const char* lo = static_cast<const char*>(p);
    span_[n_++] = Span{lo, lo + t.nbytes(), name, written};
    return p;
  }
};

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& body) {
  try {
    if (got != want) type_error("expected " + std::to_string(want) + " arguments, got " + std::to_string(got));
    const int rc = body();
    return PyErr_Occurred() ? nullptr : PyLong_FromLong(rc);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

constexpr at::ScalarType kB = at::kBFloat16, kF = at::kFloat, kU8 = at::kByte;

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error("scale and eps must be numbers");
  }
  return (float)v;
}

gemm_rs_norm_desc norm_desc(Call& c, PyObject* x, PyObject* gate, float scale, float eps) {
  const at::Tensor& t = c.tensor(x, "x");
  if (t.dim() != 2) value_error("x must have shape [M][D], got " + text(t.sizes()));
  gemm_rs_norm_desc d = {t.size(0), t.size(1), 0, scale, eps};
  if (gate != Py_None) {
    const at::Tensor& g = c.tensor(gate, "gate");
    if (g.dim() != 2 || g.size(1) != d.D || g.size(0) < 1 || d.M % g.size(0))
      value_error("gate must have shape [G][" + std::to_string(d.D) + "] with G a divisor of " +
                  std::to_string(d.M) + ", got " + text(g.sizes()));
    d.gate_rows = g.size(0);
  }
  return d;
}

// x, y, w_post, w_pre, gate, scale, eps, r, h, stats, stream
PyObject* norm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    Call c;
    const gemm_rs_norm_desc d = norm_desc(c, a[0], a[4], number(a[5]), number(a[6]));
    const int64_t rows[2] = {d.M, d.D}, col[1] = {d.D}, stat[2] = {2, d.M}, gr[2] = {d.gate_rows, d.D};
    void* x = c.in(a[0], kB, rows, "x");
    void* y = c.in(a[1], kB, rows, "y");
    void* w_post = c.in(a[2], kB, col, "w_post");
    void* w_pre = c.in(a[3], kB, col, "w_pre");
    void* gate = d.gate_rows ? c.in(a[4], kB, gr, "gate") : nullptr;
    void* r = c.out(a[7], kB, rows, "r");
    void* h = c.out(a[8], kB, rows, "h");
    void* stats = c.out(a[9], kF, stat, "stats");
    return gemm_rs_norm_forward(&d, x, y, gate, w_post, w_pre, r, h, stats, c.stream(a[10]));
  });
}

// dr, dh, x, y, w_post, w_pre, gate, stats, scale, dx, dy, dw_post, dw_pre, dgate, workspace, stream
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    Call c;
    const gemm_rs_norm_desc d = norm_desc(c, a[2], a[6], number(a[8]), 0.f);
    const int64_t rows[2] = {d.M, d.D}, col[1] = {d.D}, stat[2] = {2, d.M}, gr[2] = {d.gate_rows, d.D};
    void* dr = c.in(a[0], kB, rows, "dr");
    void* dh = c.in(a[1], kB, rows, "dh");
    void* x = c.in(a[2], kB, rows, "x");
    void* y = c.in(a[3], kB, rows, "y");
    void* w_post = c.in(a[4], kB, col, "w_post");
    void* w_pre = c.in(a[5], kB, col, "w_pre");
    void* gate = d.gate_rows ? c.in(a[6], kB, gr, "gate") : nullptr;
    void* stats = c.in(a[7], kF, stat, "stats");
    void* dx = c.out(a[9], kB, rows, "dx");
    void* dy = c.out(a[10], kB, rows, "dy");
    void* dw_post = c.out(a[11], kB, col, "dw_post");
    void* dw_pre = c.out(a[12], kB, col, "dw_pre");
    if ((a[13] != Py_None) != (d.gate_rows > 0)) value_error("dgate must be given with a gate, and only then");
    void* dgate = d.gate_rows ? c.out(a[13], kB, gr, "dgate") : nullptr;
    size_t need = 0;
    const int rc = gemm_rs_norm_workspace(&d, &need);
    if (rc) return rc;
    void* ws = c.buffer(a[14], need, "workspace", true);
    return gemm_rs_norm_backward(&d, dr, dh, x, y, gate, w_post, w_pre, stats, dx, dy, dgate, dw_post, dw_pre, ws,
                                 c.stream(a[15]));
  });
}

// A, codes, scales, restore, stream: save A into codes and scales, or restore it from them
PyObject* act8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&] {
    Call c;
    const bool restore = PyObject_IsTrue(a[3]) == 1;
    const at::Tensor& t = c.tensor(a[0], "A");
    if (t.dim() != 3 || t.size(0) != kWorld)
      value_error("A must have shape [8][M][K/8], got " + text(t.sizes()));
    const int64_t M = t.size(1), K = t.size(2) * kWorld;
    size_t code_bytes = 0, scale_bytes = 0;
    const int rc = gemm_rs_act8_layout(M, K, nullptr, &code_bytes, &scale_bytes);
    if (rc) return rc;
    void* A = restore ? c.out(a[0], kB, t.sizes(), "A") : c.in(a[0], kB, t.sizes(), "A");
    void* codes = c.buffer(a[1], code_bytes, "codes", !restore);
    void* scales = c.buffer(a[2], scale_bytes, "scales", !restore);
    void* st = c.stream(a[4]);
    return restore ? gemm_rs_act8_restore(M, K, codes, scales, A, st) : gemm_rs_act8_save(M, K, A, codes, scales, st);
  });
}

// plan handle, M, N, K, workspace bytes, dY, W, codes, scales, dA, dW, workspace, stream
PyObject* backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    Call c;
    gemm_rs_bwd_t plan = static_cast<gemm_rs_bwd_t>(PyLong_AsVoidPtr(a[0]));
    const int64_t M = PyLong_AsLongLong(a[1]), N = PyLong_AsLongLong(a[2]), K = PyLong_AsLongLong(a[3]);
    const size_t need = PyLong_AsSize_t(a[4]);
    if (!plan || PyErr_Occurred()) {
      PyErr_Clear();
      value_error("the plan is closed");
    }
    const int64_t dy_shape[2] = {M, N}, a_shape[3] = {kWorld, M, K / kWorld}, w_shape[3] = {kWorld, K / kWorld, N};
    void *W = nullptr, *dA = nullptr, *dW = nullptr, *codes = nullptr, *scales = nullptr;
    void* dY = c.in(a[5], kB, dy_shape, "dY");
    if (a[9] != Py_None) {
      W = c.in(a[6], kB, w_shape, "W");
      dA = c.out(a[9], kB, a_shape, "dA");
    }
    if (a[10] != Py_None) {
      size_t code_bytes = 0, scale_bytes = 0;
      const int rc = gemm_rs_act8_layout(M, K, nullptr, &code_bytes, &scale_bytes);
      if (rc) return rc;
      codes = c.buffer(a[7], code_bytes, "codes", false);
      scales = c.buffer(a[8], scale_bytes, "scales", false);
      dW = c.out(a[10], kB, w_shape, "dW");
    }
    void* ws = c.buffer(a[11], need, "workspace", true);
    return gemm_rs_bwd_run(plan, dY, W, codes, scales, dA, dW, ws, c.stream(a[12]));
  });
}

// x, N, K, group, has_zeros, packed weight, out, stream
PyObject* w4_matvec(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    Call c;
    const at::Tensor& t = c.tensor(a[0], "x");
    const int64_t N = PyLong_AsLongLong(a[1]), K = PyLong_AsLongLong(a[2]);
    const int group = (int)PyLong_AsLong(a[3]), zeros = PyObject_IsTrue(a[4]) == 1;
    size_t weight_bytes = 0;
    const int rc = gemm_rs_w4_bytes(N, K, group, zeros, &weight_bytes);
    if (rc) return rc;
    if (t.dim() != 3) value_error("x must have shape [8][M][K/8], got " + text(t.sizes()));
    const int64_t M = t.size(1), xs[3] = {kWorld, M, K / kWorld}, os[2] = {M, N};
    void* x = c.in(a[0], kB, xs, "x");
    void* w = c.buffer(a[5], weight_bytes, "weight", false);
    void* out = c.out(a[6], kB, os, "out");
    return gemm_rs_w4_run(M, N, K, group, zeros, x, w, out, c.stream(a[7]));
  });
}

PyMethodDef methods[] = {
    {"norm_forward", (PyCFunction)(void*)norm_forward, METH_FASTCALL, nullptr},
    {"norm_backward", (PyCFunction)(void*)norm_backward, METH_FASTCALL, nullptr},
    {"act8", (PyCFunction)(void*)act8, METH_FASTCALL, nullptr},
    {"backward", (PyCFunction)(void*)backward, METH_FASTCALL, nullptr},
    {"w4_matvec", (PyCFunction)(void*)w4_matvec, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops(void) { return PyModule_Create(&module); }
