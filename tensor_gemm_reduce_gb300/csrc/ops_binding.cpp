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

// Whether the weight's scales are powers of two (e8m0), not fp32: which of the entries serves.
bool powers_of_two(Call& c, PyObject* scales) {
  const at::Tensor& t = c.tensor(scales, "the weight's scales");
  if (t.scalar_type() != kF && t.scalar_type() != at::ScalarType::Float8_e8m0fnu)
    type_error(std::string("the weight's scales must be Float or Float8_e8m0fnu, got ") + c10::toString(t.scalar_type()));
  return t.scalar_type() != kF;
}

// W, codes, scales, stream
PyObject* fp8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&] {
    Call c;
    const at::Tensor& t = c.tensor(a[0], "W");
    if ((t.dim() != 3 && t.dim() != 4) || t.size(-3) != kWorld)
      value_error("W must have shape [8][K/8][N] or [E][8][K/8][N], got " + text(t.sizes()));
    const int64_t E = t.dim() == 4 ? t.size(0) : 1, N = t.size(-1), K = t.size(-2) * kWorld;
    const bool e8m0 = powers_of_two(c, a[2]);
    size_t code_bytes = 0, scale_bytes = 0;
    const int rc = (e8m0 ? gemm_rs_fp8_weight_bytes_e8m0 : gemm_rs_fp8_weight_bytes)(E, N, K, &code_bytes, &scale_bytes);
    if (rc) return rc;
    void* W = c.in(a[0], kB, t.sizes(), "W");
    void* codes = c.buffer(a[1], code_bytes, "the weight's codes", true);
    void* scales = c.buffer(a[2], scale_bytes, "the weight's scales", true);
    return (e8m0 ? gemm_rs_fp8_quantize_e8m0 : gemm_rs_fp8_quantize)(E, N, K, W, codes, scales, c.stream(a[3]));
  });
}

// A, M, N, K, weight codes, weight scales, checkpoint codes, checkpoint scales, out, workspace, stream
PyObject* fp8_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    Call c;
    const int64_t M = PyLong_AsLongLong(a[1]), N = PyLong_AsLongLong(a[2]), K = PyLong_AsLongLong(a[3]);
    size_t need = 0, code_bytes = 0, scale_bytes = 0, ck_codes = 0, ck_scales = 0;
    const bool e8m0 = powers_of_two(c, a[5]);
    int rc = gemm_rs_fp8_workspace(M, N, K, &need);
    if (!rc) rc = (e8m0 ? gemm_rs_fp8_weight_bytes_e8m0 : gemm_rs_fp8_weight_bytes)(1, N, K, &code_bytes, &scale_bytes);
    if (!rc) rc = gemm_rs_fp8_checkpoint_bytes(M, K, &ck_codes, &ck_scales);
    if (rc) return rc;
    const int64_t as[3] = {kWorld, M, K / kWorld}, os[2] = {M, N};
    void* A = c.in(a[0], kB, as, "A");
    void* wc = c.buffer(a[4], code_bytes, "the weight's codes", false);
    void* ws = c.buffer(a[5], scale_bytes, "the weight's scales", false);
    void* cc = a[6] == Py_None ? nullptr : c.buffer(a[6], ck_codes, "the checkpoint's codes", true);
    void* cs = a[7] == Py_None ? nullptr : c.buffer(a[7], ck_scales, "the checkpoint's scales", true);
    void* out = c.out(a[8], kB, os, "out");
    void* work = c.buffer(a[9], need, "workspace", true);
    return (e8m0 ? gemm_rs_fp8_forward_e8m0 : gemm_rs_fp8_forward)(M, N, K, A, wc, ws, cc, cs, out, work, c.stream(a[10]));
  });
}

// dY, M, N, K, weight codes, weight scales, checkpoint codes, checkpoint scales, dA, dW, workspace, stream
PyObject* fp8_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    Call c;
    const int64_t M = PyLong_AsLongLong(a[1]), N = PyLong_AsLongLong(a[2]), K = PyLong_AsLongLong(a[3]);
    size_t need = 0, code_bytes = 0, scale_bytes = 0, ck_codes = 0, ck_scales = 0;
    const bool e8m0 = powers_of_two(c, a[5]);
    int rc = gemm_rs_fp8_workspace(M, N, K, &need);
    if (!rc) rc = (e8m0 ? gemm_rs_fp8_weight_bytes_e8m0 : gemm_rs_fp8_weight_bytes)(1, N, K, &code_bytes, &scale_bytes);
    if (!rc) rc = gemm_rs_fp8_checkpoint_bytes(M, K, &ck_codes, &ck_scales);
    if (rc) return rc;
    const int64_t ys[2] = {M, N}, as[3] = {kWorld, M, K / kWorld}, ws_[3] = {kWorld, K / kWorld, N};
    void *wc = nullptr, *ws = nullptr, *cc = nullptr, *cs = nullptr, *dA = nullptr, *dW = nullptr;
    void* dY = c.in(a[0], kB, ys, "dY");
    if (a[8] != Py_None) {
      wc = c.buffer(a[4], code_bytes, "the weight's codes", false);
      ws = c.buffer(a[5], scale_bytes, "the weight's scales", false);
      dA = c.out(a[8], kB, as, "dA");
    }
    if (a[9] != Py_None) {
      cc = c.buffer(a[6], ck_codes, "the checkpoint's codes", false);
      cs = c.buffer(a[7], ck_scales, "the checkpoint's scales", false);
      dW = c.out(a[9], kB, ws_, "dW");
    }
    void* work = c.buffer(a[10], need, "workspace", true);
    return (e8m0 ? gemm_rs_fp8_backward_e8m0 : gemm_rs_fp8_backward)(M, N, K, dY, wc, ws, cc, cs, dA, dW, work,
                                                                     c.stream(a[11]));
  });
}

constexpr at::ScalarType kI = at::kInt;

int32_t int32_of(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  return v < INT32_MIN ? INT32_MIN : v > INT32_MAX ? INT32_MAX : (int32_t)v;
}

gemm_rs_route_desc route_desc(Call& c, PyObject* logits, PyObject* const* options) {
  const at::Tensor& t = c.tensor(logits, "logits");
  if (t.dim() != 2) value_error("logits must have shape [T][E], got " + text(t.sizes()));
  if (t.scalar_type() != kB && t.scalar_type() != kF)
    type_error(std::string("logits must be Float or BFloat16, got ") + c10::toString(t.scalar_type()));
  gemm_rs_route_desc d = {t.size(0), t.size(1), int32_of(options[0]), t.scalar_type() == kB,
                          int32_of(options[1]), int32_of(options[2]),
                          int32_of(options[3]), PyObject_IsTrue(options[4]) == 1,
                          (float)PyFloat_AsDouble(options[5])};
  if (PyErr_Occurred()) {
    PyErr_Clear();
    type_error("top_k, groups and top_groups must be integers, scale a number");
  }
  return d;
}

// logits, bias, mask, top_k, score, groups, top_groups, renormalize, scale, ids, weights, rows, pairs, offsets, stream
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    Call c;
    const gemm_rs_route_desc d = route_desc(c, a[0], a + 3);
    const int64_t ls[2] = {d.T, d.E}, ks[2] = {d.T, d.top_k}, ps[1] = {d.T * d.top_k}, os[1] = {d.E + 1}, es[1] = {d.E},
                  ts[1] = {d.T};
    void* logits = c.in(a[0], d.logits_bf16 ? kB : kF, ls, "logits");
    void* bias = a[1] == Py_None ? nullptr : c.in(a[1], kF, es, "bias");
    void* mask = a[2] == Py_None ? nullptr : c.in(a[2], at::kBool, ts, "mask");
    void* ids = c.out(a[9], kI, ks, "ids");
    void* weights = c.out(a[10], kF, ks, "weights");
    void* rows = c.out(a[11], kI, ks, "rows");
    void* pairs = c.out(a[12], kI, ps, "pairs");
    void* offsets = c.out(a[13], kI, os, "offsets");
    return gemm_rs_moe_route(&d, logits, bias, mask, ids, weights, rows, pairs, offsets, c.stream(a[14]));
  });
}

// dweights, logits, ids, top_k, score, groups, top_groups, renormalize, scale, dlogits, stream
PyObject* moe_route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    Call c;
    const gemm_rs_route_desc d = route_desc(c, a[1], a + 3);
    const int64_t ls[2] = {d.T, d.E}, ks[2] = {d.T, d.top_k};
    void* dweights = c.in(a[0], kF, ks, "dweights");
    void* logits = c.in(a[1], d.logits_bf16 ? kB : kF, ls, "logits");
    void* ids = c.in(a[2], kI, ks, "ids");
    void* dlogits = c.out(a[9], d.logits_bf16 ? kB : kF, ls, "dlogits");
    return gemm_rs_moe_route_backward(&d, dweights, logits, ids, dlogits, c.stream(a[10]));
  });
}

// ids, E, rows, pairs, offsets, stream
PyObject* moe_arrange(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    Call c;
    const at::Tensor& t = c.tensor(a[0], "ids");
    if (t.dim() != 2) value_error("ids must have shape [T][top_k], got " + text(t.sizes()));
    const int64_t E = PyLong_AsLongLong(a[1]), T = t.size(0), k = t.size(1);
    const int64_t ks[2] = {T, k}, ps[1] = {T * k}, os[1] = {E + 1};
    void* ids = c.in(a[0], kI, ks, "ids");
    void* rows = c.out(a[2], kI, ks, "rows");
    void* pairs = c.out(a[3], kI, ps, "pairs");
    void* offsets = c.out(a[4], kI, os, "offsets");
    return gemm_rs_moe_arrange(T, E, k, ids, rows, pairs, offsets, c.stream(a[5]));
  });
}

gemm_rs_moe_desc moe_desc(PyObject* const* a) {
  return {PyLong_AsLongLong(a[0]), PyLong_AsLongLong(a[1]), PyLong_AsLongLong(a[2]), PyLong_AsLongLong(a[3]),
          PyLong_AsLongLong(a[4])};
}

// A, T, E, top_k, N, K, weight codes, weight scales, weights, rows, offsets, checkpoint codes, scales and y, out,
// workspace, stream
PyObject* moe_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&] {
    Call c;
    const gemm_rs_moe_desc d = moe_desc(a + 1);
    size_t need = 0, code_bytes = 0, scale_bytes = 0, ck_codes = 0, ck_scales = 0, ck_y = 0;
    const bool e8m0 = powers_of_two(c, a[7]);
    int rc = gemm_rs_moe_workspace(&d, &need);
    if (!rc) rc = (e8m0 ? gemm_rs_fp8_weight_bytes_e8m0 : gemm_rs_fp8_weight_bytes)(d.E, d.N, d.K, &code_bytes, &scale_bytes);
    if (!rc) rc = gemm_rs_moe_checkpoint_bytes(&d, &ck_codes, &ck_scales, &ck_y);
    if (rc) return rc;
    const int64_t as[3] = {kWorld, d.T * d.top_k, d.K / kWorld}, ks[2] = {d.T, d.top_k}, es[1] = {d.E + 1},
                  os[2] = {d.T, d.N};
    void* A = c.in(a[0], kB, as, "A");
    void* wc = c.buffer(a[6], code_bytes, "the weight's codes", false);
    void* ws = c.buffer(a[7], scale_bytes, "the weight's scales", false);
    void* weights = c.in(a[8], kF, ks, "weights");
    void* rows = c.in(a[9], kI, ks, "rows");
    void* offsets = c.in(a[10], kI, es, "offsets");
    const bool keep = a[11] != Py_None;
    void* cc = keep ? c.buffer(a[11], ck_codes, "the checkpoint's codes", true) : nullptr;
    void* cs = keep ? c.buffer(a[12], ck_scales, "the checkpoint's scales", true) : nullptr;
    void* cy = keep ? c.buffer(a[13], ck_y, "the checkpoint's y", true) : nullptr;
    void* out = c.out(a[14], kB, os, "out");
    void* work = c.buffer(a[15], need, "workspace", true);
    return (e8m0 ? gemm_rs_moe_forward_e8m0 : gemm_rs_moe_forward)(&d, A, wc, ws, weights, rows, offsets, cc, cs, cy, out,
                                                                   work, c.stream(a[16]));
  });
}

// dout, T, E, top_k, N, K, weight codes, weight scales, weights, rows, pairs, offsets, checkpoint codes, scales and y,
// dA, dW, dweights, workspace, stream
PyObject* moe_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 20, [&] {
    Call c;
    const gemm_rs_moe_desc d = moe_desc(a + 1);
    size_t need = 0, code_bytes = 0, scale_bytes = 0, ck_codes = 0, ck_scales = 0, ck_y = 0;
    const bool e8m0 = powers_of_two(c, a[7]);
    int rc = gemm_rs_moe_workspace(&d, &need);
    if (!rc) rc = (e8m0 ? gemm_rs_fp8_weight_bytes_e8m0 : gemm_rs_fp8_weight_bytes)(d.E, d.N, d.K, &code_bytes, &scale_bytes);
    if (!rc) rc = gemm_rs_moe_checkpoint_bytes(&d, &ck_codes, &ck_scales, &ck_y);
    if (rc) return rc;
    const int64_t P = d.T * d.top_k, ds[2] = {d.T, d.N}, ks[2] = {d.T, d.top_k}, ps[1] = {P}, es[1] = {d.E + 1},
                  as[3] = {kWorld, P, d.K / kWorld}, ws_[4] = {d.E, kWorld, d.K / kWorld, d.N};
    void *wc = nullptr, *ws = nullptr, *cc = nullptr, *cs = nullptr, *cy = nullptr;
    void *dA = nullptr, *dW = nullptr, *dw = nullptr;
    void* dout = c.in(a[0], kB, ds, "dout");
    void* weights = c.in(a[8], kF, ks, "weights");
    void* rows = c.in(a[9], kI, ks, "rows");
    void* pairs = c.in(a[10], kI, ps, "pairs");
    void* offsets = c.in(a[11], kI, es, "offsets");
    if (a[15] != Py_None) {
      wc = c.buffer(a[6], code_bytes, "the weight's codes", false);
      ws = c.buffer(a[7], scale_bytes, "the weight's scales", false);
      dA = c.out(a[15], kB, as, "dA");
    }
    if (a[16] != Py_None) {
      cc = c.buffer(a[12], ck_codes, "the checkpoint's codes", false);
      cs = c.buffer(a[13], ck_scales, "the checkpoint's scales", false);
      dW = c.out(a[16], kB, ws_, "dW");
    }
    if (a[17] != Py_None) {
      cy = c.buffer(a[14], ck_y, "the checkpoint's y", false);
      dw = c.out(a[17], kF, ks, "dweights");
    }
    void* work = c.buffer(a[18], need, "workspace", true);
    return (e8m0 ? gemm_rs_moe_backward_e8m0 : gemm_rs_moe_backward)(&d, dout, wc, ws, weights, rows, pairs, offsets, cc, cs,
                                                                     cy, dA, dW, dw, work, c.stream(a[19]));
  });
}

PyMethodDef methods[] = {
    {"norm_forward", (PyCFunction)(void*)norm_forward, METH_FASTCALL, nullptr},
    {"norm_backward", (PyCFunction)(void*)norm_backward, METH_FASTCALL, nullptr},
    {"act8", (PyCFunction)(void*)act8, METH_FASTCALL, nullptr},
    {"backward", (PyCFunction)(void*)backward, METH_FASTCALL, nullptr},
    {"w4_matvec", (PyCFunction)(void*)w4_matvec, METH_FASTCALL, nullptr},
    {"fp8_quantize", (PyCFunction)(void*)fp8_quantize, METH_FASTCALL, nullptr},
    {"fp8_forward", (PyCFunction)(void*)fp8_forward, METH_FASTCALL, nullptr},
    {"fp8_backward", (PyCFunction)(void*)fp8_backward, METH_FASTCALL, nullptr},
    {"moe_route", (PyCFunction)(void*)moe_route, METH_FASTCALL, nullptr},
    {"moe_route_backward", (PyCFunction)(void*)moe_route_backward, METH_FASTCALL, nullptr},
    {"moe_arrange", (PyCFunction)(void*)moe_arrange, METH_FASTCALL, nullptr},
    {"moe_forward", (PyCFunction)(void*)moe_forward, METH_FASTCALL, nullptr},
    {"moe_backward", (PyCFunction)(void*)moe_backward, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops(void) { return PyModule_Create(&module); }
