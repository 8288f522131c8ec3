// Argument marshalling of the entry points whose smallest calls run for a few
// microseconds, as a Python extension module: torch tensors in, raw device
// pointers, sizes and enum codes out, one call of the C entry point.  With the same
// checks in Python, the norm of one row of 4096 took 7.9 us a call; it takes 4.6.
//
// Every function takes (current device, stream handle, operands...) positionally and
// returns the entry point's status (0 or negative), or 1 + the operands' device where
// that is not the current one (nothing is called then).  Wrong operands raise
// ValueError or TypeError.  The entry points' addresses come from the library that the
// package has loaded (bind), so both always call the same one.
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "fp8mi.h"

namespace {

struct Raised {};  // a Python error is set

[[noreturn]] void raise(PyObject* type, const char* format, const char* a, const char* b = "", const char* c = "") {
  PyErr_Format(type, format, a, b, c);
  throw Raised{};
}

decltype(&fp8_gemm) p_gemm;
decltype(&fp8_gemm_gated) p_gated;
decltype(&fp8_gemm_fused) p_fused;
decltype(&fp8_rmsnorm_quantize) p_norm;
decltype(&fp8_rmsnorm_quantize_blockwise) p_norm_blocks;
decltype(&fp8_rmsnorm_backward) p_norm_back;
decltype(&fp8_act_backward) p_act_back;
decltype(&fp8_gated_backward) p_gated_back;

// One call's operands: every tensor must be on the first one's device.
class Call {
 public:
  Call(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : a_(args) {
    if (n != want) raise(PyExc_TypeError, "%s", "wrong number of arguments");
    current_ = (int)PyLong_AsLong(a_[0]);
    stream = PyLong_AsVoidPtr(a_[1]);
    if (PyErr_Occurred()) throw Raised{};
  }
  void* stream;

  // Argument i, a tensor, or null for None.
  const at::Tensor* tensor(int i, const char* name) const {
    if (a_[i] == Py_None) return nullptr;
    if (!THPVariable_Check(a_[i])) raise(PyExc_TypeError, "%s must be a tensor", name);
    return &THPVariable_Unpack(a_[i]);
  }
  // The first operand: required, on a GPU, of so many dimensions.
  const at::Tensor& first(int i, const char* name, int64_t dims) {
    const at::Tensor* t = tensor(i, name);
    if (!t) raise(PyExc_ValueError, "%s must be a GPU tensor", name);
    if (!t->is_cuda()) raise(PyExc_ValueError, "%s must be a GPU tensor", name);
    if (t->dim() != dims) raise(PyExc_ValueError, "%s must have %s", name, dims == 2 ? "2 dimensions" : "another shape");
    device_ = t->get_device();
    return *t;
  }
  bool elsewhere() const { return device_ != current_; }
  PyObject* device() const { return PyLong_FromLong(1 + device_); }

  void* check(const at::Tensor* t, const char* name, at::ScalarType type, bool shaped, at::IntArrayRef shape) const {
    if (!t) return nullptr;
    if (t->scalar_type() != type)
      raise(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t->scalar_type()));
    if (shaped && t->sizes() != shape)
      raise(PyExc_ValueError, "%s must have shape %s, got %s", name, c10::str(shape).c_str(), c10::str(t->sizes()).c_str());
    if (!t->is_cuda() || t->get_device() != device_) raise(PyExc_ValueError, "%s is not on the device of the other operands", name);
    if (!t->is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
    return t->data_ptr();
  }
  void* ptr(int i, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    return check(tensor(i, name), name, type, true, shape);
  }
  void* vec(int i, const char* name, at::ScalarType type, int64_t n) const { return ptr(i, name, type, at::IntArrayRef(&n, 1)); }
  void* mat(int i, const char* name, at::ScalarType type, int64_t m, int64_t n) const {
    const int64_t s[2] = {m, n};
    return ptr(i, name, type, at::IntArrayRef(s, 2));
  }
  void* one(int i, const char* name, at::ScalarType type = at::kFloat) const {
    const at::Tensor* t = tensor(i, name);
    if (t && t->numel() != 1) raise(PyExc_ValueError, "%s must have 1 element", name);
    return check(t, name, type, false, {});
  }
  float* scalar(int i, const char* name) const { return static_cast<float*>(one(i, name)); }
  unsigned long long* count(int i) const { return static_cast<unsigned long long*>(one(i, "sat", at::kLong)); }
  // Workspace and its size.
  void* space(int i, size_t* bytes) const {
    const at::Tensor* t = tensor(i, "workspace");
    *bytes = t ? (size_t)t->numel() : 0;
    return check(t, "workspace", at::kByte, false, {});
  }
  int coded(int i, const char* what, const char* const* names, int n, bool codes) const {
    PyObject* o = a_[i];
    if (PyUnicode_Check(o)) {
      for (int k = 0; k < n; ++k)
        if (PyUnicode_CompareWithASCIIString(o, names[k]) == 0) return k;
    } else if (codes && PyIndex_Check(o) && !THPVariable_Check(o)) {
      const Py_ssize_t v = PyNumber_AsSsize_t(o, nullptr);
      if (v >= 0 && v < n) return (int)v;
      PyErr_Clear();
    }
    PyObject* r = PyObject_Repr(o);
    const char* s = r ? PyUnicode_AsUTF8(r) : "?";
    PyErr_Format(PyExc_ValueError, "unknown %s %s", what, s ? s : "?");
    Py_XDECREF(r);
    throw Raised{};
  }
  int format(int i) const {
    static const char* const names[] = {"e4m3", "e5m2"};
    return coded(i, "FP8 format", names, 2, true);
  }
  int accum(int i) const {
    static const char* const names[] = {"exact", "mfma_fp8"};
    return coded(i, "accumulation mode", names, 2, true);
  }
  int activation(int i) const {
    static const char* const names[] = {"none", "relu", "silu", "gelu"};
    return coded(i, "activation", names, 4, false);
  }
  bool none(int i) const { return a_[i] == Py_None; }
  double number(int i) const {
    const double v = PyFloat_AsDouble(a_[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
  }
  bool truth(int i) const {
    const int v = PyObject_IsTrue(a_[i]);
    if (v < 0) throw Raised{};
    return v != 0;
  }

 private:
  PyObject* const* a_;
  int current_ = -1;
  int device_ = -1;
};

int float_type(const at::Tensor& t, const char* name, PyObject* error) {
  if (t.scalar_type() == at::kFloat) return FP8MI_F32;
  if (t.scalar_type() == at::kBFloat16) return FP8MI_BF16;
  raise(error, "%s must be float32 or bfloat16, got %s", name, c10::toString(t.scalar_type()));
}

// Output of a fused product: codes where a format is given, else fp32 or bf16.
void* output(const Call& c, int i, const char* name, int fmt_at, int64_t m, int64_t n, int* kind) {
  if (!c.none(fmt_at)) {
    *kind = c.format(fmt_at) == FP8MI_E4M3 ? FP8MI_OUT_E4M3 : FP8MI_OUT_E5M2;
    return c.mat(i, name, at::kByte, m, n);
  }
  const at::Tensor* t = c.tensor(i, name);
  if (!t) raise(PyExc_ValueError, "%s must be a GPU tensor", name);
  *kind = float_type(*t, name, PyExc_TypeError) == FP8MI_F32 ? FP8MI_OUT_F32 : FP8MI_OUT_BF16;
  return c.mat(i, name, t->scalar_type(), m, n);
}

const uint8_t* codes(const Call& c, const char* name, const at::Tensor& t) {
  return static_cast<const uint8_t*>(c.check(&t, name, at::kByte, false, {}));
}

// The second operand of a product: [n x k] codes.
const at::Tensor& second(const Call& c, int i, const at::Tensor& a, int64_t k_at) {
  const at::Tensor* b = c.tensor(i, "b");
  if (!b || b->dim() != 2 || b->size(k_at) != a.size(1)) raise(PyExc_ValueError, "%s", "shape mismatch of a and b");
  return *b;
}

typedef uint16_t* bf16p;

// The entry point's status.  Other threads run meanwhile: a launch may have to wait for room in its queue.
template <class F, class... A>
PyObject* invoke(F* f, A... args) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f(args...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

// cur stream x weight eps fmt scale q residual sum_out rstd amax sat workspace
PyObject* norm(PyObject* const* args, Py_ssize_t n) {
  Call c(args, n, 14);
  const at::Tensor& x = c.first(2, "x", 2);
  const int xt = float_type(x, "x", PyExc_ValueError);
  const at::ScalarType t = x.scalar_type();
  const int64_t rows = x.size(0), cols = x.size(1);
  size_t bytes;
  void* px = c.check(&x, "x", t, false, {});
  void* pw = c.vec(3, "weight", t, cols);
  const float eps = (float)c.number(4);
  const int fmt = c.format(5);
  float* scale = c.scalar(6, "scale");
  void* q = c.mat(7, "q", at::kByte, rows, cols);
  void* res = c.mat(8, "residual", t, rows, cols);
  void* sum = c.mat(9, "sum_out", t, rows, cols);
  void* rstd = c.vec(10, "rstd", at::kFloat, rows);
  float* amax = c.scalar(11, "amax");
  unsigned long long* sat = c.count(12);
  void* ws = c.space(13, &bytes);
  if (c.elsewhere()) return c.device();
  return invoke(p_norm, px, res, pw, xt, rows, cols, eps, fmt, scale, sum, (uint8_t*)q, (float*)rstd, amax, sat, ws,
                                bytes, c.stream);
}

// cur stream x weight eps fmt q scale_inv residual sum_out rstd
PyObject* norm_blocks(PyObject* const* args, Py_ssize_t n) {
  Call c(args, n, 11);
  const at::Tensor& x = c.first(2, "x", 2);
  const int xt = float_type(x, "x", PyExc_ValueError);
  const at::ScalarType t = x.scalar_type();
  const int64_t rows = x.size(0), cols = x.size(1);
  void* px = c.check(&x, "x", t, false, {});
  void* pw = c.vec(3, "weight", t, cols);
  const float eps = (float)c.number(4);
  const int fmt = c.format(5);
  void* q = c.mat(6, "q", at::kByte, rows, cols);
  void* si = c.mat(7, "scale_inv", at::kFloat, rows, (cols + 127) / 128);
  void* res = c.mat(8, "residual", t, rows, cols);
  void* sum = c.mat(9, "sum_out", t, rows, cols);
  void* rstd = c.vec(10, "rstd", at::kFloat, rows);
  if (c.elsewhere()) return c.device();
  return invoke(p_norm_blocks, px, res, pw, xt, rows, cols, eps, fmt, sum, (uint8_t*)q, (float*)si, (float*)rstd,
                                       c.stream);
}

// cur stream dy h rstd weight dx dweight dresidual workspace
PyObject* norm_back(PyObject* const* args, Py_ssize_t n) {
  Call c(args, n, 10);
  const at::Tensor& dy = c.first(2, "dy", 2);
  const int xt = float_type(dy, "dy", PyExc_ValueError);
  const at::ScalarType t = dy.scalar_type();
  const int64_t rows = dy.size(0), cols = dy.size(1);
  size_t bytes;
  void* pdy = c.check(&dy, "dy", t, false, {});
  void* h = c.mat(3, "h", t, rows, cols);
  void* rstd = c.vec(4, "rstd", at::kFloat, rows);
  void* w = c.vec(5, "weight", t, cols);
  void* dx = c.mat(6, "dx", t, rows, cols);
  void* dw = c.vec(7, "dweight", at::kFloat, cols);
  void* dres = c.mat(8, "dresidual", t, rows, cols);
  void* ws = c.space(9, &bytes);
  if (c.elsewhere()) return c.device();
  return invoke(p_norm_back, pdy, h, (const float*)rstd, w, dres, xt, rows, cols, dx, (float*)dw, ws, bytes, c.stream);
}

// cur stream a fa b fb sinv_a sinv_b act h gu out_fmt out_scale amax sat accum workspace
PyObject* gated(PyObject* const* args, Py_ssize_t n) {
  Call c(args, n, 17);
  const at::Tensor& a = c.first(2, "a", 2);
  const at::Tensor& b = second(c, 4, a, 1);
  const int64_t M = a.size(0), K = a.size(1), rows = b.size(0);
  if (rows & 1) raise(PyExc_ValueError, "%s", "b must hold as many gate as up rows");
  size_t bytes;
  int kind;
  const uint8_t *pa = codes(c, "a", a), *pb = codes(c, "b", b);
  const int fa = c.format(3), fb = c.format(5);
  float *sa = c.scalar(6, "sinv_a"), *sb = c.scalar(7, "sinv_b");
  const int act = c.activation(8);
  void* h = output(c, 9, "h", 11, M, rows / 2, &kind);
  void* gu = c.mat(10, "gu", at::kBFloat16, M, rows);
  float* os = c.scalar(12, "out_scale");
  float* amax = c.scalar(13, "amax");
  unsigned long long* sat = c.count(14);
  const int accum = c.accum(15);
  void* ws = c.space(16, &bytes);
  if (c.elsewhere()) return c.device();
  return invoke(p_gated, pa, fa, pb, fb, M, rows / 2, K, sa, sb, act, h, kind, os, (bf16p)gu, amax, sat, accum, ws, bytes,
                                 c.stream);
}

// cur stream a fa b fb sinv_a sinv_b y bias act residual z out_fmt out_scale amax sat accum workspace
PyObject* fused(PyObject* const* args, Py_ssize_t n) {
  Call c(args, n, 19);
  const at::Tensor& a = c.first(2, "a", 2);
  const at::Tensor& b = second(c, 4, a, 1);
  const int64_t M = a.size(0), K = a.size(1), N = b.size(0);
  size_t bytes;
  int kind;
  const uint8_t *pa = codes(c, "a", a), *pb = codes(c, "b", b);
  const int fa = c.format(3), fb = c.format(5);
  float *sa = c.scalar(6, "sinv_a"), *sb = c.scalar(7, "sinv_b");
  void* y = output(c, 8, "y", 13, M, N, &kind);
  void* bias = c.vec(9, "bias", at::kBFloat16, N);
  const int act = c.activation(10);
  void* res = c.mat(11, "residual", at::kBFloat16, M, N);
  void* z = c.mat(12, "z", at::kBFloat16, M, N);
  float* os = c.scalar(14, "out_scale");
  float* amax = c.scalar(15, "amax");
  unsigned long long* sat = c.count(16);
  const int accum = c.accum(17);
  void* ws = c.space(18, &bytes);
  if (c.elsewhere()) return c.device();
  return invoke(p_fused, pa, fa, pb, fb, M, N, K, sa, sb, (bf16p)bias, act, (bf16p)res, y, kind, os, (bf16p)z, amax, sat,
                                 accum, ws, bytes, c.stream);
}

// cur stream dy z act fmt scale q q_t dbias amax sat workspace
PyObject* act_back(PyObject* const* args, Py_ssize_t n) {
  Call c(args, n, 13);
  const at::Tensor& dy = c.first(2, "dy", 2);
  const int xt = float_type(dy, "dy", PyExc_ValueError);
  const int64_t M = dy.size(0), N = dy.size(1);
  size_t bytes;
  void* pd = c.check(&dy, "dy", dy.scalar_type(), false, {});
  void* z = c.mat(3, "z", at::kBFloat16, M, N);
  const int act = c.activation(4), fmt = c.format(5);
  float* scale = c.scalar(6, "scale");
  void* q = c.mat(7, "q", at::kByte, M, N);
  void* qt = c.mat(8, "q_t", at::kByte, N, M);
  void* db = c.vec(9, "dbias", at::kFloat, N);
  float* amax = c.scalar(10, "amax");
  unsigned long long* sat = c.count(11);
  void* ws = c.space(12, &bytes);
  if (c.elsewhere()) return c.device();
  return invoke(p_act_back, pd, xt, (bf16p)z, act, M, N, fmt, scale, (uint8_t*)q, (uint8_t*)qt, (float*)db, amax, sat, ws,
                                    bytes, c.stream);
}

// cur stream dh gu act fmt scale q q_t amax sat workspace
PyObject* gated_back(PyObject* const* args, Py_ssize_t n) {
  Call c(args, n, 12);
  const at::Tensor& dh = c.first(2, "dh", 2);
  const int xt = float_type(dh, "dh", PyExc_ValueError);
  const int64_t M = dh.size(0), F = dh.size(1);
  size_t bytes;
  void* pd = c.check(&dh, "dh", dh.scalar_type(), false, {});
  void* gu = c.mat(3, "gu", at::kBFloat16, M, 2 * F);
  const int act = c.activation(4), fmt = c.format(5);
  float* scale = c.scalar(6, "scale");
  void* q = c.mat(7, "q", at::kByte, M, 2 * F);
  void* qt = c.mat(8, "q_t", at::kByte, 2 * F, M);
  float* amax = c.scalar(9, "amax");
  unsigned long long* sat = c.count(10);
  void* ws = c.space(11, &bytes);
  if (c.elsewhere()) return c.device();
  return invoke(p_gated_back, pd, xt, (bf16p)gu, act, M, F, fmt, scale, (uint8_t*)q, (uint8_t*)qt, amax, sat, ws, bytes,
                                      c.stream);
}

// cur stream a fa b fb sinv_a sinv_b c accum b_trans
PyObject* gemm(PyObject* const* args, Py_ssize_t n) {
  Call c(args, n, 11);
  const at::Tensor& a = c.first(2, "a", 2);
  const bool trans = c.truth(10);
  const at::Tensor& b = second(c, 4, a, trans ? 0 : 1);
  const int64_t M = a.size(0), K = a.size(1), N = b.size(trans ? 1 : 0);
  const uint8_t *pa = codes(c, "a", a), *pb = codes(c, "b", b);
  const int fa = c.format(3), fb = c.format(5);
  float *sa = c.scalar(6, "sinv_a"), *sb = c.scalar(7, "sinv_b");
  const at::Tensor* out = c.tensor(8, "c");
  if (!out) raise(PyExc_ValueError, "%s must be a GPU tensor", "c");
  const int type = float_type(*out, "c", PyExc_TypeError);
  void* pc = c.mat(8, "c", out->scalar_type(), M, N);
  const int accum = c.accum(9);
  if (c.elsewhere()) return c.device();
  return invoke(p_gemm, pa, fa, pb, fb, trans ? 1 : 0, M, N, K, sa, sb, pc, type, accum, c.stream);
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// Addresses of the entry points, in the order of the declarations above.
PyObject* bind(PyObject* const* args, Py_ssize_t n) {
  if (n != 8) raise(PyExc_TypeError, "%s", "eight addresses");
  void* p[8];
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) throw Raised{};
  }
  std::memcpy(&p_gemm, &p[0], sizeof(void*));
  std::memcpy(&p_gated, &p[1], sizeof(void*));
  std::memcpy(&p_fused, &p[2], sizeof(void*));
  std::memcpy(&p_norm, &p[3], sizeof(void*));
  std::memcpy(&p_norm_blocks, &p[4], sizeof(void*));
  std::memcpy(&p_norm_back, &p[5], sizeof(void*));
  std::memcpy(&p_act_back, &p[6], sizeof(void*));
  std::memcpy(&p_gated_back, &p[7], sizeof(void*));
  Py_RETURN_NONE;
}

#define ENTRY(name, fn) {name, (PyCFunction)(void (*)(void))entry<fn>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY("bind", bind), ENTRY("gemm", gemm), ENTRY("gated", gated), ENTRY("fused", fused),
                         ENTRY("norm", norm), ENTRY("norm_blocks", norm_blocks), ENTRY("norm_back", norm_back),
                         ENTRY("act_back", act_back), ENTRY("gated_back", gated_back), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8mi_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__fp8mi_marshal() { return PyModule_Create(&module); }
