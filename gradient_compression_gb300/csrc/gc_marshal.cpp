// Argument marshalling of activations.py: the checks of tensors and the calls
// of libgc's activation entry points.  A call of one token takes the GPU 1 to 5
// us; checked in Python and passed through ctypes, its host side took 7 (norm)
// to 13 us (gated activation, with the slices of its projection).
//
// Functions return the entry point's status; what is wrong with a tensor
// raises ValueError before anything is enqueued.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <utility>

#include "../../include/gc.h"

namespace {

// ---------------------------------------------------------------- entry points
struct Entry {
  decltype(&gc_act_compress) act_compress;
  decltype(&gc_act_decompress) act_decompress;
  decltype(&gc_rmsnorm) rmsnorm;
  decltype(&gc_rmsnorm_backward) rmsnorm_backward;
  decltype(&gc_gated_act) gated_act;
  decltype(&gc_gated_act_backward) gated_act_backward;
  decltype(&gc_act_weight_grad) act_weight_grad;
} entry;

// bind(addresses of the entry points in the order above), as loaded by the package
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void** slots = reinterpret_cast<void**>(&entry);
  if (n != (Py_ssize_t)(sizeof(entry) / sizeof(void*))) {
    PyErr_SetString(PyExc_TypeError, "bind: wrong number of entry points");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    slots[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_RETURN_NONE;
}

// ---------------------------------------------------------------- checks
struct Bad {};  // a Python exception is set

[[noreturn]] void bad(const char* format, ...) {
  va_list va;
  va_start(va, format);
  PyErr_FormatV(PyExc_ValueError, format, va);
  va_end(va);
  throw Bad{};
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    default: return c10::toString(t);
  }
}
int type_code(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return GC_F32;
    case at::kBFloat16: return GC_BF16;
    case at::kHalf: return GC_F16;
    default: bad("%s: %s is not supported", name, c10::toString(t.scalar_type()));
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad("%s: a tensor is needed", name);
  return THPVariable_Unpack(o);
}

// The GPU of a call's tensors, the first one's: the others have to be there too.
struct Gpu {
  c10::DeviceIndex index = -1;
  bool holds(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) return false;
    const c10::DeviceIndex i = t.device().index();
    if (index < 0) index = i;
    if (i != index) bad("%s: on cuda:%d where cuda:%d is needed", name, (int)i, (int)index);
    return true;
  }
};

struct Mat {
  void* p = nullptr;
  int64_t ld = 0;
};
void check_matrix(Gpu& on, const at::Tensor& t, const char* name) {
  if (t.dim() != 2 || !on.holds(t, name)) bad("%s: a 2-D CUDA tensor is needed", name);
}
// A matrix argument after its checks; rows < 0 takes any shape.
Mat matrix(Gpu& on, const at::Tensor& t, const char* name, int64_t rows = -1, int64_t cols = -1) {
  check_matrix(on, t, name);
  const at::IntArrayRef size = t.sizes(), stride = t.strides();
  const int64_t r = size[0], c = size[1];
  if (rows >= 0 && (r != rows || c != cols))
    bad("%s: shape (%lld, %lld) where (%lld, %lld) is needed", name, (long long)r, (long long)c, (long long)rows, (long long)cols);
  if (stride[1] != 1 && c > 1) bad("%s: columns are not consecutive", name);
  Mat m;
  m.ld = stride[0];
  if (m.ld < c) {
    if (r > 1) bad("%s: rows overlap", name);
    m.ld = c;
  }
  m.p = t.data_ptr();
  return m;
}
// The same where an argument may be None, of the type of another.
Mat matrix(Gpu& on, PyObject* o, const char* name, int64_t rows, int64_t cols, at::ScalarType type) {
  if (o == Py_None) return Mat();
  const at::Tensor& t = tensor(o, name);
  const Mat m = matrix(on, t, name, rows, cols);
  if (t.scalar_type() != type) bad("%s: %s where %s is needed", name, type_name(t.scalar_type()), type_name(type));
  return m;
}
Mat needed(Gpu& on, PyObject* o, const char* name, int64_t rows, int64_t cols, at::ScalarType type) {
  tensor(o, name);
  return matrix(on, o, name, rows, cols, type);
}

// A contiguous vector argument, fp32 or (code given) of any of the types.
void* vector(Gpu& on, PyObject* o, const char* name, int64_t n, int* code) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  const at::ScalarType s = t.scalar_type();
  const bool fits = s == at::kFloat || (code && (s == at::kBFloat16 || s == at::kHalf));
  if (t.dim() != 1 || t.size(0) != n || !on.holds(t, name) || !fits || !t.is_contiguous())
    bad("%s: a contiguous CUDA vector of %lld elements of torch.float32%s is needed", name, (long long)n,
        code ? " or torch.bfloat16 or torch.float16" : "");
  if (code) *code = type_code(t, name);
  return t.data_ptr();
}

struct Space {
  void* p = nullptr;
  size_t bytes = 0;
};
Space workspace(Gpu& on, PyObject* o) {
  Space w;
  if (o == Py_None) return w;
  const at::Tensor& t = tensor(o, "workspace");
  if (!on.holds(t, "workspace") || t.scalar_type() != at::kByte || !t.is_contiguous()) bad("workspace: a contiguous CUDA uint8 tensor is needed");
  w.p = t.data_ptr(), w.bytes = (size_t)t.numel();
  return w;
}

// An ActCheckpoint: its size and its arrays as they are at the call (they may
// have been replaced, moved or resized since it was made), held on to until it returns.
PyObject *s_rows, *s_cols, *s_codes, *s_steps, *s_stream;
PyObject* attribute(PyObject* o, PyObject* field, const char* name) {
  PyObject* v = PyObject_GetAttr(o, field);
  if (v) return v;
  if (!PyErr_ExceptionMatches(PyExc_AttributeError)) throw Bad{};
  PyErr_Clear();
  bad("%s: an ActCheckpoint is needed", name);
}
int64_t number(PyObject* o, PyObject* field, const char* name) {
  PyObject* v = attribute(o, field, name);
  const int64_t x = PyLong_AsLongLong(v);
  Py_DECREF(v);
  if (x == -1 && PyErr_Occurred()) throw Bad{};
  return x;
}
// A tensor attribute, held on to.
struct Array {
  PyObject* of = nullptr;
  Array() = default;
  Array(PyObject* o, PyObject* field, const char* name) : of(attribute(o, field, name)) {
    if (THPVariable_Check(of)) return;
    Py_DECREF(of);
    bad("%s: its %U is no tensor", name, field);
  }
  Array(Array&& a) noexcept : of(a.of) { a.of = nullptr; }
  Array& operator=(Array&& a) noexcept {
    std::swap(of, a.of);
    return *this;
  }
  ~Array() { Py_XDECREF(of); }
  const at::Tensor& tensor() const { return THPVariable_Unpack(of); }
};
void check_array(Gpu& on, const at::Tensor& t, const char* name, int64_t rows, int64_t cols, at::ScalarType type, const char* what) {
  const at::IntArrayRef size = t.sizes();
  if (size.size() != 2 || size[0] != rows || size[1] != cols || t.scalar_type() != type || !t.is_contiguous() || !on.holds(t, name))
    bad("%s: a contiguous CUDA %s tensor of shape (%lld, %lld) is needed", name, what, (long long)rows, (long long)cols);
}
void check_arrays(Gpu& on, const at::Tensor& codes, const at::Tensor& steps, int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1 || cols > INT64_C(2147483647))
    bad("a checkpoint of (%lld, %lld)", (long long)rows, (long long)cols);
  const int64_t groups = (cols + 31) / 32;
  check_array(on, codes, "codes", rows, 32 * groups, at::kChar, "int8");
  check_array(on, steps, "steps", rows, groups, at::kByte, "uint8");
}
struct Held {
  int64_t rows = 0, cols = 0;
  int8_t* codes = nullptr;
  uint8_t* steps = nullptr;
  Array arrays[2];
};
Held held(Gpu& on, PyObject* o, const char* name) {
  Held h;
  h.rows = number(o, s_rows, name), h.cols = number(o, s_cols, name);
  h.arrays[0] = Array(o, s_codes, name), h.arrays[1] = Array(o, s_steps, name);
  const at::Tensor &codes = h.arrays[0].tensor(), &steps = h.arrays[1].tensor();
  check_arrays(on, codes, steps, h.rows, h.cols);
  h.codes = static_cast<int8_t*>(codes.data_ptr()), h.steps = static_cast<uint8_t*>(steps.data_ptr());
  return h;
}
Held held(Gpu& on, PyObject* o, const char* name, int64_t rows, int64_t cols) {
  if (o == Py_None) return Held();
  Held h = held(on, o, name);
  if (h.rows != rows || h.cols != cols)
    bad("%s: a checkpoint of (%lld, %lld) where (%lld, %lld) is needed", name, (long long)h.rows, (long long)h.cols,
        (long long)rows, (long long)cols);
  return h;
}

// A torch stream, a number, or None for the current stream of the tensor's device.
void* stream_of(PyObject* o, const at::Tensor& t) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
  PyObject* v = PyObject_HasAttr(o, s_stream) ? PyObject_GetAttr(o, s_stream) : PyNumber_Long(o);
  if (!v) throw Bad{};
  void* s = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (!s && PyErr_Occurred()) throw Bad{};
  return s;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Bad{};
  return v != 0;
}

// The entry point, with the tensors' GPU the thread's current one (whose streams
// and kernels the launches take), and the thread's own again after it.
template <typename F, typename... A>
PyObject* call(const Gpu& on, F f, A... a) {
  gc_status st;
  Py_BEGIN_ALLOW_THREADS;
  c10::DeviceIndex was = on.index;
  const bool elsewhere = c10::cuda::GetDevice(&was) == cudaSuccess && was != on.index;
  st = elsewhere && c10::cuda::SetDevice(on.index) != cudaSuccess ? GC_ERR_CUDA : f(a...);
  if (elsewhere) (void)c10::cuda::SetDevice(was);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

// ---------------------------------------------------------------- calls
using Args = PyObject* const*;

PyObject* act_compress(Args a) {  // x, ckpt, stream
  Gpu on;
  const at::Tensor& x = tensor(a[0], "x");
  check_matrix(on, x, "x");
  const Held h = held(on, a[1], "ckpt");
  const Mat m = matrix(on, x, "x", h.rows, h.cols);
  return call(on, entry.act_compress, m.p, m.ld, type_code(x, "x"), h.rows, h.cols, h.codes, h.steps, stream_of(a[2], x));
}

PyObject* act_decompress(Args a) {  // ckpt, out, stream
  Gpu on;
  const at::Tensor& out = tensor(a[1], "out");
  check_matrix(on, out, "out");
  const Held h = held(on, a[0], "ckpt");
  const Mat m = matrix(on, out, "out", h.rows, h.cols);
  return call(on, entry.act_decompress, h.codes, h.steps, h.rows, h.cols, m.p, m.ld, type_code(out, "out"), stream_of(a[2], out));
}

PyObject* rmsnorm(Args a) {  // x, weight, eps, y, residual, h, rstd, ckpt, stream
  Gpu on;
  const at::Tensor& x = tensor(a[0], "x");
  const Mat mx = matrix(on, x, "x");
  const int64_t rows = x.size(0), cols = x.size(1);
  const at::ScalarType type = x.scalar_type();
  const int code = type_code(x, "x");
  const Mat r = matrix(on, a[4], "residual", rows, cols, type), y = matrix(on, a[3], "y", rows, cols, type),
            h = matrix(on, a[5], "h", rows, cols, type);
  int wcode = 0;
  void* const w = vector(on, a[1], "weight", cols, &wcode);
  float* const rstd = static_cast<float*>(vector(on, a[6], "rstd", rows, nullptr));
  const Held c = held(on, a[7], "ckpt", rows, cols);
  const double eps = PyFloat_AsDouble(a[2]);
  if (eps == -1.0 && PyErr_Occurred()) throw Bad{};
  return call(on, entry.rmsnorm, mx.p, mx.ld, r.p, r.ld, code, w, wcode, (float)eps, rows, cols, y.p, y.ld, h.p, h.ld, rstd,
              c.codes, c.steps, stream_of(a[8], x));
}

PyObject* rmsnorm_backward(Args a) {  // dy, ckpt, rstd, weight, dx, dw, workspace, dh, accumulate, stream
  Gpu on;
  const at::Tensor& dy = tensor(a[0], "dy");
  check_matrix(on, dy, "dy");
  const Held c = held(on, a[1], "ckpt");
  const Mat d = matrix(on, dy, "dy", c.rows, c.cols);
  const at::ScalarType type = dy.scalar_type();
  const int code = type_code(dy, "dy");
  const Mat dx = needed(on, a[4], "dx", c.rows, c.cols, type), dh = matrix(on, a[7], "dh", c.rows, c.cols, type);
  int wcode = 0;
  void* const w = vector(on, a[3], "weight", c.cols, &wcode);
  float* const dw = static_cast<float*>(vector(on, a[5], "dw", c.cols, nullptr));
  const Space ws = dw ? workspace(on, a[6]) : Space();
  if (a[2] == Py_None) bad("rstd is needed");
  float* const rstd = static_cast<float*>(vector(on, a[2], "rstd", c.rows, nullptr));
  return call(on, entry.rmsnorm_backward, d.p, d.ld, dh.p, dh.ld, code, c.codes, c.steps, rstd, w, wcode, c.rows, c.cols, dx.p,
              dx.ld, dw, truth(a[8]) ? GC_ACCUMULATE : 0u, ws.p, ws.bytes, stream_of(a[9], dy));
}

int kind_of(PyObject* o) {
  const long k = PyLong_AsLong(o);
  if (k == -1 && PyErr_Occurred()) throw Bad{};
  return (int)k;
}

PyObject* gated_act(Args a) {  // kind, gate, up, out, ckpt_gate, ckpt_up, stream
  Gpu on;
  const at::Tensor& gate = tensor(a[1], "gate");
  const Mat g = matrix(on, gate, "gate");
  const int64_t rows = gate.size(0), cols = gate.size(1);
  const at::ScalarType type = gate.scalar_type();
  const int code = type_code(gate, "gate");
  const Mat u = needed(on, a[2], "up", rows, cols, type), out = needed(on, a[3], "out", rows, cols, type);
  const Held cg = held(on, a[4], "ckpt_gate", rows, cols), cu = held(on, a[5], "ckpt_up", rows, cols);
  return call(on, entry.gated_act, kind_of(a[0]), g.p, g.ld, u.p, u.ld, code, rows, cols, out.p, out.ld, cg.codes, cg.steps,
              cu.codes, cu.steps, stream_of(a[6], gate));
}

PyObject* gated_act_backward(Args a) {  // kind, dout, ckpt_gate, ckpt_up, dgate, dup, ckpt_out, stream
  Gpu on;
  const at::Tensor& dout = tensor(a[1], "dout");
  check_matrix(on, dout, "dout");
  const Held cg = held(on, a[2], "ckpt_gate");
  const Mat d = matrix(on, dout, "dout", cg.rows, cg.cols);
  const at::ScalarType type = dout.scalar_type();
  const int code = type_code(dout, "dout");
  const Mat dg = needed(on, a[4], "dgate", cg.rows, cg.cols, type), du = needed(on, a[5], "dup", cg.rows, cg.cols, type);
  const Held cu = held(on, a[3], "ckpt_up", cg.rows, cg.cols), co = held(on, a[6], "ckpt_out", cg.rows, cg.cols);
  return call(on, entry.gated_act_backward, kind_of(a[0]), d.p, d.ld, code, cg.codes, cg.steps, cu.codes, cu.steps, cg.rows,
              cg.cols, dg.p, dg.ld, du.p, du.ld, co.codes, co.steps, stream_of(a[7], dout));
}

PyObject* act_weight_grad(Args a) {  // dy, ckpt, dw, workspace, col_scale, accumulate, stream
  Gpu on;
  const at::Tensor& dy = tensor(a[0], "dy");
  check_matrix(on, dy, "dy");
  const Held c = held(on, a[1], "ckpt");
  const int64_t n = dy.size(1);
  const Mat d = matrix(on, dy, "dy", c.rows, n), dw = needed(on, a[2], "dw", n, c.cols, at::kFloat);
  const int code = type_code(dy, "dy");
  int scode = 0;
  void* const scale = vector(on, a[4], "col_scale", c.cols, &scode);
  const Space ws = workspace(on, a[3]);
  return call(on, entry.act_weight_grad, d.p, d.ld, code, c.rows, n, c.codes, c.steps, c.cols, scale, scode,
              static_cast<float*>(dw.p), dw.ld, truth(a[5]) ? GC_ACCUMULATE : 0u, ws.p, ws.bytes, stream_of(a[6], dy));
}

// checkpoint(codes, steps, rows, cols): the checks of an ActCheckpoint's arrays
PyObject* checkpoint(Args a) {
  Gpu on;
  const int64_t rows = PyLong_AsLongLong(a[2]), cols = PyLong_AsLongLong(a[3]);
  if (PyErr_Occurred()) throw Bad{};
  check_arrays(on, tensor(a[0], "codes"), tensor(a[1], "steps"), rows, cols);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(Args), int N>
PyObject* checked(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are needed", N);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Bad&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define GC_METHOD(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&checked<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&bind)), METH_FASTCALL, nullptr},
                         GC_METHOD(checkpoint, 4),
                         GC_METHOD(act_compress, 3),
                         GC_METHOD(act_decompress, 3),
                         GC_METHOD(rmsnorm, 9),
                         GC_METHOD(rmsnorm_backward, 10),
                         GC_METHOD(gated_act, 7),
                         GC_METHOD(gated_act_backward, 8),
                         GC_METHOD(act_weight_grad, 7),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  s_rows = PyUnicode_InternFromString("rows"), s_cols = PyUnicode_InternFromString("cols");
  s_codes = PyUnicode_InternFromString("codes"), s_steps = PyUnicode_InternFromString("steps");
  s_stream = PyUnicode_InternFromString("cuda_stream");
  return PyModule_Create(&module);
}
