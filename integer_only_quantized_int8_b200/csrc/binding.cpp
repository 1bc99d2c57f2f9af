// binding.cpp -- the Python calls of the serving operators, marshalled natively.
//
// Their small calls run for 3 to 10 us on the GPU, less than a dozen tensors took
// to check and pass through ctypes (9.8 to 13.7 us a call; 3.3 to 6.4 here).  The
// checks and errors are those of the ctypes wrappers in __init__.py: every tensor must
// be a contiguous CUDA tensor of its type on the current device and hold what
// the library reads or writes; a non-OK status comes back as a number for the
// caller to raise.  Sizes and plain arguments come first, so that a call which
// they spoil is refused whatever device its tensors are on.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ivit.h"

namespace {

struct Error {};  // a Python exception is set

[[noreturn]] void fail(PyObject* type, const char* fmt, const char* name = "") {
  PyErr_Format(type, fmt, name);
  throw Error{};
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
  if (PyLong_Check(o) && !(v == -1 && PyErr_Occurred())) return v;
  PyErr_Clear();
  PyObject* n = PyNumber_Index(o);  // numpy integers and the like
  if (!n) throw Error{};
  const int64_t w = PyLong_AsLongLong(n);
  Py_DECREF(n);
  if (w == -1 && PyErr_Occurred()) throw Error{};
  return w;
}

int32_t int32(PyObject* o) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) fail(PyExc_OverflowError, "integer argument out of range%s");
  return (int32_t)v;
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a torch tensor", name);
  return THPVariable_Unpack(o);
}

// the current device, once a tensor of the call is seen to be on a GPU
int device(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", name);
  return c10::cuda::current_device();
}

template <typename T>
T* pointer(const at::Tensor& t, at::ScalarType type, int dev, const char* name) {
  if (t.scalar_type() != type) fail(PyExc_TypeError, "%s has the wrong dtype", name);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", name);
  if (t.get_device() != dev) fail(PyExc_ValueError, "%s is not on the current device", name);
  return static_cast<T*>(t.data_ptr());
}
int8_t* i8(const at::Tensor& t, int dev, const char* name) { return pointer<int8_t>(t, at::kChar, dev, name); }
int32_t* i32(const at::Tensor& t, int dev, const char* name) { return pointer<int32_t>(t, at::kInt, dev, name); }

void holds(const at::Tensor& t, int64_t n, const char* name) {
  if (t.numel() < n) {
    PyErr_Format(PyExc_ValueError, "%s holds %lld elements, needs %lld", name, (long long)t.numel(), (long long)n);
    throw Error{};
  }
}

bool is(const at::Tensor& t, int64_t a, int64_t b) { return t.dim() == 2 && t.size(0) == a && t.size(1) == b; }
bool is(const at::Tensor& t, int64_t a, int64_t b, int64_t c) {
  return t.dim() == 3 && t.size(0) == a && t.size(1) == b && t.size(2) == c;
}
void shape(bool ok, const char* name = "") {
  if (!ok) fail(PyExc_ValueError, *name ? "%s shape mismatch" : "shape mismatch%s", name);
}

// A stream argument: a handle, an object with a cuda_stream, or None for the
// current stream of the call's device, which is looked up once that is known.
struct Stream {
  bool current;
  ivit_stream_t handle;
  ivit_stream_t on(int dev) const {
    return current ? (ivit_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream() : handle;
  }
};

Stream stream_of(PyObject* o) {
  if (o == Py_None) return Stream{true, nullptr};
  PyObject* v = PyIndex_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  PyObject* n = v ? PyNumber_Index(v) : nullptr;
  Py_XDECREF(v);
  if (!n) throw Error{};
  void* const h = PyLong_AsVoidPtr(n);
  Py_DECREF(n);
  if (!h && PyErr_Occurred()) throw Error{};
  return Stream{false, (ivit_stream_t)h};
}

// n integers from a sequence
void numbers(PyObject* o, int32_t* out, Py_ssize_t n) {
  PyObject* f = PySequence_Fast(o, "expected a sequence of integers");
  if (!f) throw Error{};
  bool ok = PySequence_Fast_GET_SIZE(f) == n;
  try {
    for (Py_ssize_t i = 0; ok && i < n; ++i) {
      out[i] = int32(PySequence_Fast_GET_ITEM(f, i));
      ok = PySequence_Fast_GET_SIZE(f) == n;  // a conversion may run any code
    }
  } catch (Error&) {
    Py_DECREF(f);
    throw;
  }
  Py_DECREF(f);
  if (!ok) fail(PyExc_ValueError, "wrong number of integers%s");
}
// a (b, c) pair or a ctypes Dyadic
ivit_dyadic dyadic(PyObject* o) {
  int32_t v[2];
  if (PySequence_Check(o)) {
    numbers(o, v, 2);
  } else {
    for (int i = 0; i < 2; ++i) {
      PyObject* a = PyObject_GetAttrString(o, i ? "c" : "b");
      if (!a) throw Error{};
      try {
        v[i] = int32(a);
      } catch (Error&) {
        Py_DECREF(a);
        throw;
      }
      Py_DECREF(a);
    }
  }
  return ivit_dyadic{v[0], v[1]};
}

// addresses in the library, set by bind()
struct {
  decltype(&ivit_linear_lora) linear_lora;
  decltype(&ivit_linear_lora_shiftgelu) linear_lora_shiftgelu;
  decltype(&ivit_residual_norm) residual_norm;
  decltype(&ivit_attention_diff) attention_diff;
} g;

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) return PyErr_Format(PyExc_TypeError, "bind takes 4 addresses"), nullptr;
  g.linear_lora = (decltype(g.linear_lora))PyLong_AsVoidPtr(a[0]);
  g.linear_lora_shiftgelu = (decltype(g.linear_lora_shiftgelu))PyLong_AsVoidPtr(a[1]);
  g.residual_norm = (decltype(g.residual_norm))PyLong_AsVoidPtr(a[2]);
  g.attention_diff = (decltype(g.attention_diff))PyLong_AsVoidPtr(a[3]);
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

// runs f without the interpreter lock (a launch may wait for room in the queue)
template <typename F>
PyObject* status(F&& f) {
  ivit_status st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return PyLong_FromLong(st);
}

// C++ exceptions (of c10, say) become Python ones too
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (Error&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool arity(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
  return false;
}

// What the linear layers with adapters share: X, W, bias, b, c, adapters, idx, rows, Y, workspace (and skip).
struct Layer {
  int dev;
  int64_t M, rows;
  int32_t K, N;
  ivit_lora lora;
  const int8_t *X, *W, *c, *skip;
  const int32_t *bias, *b, *idx;
  int8_t* Y;
  void* ws;
  size_t ws_bytes;
};

Layer layer(PyObject* const* a, PyObject* skip) {
  Layer l{};
  const at::Tensor &X = tensor(a[0], "X"), &W = tensor(a[1], "W"), &b = tensor(a[3], "b"), &c = tensor(a[4], "c");
  const at::Tensor &idx = tensor(a[6], "idx"), &Y = tensor(a[8], "Y"), &ws = tensor(a[9], "workspace");
  if (!PyTuple_Check(a[5]) || PyTuple_GET_SIZE(a[5]) != 4)
    fail(PyExc_TypeError, "adapters must be a tuple (A, b_t, c_t, B)%s");
  const at::Tensor &A = tensor(PyTuple_GET_ITEM(a[5], 0), "A"), &bt = tensor(PyTuple_GET_ITEM(a[5], 1), "b_t"),
                   &ct = tensor(PyTuple_GET_ITEM(a[5], 2), "c_t"), &B = tensor(PyTuple_GET_ITEM(a[5], 3), "B");
  shape(X.dim() == 2 && W.dim() == 2 && A.dim() == 3);
  const int64_t M = X.size(0), K = X.size(1), N = W.size(0), n = A.size(0), R = A.size(1);
  l.rows = integer(a[7]);
  shape(W.size(1) == K && is(Y, M, N) && is(A, n, R, K) && is(B, n, N, R) && K <= INT32_MAX && N <= INT32_MAX &&
        n <= INT32_MAX && R <= INT32_MAX);
  shape(l.rows >= 1 && M % l.rows == 0, "rows");
  holds(b, N, "b");
  holds(c, N, "c");
  if (a[2] != Py_None) holds(tensor(a[2], "bias"), N, "bias");
  holds(bt, n * R, "b_t");
  holds(ct, n * R, "c_t");
  holds(idx, M / l.rows, "idx");
  if (skip != Py_None) shape(is(tensor(skip, "skip"), M, N), "skip");
  l.dev = device(X, "X");
  l.M = M;
  l.K = (int32_t)K;
  l.N = (int32_t)N;
  l.X = i8(X, l.dev, "X");
  l.W = i8(W, l.dev, "W");
  if (a[2] != Py_None) l.bias = i32(tensor(a[2], "bias"), l.dev, "bias");
  l.b = i32(b, l.dev, "b");
  l.c = i8(c, l.dev, "c");
  l.lora = ivit_lora{(int32_t)n, (int32_t)R, i8(A, l.dev, "A"), i32(bt, l.dev, "b_t"), i8(ct, l.dev, "c_t"),
                     i8(B, l.dev, "B")};
  l.idx = i32(idx, l.dev, "idx");
  if (skip != Py_None) l.skip = i8(tensor(skip, "skip"), l.dev, "skip");
  l.Y = i8(Y, l.dev, "Y");
  l.ws = pointer<uint8_t>(ws, at::kByte, l.dev, "workspace");
  l.ws_bytes = (size_t)ws.numel();
  return l;
}

// X, W, bias, b, c, adapters, idx, rows, Y, workspace, out_bits, skip, res, stream, rounding
PyObject* linear_lora(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 15)) return nullptr;
  return guarded([&]() -> PyObject* {
    const int32_t out_bits = int32(a[10]), rounding = int32(a[14]);
    int32_t r[3] = {0, 0, 0};
    if (a[12] != Py_None) numbers(a[12], r, 3);
    const Stream stream = stream_of(a[13]);
    const Layer l = layer(a, a[11]);
    const ivit_stream_t s = stream.on(l.dev);
    return status([&] {
      return g.linear_lora(l.X, l.M, l.K, l.W, l.N, l.bias, l.b, l.c, out_bits, rounding, &l.lora, l.idx, l.rows, l.skip,
                           ivit_residual{r[0], r[1], r[2]}, l.Y, l.ws, l.ws_bytes, s);
    });
  });
}

// X, W, bias, b, c, adapters, idx, rows, Y, workspace, I0, M, k_out, out, stream, rounding
PyObject* linear_lora_shiftgelu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 16)) return nullptr;
  return guarded([&]() -> PyObject* {
    const int32_t I0 = int32(a[10]), M = int32(a[11]), k_out = int32(a[12]), rounding = int32(a[15]);
    const ivit_dyadic out = dyadic(a[13]);
    const Stream stream = stream_of(a[14]);
    const Layer l = layer(a, Py_None);
    const ivit_stream_t s = stream.on(l.dev);
    return status([&] {
      return g.linear_lora_shiftgelu(l.X, l.M, l.K, l.W, l.N, l.bias, l.b, l.c, rounding, &l.lora, l.idx, l.rows, I0, M,
                                     k_out, out, l.Y, l.ws, l.ws_bytes, s);
    });
  });
}

// gamma, beta, F, M_ln, out; shapes and numbers first, so that all of them are checked before any pointer is taken
ivit_norm norm_shape(PyObject* o, int64_t cols, const char* name) {
  if (o == Py_None) return ivit_norm{};
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5)
    fail(PyExc_TypeError, "%s must be a tuple (gamma, beta, F, M_ln, out)", name);
  shape(tensor(PyTuple_GET_ITEM(o, 0), name).numel() == cols && tensor(PyTuple_GET_ITEM(o, 1), name).numel() == cols, name);
  return ivit_norm{nullptr, nullptr, int32(PyTuple_GET_ITEM(o, 2)), int32(PyTuple_GET_ITEM(o, 3)),
                   dyadic(PyTuple_GET_ITEM(o, 4))};
}
const ivit_norm* norm(PyObject* o, int dev, const char* name, ivit_norm* n) {
  if (o == Py_None) return nullptr;
  n->gamma = i8(THPVariable_Unpack(PyTuple_GET_ITEM(o, 0)), dev, name);
  n->beta = i32(THPVariable_Unpack(PyTuple_GET_ITEM(o, 1)), dev, name);
  return n;
}

// skip, branch, scale, b_skip, c, y, post, gate, gate_rows, pre, z, stream
PyObject* residual_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 12)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &skip = tensor(a[0], "skip"), &branch = tensor(a[1], "branch"), &scale = tensor(a[2], "scale"),
                     &y = tensor(a[5], "y");
    shape(skip.dim() == 2);
    const int64_t rows = skip.size(0), cols = skip.size(1), gate_rows = integer(a[8]);
    shape(is(branch, rows, cols) && is(y, rows, cols) && scale.numel() == cols && cols <= INT32_MAX);
    shape((a[9] == Py_None) == (a[10] == Py_None) && (a[10] == Py_None || is(tensor(a[10], "z"), rows, cols)), "z");
    if (a[7] != Py_None) {
      shape(gate_rows >= 1, "gate");
      holds(tensor(a[7], "gate"), rows == 0 ? 0 : ((rows - 1) / gate_rows + 1) * cols, "gate");
    }
    ivit_norm np = norm_shape(a[6], cols, "post"), nn = norm_shape(a[9], cols, "pre");
    const int32_t b_skip = int32(a[3]), c = int32(a[4]);
    const Stream stream = stream_of(a[11]);
    const int dev = device(skip, "skip");
    const ivit_norm *post = norm(a[6], dev, "post", &np), *pre = norm(a[9], dev, "pre", &nn);
    const int8_t *ps = i8(skip, dev, "skip"), *pb = i8(branch, dev, "branch");
    const int8_t* pg = a[7] == Py_None ? nullptr : i8(THPVariable_Unpack(a[7]), dev, "gate");
    const int32_t* sc = i32(scale, dev, "scale");
    int8_t *py = i8(y, dev, "y"), *pz = a[10] == Py_None ? nullptr : i8(THPVariable_Unpack(a[10]), dev, "z");
    const ivit_stream_t s = stream.on(dev);
    return status([&] {
      return g.residual_norm(ps, pb, rows, (int32_t)cols, post, pg, gate_rows, sc, b_skip, c, pre, py, pz, s);
    });
  });
}

// qkv, B, N, H, logit, k_s, I0, M, k_out, lam, out, ctx, stream
PyObject* attention_diff(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &qkv = tensor(a[0], "qkv"), &lam = tensor(a[9], "lam"), &ctx = tensor(a[11], "ctx");
    const int32_t B = int32(a[1]), N = int32(a[2]), H = int32(a[3]);
    shape(is(qkv, (int64_t)B * N, 384 * (int64_t)H) && is(ctx, (int64_t)B * N, 128 * (int64_t)H));
    holds(lam, H, "lam");
    const ivit_dyadic logit = dyadic(a[4]), out = dyadic(a[10]);
    const int32_t k_s = int32(a[5]), I0 = int32(a[6]), M = int32(a[7]), k_out = int32(a[8]);
    const Stream stream = stream_of(a[12]);
    const int dev = device(qkv, "qkv");
    const int8_t* q = i8(qkv, dev, "qkv");
    const int32_t* l = i32(lam, dev, "lam");
    int8_t* o = i8(ctx, dev, "ctx");
    const ivit_stream_t s = stream.on(dev);
    return status([&] { return g.attention_diff(q, B, N, H, logit, k_s, I0, M, k_out, l, out, o, s); });
  });
}

#define IVIT_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {IVIT_METHOD(bind),          IVIT_METHOD(linear_lora),    IVIT_METHOD(linear_lora_shiftgelu),
                         IVIT_METHOD(residual_norm), IVIT_METHOD(attention_diff), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
