// binding.cpp — the Python binding of the norm and 4-bit entry points as a CPython extension.
//
// These calls are made per layer on as little as one token, where the GPU needs 3 to 10 us and a ctypes
// call with its checks in Python needs 10 (norm) to 22 us (norm and product): the host would be what
// bounds them. Here a call takes the tensors' addresses from torch's C++ objects, checks what the C side
// cannot see (types, shapes, sizes, device, layout), fills the C structure and calls the library, whose
// entry points are handed over by address (`bind`), so the extension links against torch only.
// Errors: ValueError / TypeError for what is checked here; a non-OK status goes to the callable that
// `bind` was given, which raises.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <vector>

#include "fp8train.h"

namespace {

struct Error {};                            // a Python exception is set

[[noreturn]] void value_error(const char* what, const char* must) {
  PyErr_Format(PyExc_ValueError, "%s: must be %s", what, must);
  throw Error{};
}

struct Library {
  decltype(&fp8_rmsnorm_cast) rmsnorm_cast = nullptr;
  decltype(&fp8_rmsnorm_backward) rmsnorm_backward = nullptr;
  decltype(&fp8_rmsnorm_backward_workspace_bytes) rmsnorm_backward_workspace_bytes = nullptr;
  decltype(&fp4_cast_multi) cast_multi = nullptr;
  decltype(&fp4_gemm_multi) gemm_multi = nullptr;
  PyObject* check = nullptr;                // check(status, where) raises
} lib;

void check_status(fp8t_status status, const char* where) {
  if (status == FP8T_OK) return;
  PyObject* r = PyObject_CallFunction(lib.check, "is", static_cast<int>(status), where);
  Py_XDECREF(r);
  if (r) PyErr_SetString(PyExc_RuntimeError, where);
  throw Error{};
}

// ------------------------------------------------------------------ arguments
const at::Tensor* tensor(PyObject* o, const char* what) {
  if (!o || o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: must be a tensor or None, got %s", what, Py_TYPE(o)->tp_name);
    throw Error{};
  }
  return &THPVariable_Unpack(o);
}

struct Call {
  int device = -1;                          // the current device, looked up once a call
  void* address(const at::Tensor& t, const char* what) {
    if (!t.is_cuda()) value_error(what, "a CUDA tensor on the current device");
    if (device < 0) device = static_cast<int>(c10::cuda::current_device());
    if (t.get_device() != device) value_error(what, "a CUDA tensor on the current device");
    if (!t.is_contiguous()) value_error(what, "contiguous");
    return t.data_ptr();
  }
  void* of(PyObject* o, at::ScalarType type, int64_t n, const char* what, const char* must) {
    const at::Tensor* t = tensor(o, what);
    if (!t) return nullptr;
    if (t->scalar_type() != type || t->numel() < n) value_error(what, must);
    return address(*t, what);
  }
  float* f32(PyObject* o, int64_t n, const char* what) {
    return static_cast<float*>(of(o, at::kFloat, n, what, "float32 with an element for each value it holds"));
  }
  void* bytes(PyObject* o, int64_t n, const char* what) {
    return of(o, at::kByte, n, what, "uint8 with a byte for each value it holds");
  }
  void* bf16(PyObject* o, int64_t rows, int64_t cols, const char* what) {      // [rows, cols]
    const at::Tensor* t = tensor(o, what);
    if (!t) return nullptr;
    if (t->scalar_type() != at::kBFloat16 || t->dim() != 2 || t->size(0) != rows || t->size(1) != cols)
      value_error(what, "a bfloat16 matrix of the call's rows and columns");
    return address(*t, what);
  }
  void* bf16(PyObject* o, int64_t n, const char* what) {                       // [n]
    const at::Tensor* t = tensor(o, what);
    if (!t) return nullptr;
    if (t->scalar_type() != at::kBFloat16 || t->dim() != 1 || t->size(0) != n)
      value_error(what, "a bfloat16 vector with one element per column");
    return address(*t, what);
  }
  void* stream(PyObject* o) {
    if (!o || o == Py_None) return static_cast<void*>(c10::cuda::getCurrentCUDAStream().stream());
    PyObject* v = PyObject_GetAttrString(o, "cuda_stream");
    if (!v) throw Error{};
    void* s = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (!s && PyErr_Occurred()) throw Error{};
    return s;
  }
};

const at::Tensor& matrix(PyObject* o, const char* what) {
  const at::Tensor* t = tensor(o, what);
  if (!t || t->dim() != 2) value_error(what, "a matrix");
  return *t;
}

int integer(PyObject* o, int otherwise) {
  if (!o || o == Py_None) return otherwise;
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Error{};
  if (v != static_cast<int>(v)) value_error("quant and fmt", "a constant of the package");
  return static_cast<int>(v);
}

int64_t fp4_sf_bytes(int64_t mn, int64_t k, int quant) {      // 0 for what the library refuses
  if (quant != FP8T_Q_MXFP4 && quant != FP8T_Q_NVFP4) return 0;
  return (mn + 127) / 128 * ((k + 255) / 256) * (quant == FP8T_Q_MXFP4 ? 1024 : 2048);
}

// Positional and keyword arguments into slots, in the order of `names` (interned).
template <int N>
void parse(PyObject* const* args, Py_ssize_t n, PyObject* kwnames, PyObject* const (&names)[N], int positional,
           const char* function, PyObject* (&out)[N]) {
  if (n > positional) {
    PyErr_Format(PyExc_TypeError, "%s() takes at most %d positional arguments (%zd given)", function, positional, n);
    throw Error{};
  }
  for (int i = 0; i < N; ++i) out[i] = i < n ? args[i] : nullptr;
  const Py_ssize_t nk = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
  for (Py_ssize_t k = 0; k < nk; ++k) {
    PyObject* name = PyTuple_GET_ITEM(kwnames, k);
    int at = -1;
    for (int i = 0; i < N && at < 0; ++i)
      if (names[i] == name) at = i;
    for (int i = 0; i < N && at < 0; ++i)
      if (PyUnicode_Compare(names[i], name) == 0) at = i;
    if (at < 0 || out[at]) {
      PyErr_Format(PyExc_TypeError, "%s() got %s argument '%U'", function, at < 0 ? "an unexpected" : "two values for", name);
      throw Error{};
    }
    out[at] = args[n + k];
  }
}
void required(PyObject* o, const char* function, const char* name) {
  if (o) return;
  PyErr_Format(PyExc_TypeError, "%s() missing argument '%s'", function, name);
  throw Error{};
}

// Runs f and turns its exceptions into Python's.
template <class F>
PyObject* guarded(F&& f) {
  try {
    f();
    Py_RETURN_NONE;
  } catch (const Error&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <int N>
struct Names {
  PyObject* v[N];
  Names(const char* const (&s)[N]) {
    for (int i = 0; i < N; ++i) v[i] = PyUnicode_InternFromString(s[i]);
  }
};

// ------------------------------------------------------------------ the calls
PyObject* rmsnorm_cast(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const Names<15> names({"x", "gamma", "eps", "residual", "h", "rstd", "y", "quant", "fmt", "q", "sf", "scale",
                                "amax", "scale_inv", "stream"});
  return guarded([&] {
    PyObject* a[15];
    parse(args, n, kw, names.v, 3, "fp8_rmsnorm_cast", a);
    required(a[0], "fp8_rmsnorm_cast", "x");
    required(a[1], "fp8_rmsnorm_cast", "gamma");
    required(a[2], "fp8_rmsnorm_cast", "eps");
    Call c;
    const at::Tensor& x = matrix(a[0], "x");
    fp8t_rmsnorm d = {};
    d.rows = x.size(0);
    d.cols = x.size(1);
    d.eps = static_cast<float>(PyFloat_AsDouble(a[2]));
    if (PyErr_Occurred()) throw Error{};
    const int quant = integer(a[7], FP8T_Q_NONE);
    const bool four = quant == FP8T_Q_MXFP4 || quant == FP8T_Q_NVFP4;
    d.quant = static_cast<fp8t_quant>(quant);
    d.fmt = static_cast<fp8t_format>(integer(a[8], FP8T_E4M3));
    d.x_bf16 = c.bf16(a[0], d.rows, d.cols, "x");
    d.gamma_bf16 = c.bf16(a[1], d.cols, "gamma");
    d.residual_bf16 = c.bf16(a[3], d.rows, d.cols, "residual");
    d.h_bf16 = c.bf16(a[4], d.rows, d.cols, "h");
    d.d_rstd_out = c.f32(a[5], d.rows, "rstd");
    d.y_bf16 = c.bf16(a[6], d.rows, d.cols, "y");
    d.q = c.bytes(a[9], four ? d.rows * (d.cols / 2) : d.rows * d.cols, "q");
    d.scales = c.bytes(a[10], four ? fp4_sf_bytes(d.rows, d.cols, quant)
                                   : (d.rows + 127) / 128 * ((d.cols + 127) / 128) * 512, "sf");
    d.d_scale = c.f32(a[11], 1, "scale");
    d.d_amax_inout = c.f32(a[12], 1, "amax");
    d.d_scale_inv_out = c.f32(a[13], 1, "scale_inv");
    check_status(lib.rmsnorm_cast(&d, c.stream(a[14])), "fp8_rmsnorm_cast");
  });
}

PyObject* rmsnorm_backward(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const Names<10> names({"dy", "h", "gamma", "rstd", "dh", "dres", "dgamma", "dgamma_bf16", "workspace", "stream"});
  return guarded([&] {
    PyObject* a[10];
    parse(args, n, kw, names.v, 5, "fp8_rmsnorm_backward", a);
    for (int i = 0; i < 5; ++i) required(a[i], "fp8_rmsnorm_backward", "dy, h, gamma, rstd or dh");
    Call c;
    const at::Tensor& dy = matrix(a[0], "dy");
    fp8t_rmsnorm_grad d = {};
    d.rows = dy.size(0);
    d.cols = dy.size(1);
    d.dy_bf16 = c.bf16(a[0], d.rows, d.cols, "dy");
    d.h_bf16 = c.bf16(a[1], d.rows, d.cols, "h");
    d.gamma_bf16 = c.bf16(a[2], d.cols, "gamma");
    d.d_rstd = c.f32(a[3], d.rows, "rstd");
    d.dh_bf16 = c.bf16(a[4], d.rows, d.cols, "dh");
    d.dres_bf16 = c.bf16(a[5], d.rows, d.cols, "dres");
    d.dgamma_f32 = c.f32(a[6], d.cols, "dgamma");
    d.dgamma_bf16 = c.bf16(a[7], d.cols, "dgamma_bf16");
    void* stream = c.stream(a[9]);
    const at::Tensor* ws = tensor(a[8], "workspace");
    at::Tensor own;
    if (!ws && (d.dgamma_f32 || d.dgamma_bf16)) {
      // Memory of the stream that the kernels run on, freed on return for that stream's later work: a block of another
      // stream's may still be in use by what is queued there, and nothing orders this call behind it.
      c10::cuda::OptionalCUDAStreamGuard on;
      if (a[9] && a[9] != Py_None)
        on.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), c.device));
      own = at::empty({static_cast<int64_t>(lib.rmsnorm_backward_workspace_bytes(d.rows, d.cols))},
                      dy.options().dtype(at::kByte));
      ws = &own;
    }
    void* p = nullptr;
    size_t bytes = 0;
    if (ws) {
      if (ws->scalar_type() != at::kByte) value_error("workspace", "a uint8 tensor");
      p = c.address(*ws, "workspace");
      bytes = static_cast<size_t>(ws->numel());
    }
    check_status(lib.rmsnorm_backward(&d, p, bytes, stream), "fp8_rmsnorm_backward");
  });
}

// Values of a descriptor dict (borrowed), null where absent.
template <int N>
void dict_values(PyObject* o, PyObject* const (&names)[N], PyObject* (&out)[N]) {
  if (!PyDict_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "a list of dicts is needed");
    throw Error{};
  }
  for (int i = 0; i < N; ++i) {
    out[i] = PyDict_GetItemWithError(o, names[i]);
    if (!out[i] && PyErr_Occurred()) throw Error{};
  }
}
void list_and_stream(PyObject* const* args, Py_ssize_t n, PyObject* kw, const char* first, const char* function,
                     PyObject*& list, PyObject*& stream) {
  PyObject* names[2] = {PyUnicode_InternFromString(first), PyUnicode_InternFromString("stream")};
  PyObject* a[2];
  parse(args, n, kw, names, 2, function, a);
  Py_DECREF(names[0]);
  Py_DECREF(names[1]);
  required(a[0], function, first);
  if (!PyList_Check(a[0])) {
    PyErr_Format(PyExc_TypeError, "%s: must be a list of dicts", first);
    throw Error{};
  }
  list = a[0];
  stream = a[1];
}

PyObject* cast_multi(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const Names<9> names({"x", "quant", "q_row", "sf_row", "q_col", "sf_col", "scale", "amax", "scale_inv"});
  return guarded([&] {
    PyObject *list, *stream, *a[9];
    list_and_stream(args, n, kw, "casts", "fp4_cast_multi", list, stream);
    Call c;
    std::vector<fp8t_fp4_cast_tensor> d(PyList_GET_SIZE(list));
    for (size_t i = 0; i < d.size(); ++i) {
      dict_values(PyList_GET_ITEM(list, i), names.v, a);
      const at::Tensor& x = matrix(a[0], "x");
      fp8t_fp4_cast_tensor& t = d[i];
      const int quant = integer(a[1], -1);
      const int64_t r = x.size(0), k = x.size(1);
      t.rows = r;
      t.cols = k;
      t.quant = static_cast<fp8t_quant>(quant);
      t.x_bf16 = c.bf16(a[0], r, k, "x");
      t.q_row = c.bytes(a[2], r * (k / 2), "q_row");
      t.scales_row = c.bytes(a[3], t.q_row ? fp4_sf_bytes(r, k, quant) : 0, "sf_row");
      t.q_col = c.bytes(a[4], k * (r / 2), "q_col");
      t.scales_col = c.bytes(a[5], t.q_col ? fp4_sf_bytes(k, r, quant) : 0, "sf_col");
      t.d_scale = c.f32(a[6], 1, "scale");
      t.d_amax_inout = c.f32(a[7], 1, "amax");
      t.d_scale_inv_out = c.f32(a[8], 1, "scale_inv");
    }
    check_status(lib.cast_multi(d.data(), static_cast<int32_t>(d.size()), c.stream(stream)), "fp4_cast_multi");
  });
}

PyObject* gemm_multi(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  static const Names<8> names({"A", "a_sf", "B", "b_sf", "quant", "D", "a_scale_inv", "b_scale_inv"});
  return guarded([&] {
    PyObject *list, *stream, *a[8];
    list_and_stream(args, n, kw, "gemms", "fp4_gemm_multi", list, stream);
    Call c;
    std::vector<fp8t_fp4_gemm_desc> d(PyList_GET_SIZE(list));
    for (size_t i = 0; i < d.size(); ++i) {
      dict_values(PyList_GET_ITEM(list, i), names.v, a);
      const at::Tensor &A = matrix(a[0], "A"), &B = matrix(a[2], "B");
      fp8t_fp4_gemm_desc& t = d[i];
      const int quant = integer(a[4], -1);
      t.M = A.size(0);
      t.N = B.size(0);
      t.K = 2 * A.size(1);
      if (B.size(1) != A.size(1)) value_error("A and B", "codes [M, K / 2] and [N, K / 2] of one K");
      t.quant = static_cast<fp8t_quant>(quant);
      t.A = c.bytes(a[0], 0, "A");
      t.A_scales = c.bytes(a[1], fp4_sf_bytes(t.M, t.K, quant), "a_sf");
      t.B = c.bytes(a[2], 0, "B");
      t.B_scales = c.bytes(a[3], fp4_sf_bytes(t.N, t.K, quant), "b_sf");
      t.D_bf16 = c.bf16(a[5], t.M, t.N, "D");
      t.d_a_scale_inv = c.f32(a[6], 1, "a_scale_inv");
      t.d_b_scale_inv = c.f32(a[7], 1, "b_scale_inv");
    }
    check_status(lib.gemm_multi(d.data(), static_cast<int32_t>(d.size()), c.stream(stream)), "fp4_gemm_multi");
  });
}

// bind(rmsnorm_cast, rmsnorm_backward, workspace_bytes, cast_multi, gemm_multi, check)
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long p[5];
  PyObject* check;
  if (!PyArg_ParseTuple(args, "KKKKKO", &p[0], &p[1], &p[2], &p[3], &p[4], &check)) return nullptr;
  lib.rmsnorm_cast = reinterpret_cast<decltype(lib.rmsnorm_cast)>(p[0]);
  lib.rmsnorm_backward = reinterpret_cast<decltype(lib.rmsnorm_backward)>(p[1]);
  lib.rmsnorm_backward_workspace_bytes = reinterpret_cast<decltype(lib.rmsnorm_backward_workspace_bytes)>(p[2]);
  lib.cast_multi = reinterpret_cast<decltype(lib.cast_multi)>(p[3]);
  lib.gemm_multi = reinterpret_cast<decltype(lib.gemm_multi)>(p[4]);
  Py_INCREF(check);
  lib.check = check;
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL | METH_KEYWORDS
PyMethodDef methods[] = {
    {"fp8_rmsnorm_cast", FAST(rmsnorm_cast),
     "fp8_rmsnorm_cast(x, gamma, eps, *, residual=None, h=None, rstd=None, y=None, quant=0, fmt=0, q=None, sf=None, "
     "scale=None, amax=None, scale_inv=None, stream=None)\n--\n\n"
     "h = bf16(x + residual); y = h / sqrt(mean(h^2) + eps) * gamma for each row of x (BF16 [rows, cols]).\n\n"
     "Writes h (BF16, with a residual; may be x or residual), rstd (float32 [rows], for the backward pass), y\n"
     "(BF16) and, as quant says, y's codes q (uint8): Q_FP8 with scale, amax (max-accumulated) and scale_inv\n"
     "(float32 [1] each), Q_MXFP8 / Q_MXFP4 / Q_NVFP4 with sf (uint8 scale atoms along the rows), Q_NVFP4 also\n"
     "with scale and optionally amax and scale_inv."},
    {"fp8_rmsnorm_backward", FAST(rmsnorm_backward),
     "fp8_rmsnorm_backward(dy, h, gamma, rstd, dh, *, dres=None, dgamma=None, dgamma_bf16=None, workspace=None, "
     "stream=None)\n--\n\n"
     "Gradients of fp8_rmsnorm_cast: dh (BF16 [rows, cols]; may be dy or dres) from dy and the forward pass's h\n"
     "and rstd, with dres added where given; dgamma (float32 [cols]) and / or dgamma_bf16.\n\n"
     "workspace is a uint8 CUDA tensor of at least fp8_rmsnorm_backward_workspace_bytes bytes (allocated per\n"
     "call where it is missing)."},
    {"fp4_cast_multi", FAST(cast_multi),
     "fp4_cast_multi(casts, stream=None)\n--\n\n"
     "4-bit quantisation. casts: a list of dicts with x (BF16 [rows, cols]), quant (Q_MXFP4 or Q_NVFP4), q_row\n"
     "(uint8 [rows, cols / 2]) / sf_row and / or q_col (uint8 [cols, rows / 2]: transposed) / sf_col, scales uint8\n"
     "tensors of fp4_scale_bytes; for NVFP4 also scale (float32 [1]) and optionally amax (max-accumulated) and\n"
     "scale_inv."},
    {"fp4_gemm_multi", FAST(gemm_multi),
     "fp4_gemm_multi(gemms, stream=None)\n--\n\n"
     "4-bit block-scaled GEMMs: a list of dicts with A (uint8 [M, K / 2]), a_sf, B (uint8 [N, K / 2]), b_sf, quant,\n"
     "D (BF16 [M, N]) and optionally a_scale_inv, b_scale_inv (float32 [1]); D = bf16(A . B^T) with the operands'\n"
     "block scales, times the scale inverses."},
    {"bind", bind, METH_VARARGS, "Hands over the library's entry points and the Python callables."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// FP8T_BUILT_FOR: the versions that this was compiled against, which the loader compares with those it runs under.
PyMODINIT_FUNC PyInit__binding(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", FP8T_BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
