// Marshalling of torch tensors for the operators around the experts (block.py): checks shapes, types,
// devices and strides, allocates the outputs that are not given and calls the C ABI.
//
// Native because a serving step calls these operators once per layer and token: at one token the
// kernels take 1.5 to 3.4 us, a ctypes call with its Python checks took 12-18 us of host time (Grace core),
// this one 3.1 to 4.3.  The C functions come as addresses from the library that the package has loaded, so
// nothing is linked to it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "../../../include/moe_gb300.h"

namespace {

decltype(&moe_block_enter) g_enter;
decltype(&moe_block_leave) g_leave;
decltype(&moe_route_scored) g_route;
decltype(&moe_adapters_add) g_adapters;
PyObject* g_refuse;  // block._refuse(where, why, status): raises MoEError
PyObject* g_key;     // "_key"

struct NormKey {  // block._NormKey
  moe_norm_t desc;           // kind, eps, weight_offset
  PyObject *weight, *bias;  // tensors that the Norm holds, or null
};

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(const char* where, const char* name, const char* why, int status = MOE_ERR_INVALID_ARG) {
  PyObject* r = PyObject_CallFunction(g_refuse, "sNi", where, PyUnicode_FromFormat("%s%s", name, why), status);
  Py_XDECREF(r);  // null: it has raised
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "refused");
  throw Refused();
}

int code(at::ScalarType t) {
  return t == at::kBFloat16 ? MOE_DT_BF16 : t == at::kHalf ? MOE_DT_F16 : t == at::kFloat ? MOE_DT_F32 : 0;
}

const at::Tensor& tensor(PyObject* o, const char* where, const char* name) {
  if (!THPVariable_Check(o)) refuse(where, name, " is not a tensor");
  return THPVariable_Unpack(o);
}

// A [rows, cols] CUDA tensor with unit column stride (rows, cols < 0: any size); its row pitch.
int64_t matrix(const at::Tensor& t, const char* where, const char* name, int64_t rows, int64_t cols,
               std::optional<at::ScalarType> type, std::optional<at::Device> dev) {
  if (t.dim() != 2 || !t.is_cuda() || !code(t.scalar_type()))
    refuse(where, name, " is not a 2-D CUDA tensor of bf16, fp16 or fp32");
  if ((rows >= 0 && t.size(0) != rows) || (cols >= 0 && t.size(1) != cols)) refuse(where, name, " has another shape");
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) refuse(where, name, " has over 2^31 - 1 rows or columns");
  if (type && t.scalar_type() != *type) refuse(where, name, " has another type");
  if (dev && t.device() != *dev) refuse(where, name, " is on another device");
  int64_t ld = t.stride(0);
  if (t.size(0) <= 1 && ld < t.size(1)) ld = t.size(1);
  if ((t.stride(1) != 1 && t.size(1) > 1) || ld < t.size(1))
    refuse(where, name, " needs unit column stride and rows that do not overlap");
  return ld;
}

// A one-row matrix may have any row stride; where a pitch has to be a multiple, use the row's length.
int64_t pitch(const at::Tensor& t, int64_t ld) { return t.size(0) <= 1 ? t.size(1) : ld; }

// Address of a contiguous [n] vector, or null for None.
void* vector(PyObject* o, const char* where, const char* name, int64_t n, at::ScalarType type, at::Device dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, where, name);
  if (t.dim() != 1 || t.size(0) != n || t.scalar_type() != type || t.device() != dev || !t.is_contiguous())
    refuse(where, name, " is not a contiguous vector of the right type, length and device");
  return t.data_ptr();
}

// The descriptor of a Norm (null for None), in d.  The parameters are read here and not when the Norm is made: they may
// have been given other storage since.
const moe_norm_t* norm(PyObject* o, const char* where, int64_t H, at::Device dev, moe_norm_t& d) {
  if (o == Py_None) return nullptr;
  PyObject* k = PyObject_GetAttr(o, g_key);
  if (!k) throw Refused();
  const NormKey* n = (const NormKey*)PyLong_AsVoidPtr(k);
  Py_DECREF(k);
  if (!n) throw Refused();
  d = n->desc;
  d.dtype = 0;
  auto parameter = [&](PyObject* p) -> const void* {
    if (!p) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(p);
    if (t.dim() != 1 || t.size(0) != H || t.device() != dev)
      refuse(where, "", "the norm's parameters have another length or device than the rows");
    const int c = code(t.scalar_type());
    if (!c || !t.is_contiguous() || (d.dtype && d.dtype != c))
      refuse(where, "", "the norm's parameters are not contiguous and of one type, bf16, fp16 or fp32");
    d.dtype = c;
    return t.data_ptr();
  };
  d.weight = parameter(n->weight);
  d.bias = parameter(n->bias);
  return &d;
}

// The device, and where the caller names a stream that stream, for the length of a call: outputs are
// then allocated for the stream that writes them.
struct Place {
  c10::cuda::CUDAGuard dev;
  std::optional<c10::cuda::CUDAStreamGuard> on;
  cudaStream_t stream;
  Place(const at::Tensor& t, PyObject* s) : dev(t.device()) {
    if (s == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
    } else {
      stream = (cudaStream_t)PyLong_AsVoidPtr(s);
      if (PyErr_Occurred()) throw Refused();
      on.emplace(c10::cuda::getStreamFromExternal(stream, t.device().index()));
    }
  }
};

at::Tensor fresh(int64_t rows, int64_t cols, at::ScalarType type, at::Device dev) {
  return at::Tensor(at::detail::empty_cuda({rows, cols}, type, dev, std::nullopt));
}

void check(int status, const char* where) {
  if (status == MOE_OK) return;
  refuse(where, "", status == MOE_ERR_UNSUPPORTED ? "unsupported types or device" : "refused by the library", status);
}

int whole(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v > INT32_MAX || v < INT32_MIN ? INT32_MIN : (int)v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return (float)v;
}

template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused&) {
  } catch (const std::exception& e) {  // torch's: out of memory, a device that is gone
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", n, want);
  return false;
}

// enter(x, norm, dtype, out, stream)
PyObject* enter(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* w = "moe_block_enter";
    const at::Tensor& x = tensor(a[0], w, "x");
    const int64_t ldx = matrix(x, w, "x", -1, -1, std::nullopt, std::nullopt), T = x.size(0), H = x.size(1);
    const at::Device dev = x.device();
    if (a[1] == Py_None) refuse(w, "", "a norm is needed");
    moe_norm_t desc;
    const moe_norm_t* nm = norm(a[1], w, H, dev, desc);
    std::optional<at::ScalarType> type;
    if (a[2] != Py_None) {
      if (!THPDtype_Check(a[2])) refuse(w, "dtype", " is not a torch.dtype");
      type = ((THPDtype*)a[2])->scalar_type;
      if (!code(*type)) refuse(w, "dtype", " is not bf16, fp16 or fp32");
    }
    const Place place(x, a[4]);
    at::Tensor y;
    int64_t ldy = H;
    if (a[3] == Py_None) {
      y = fresh(T, H, type.value_or(x.scalar_type()), dev);
    } else {
      y = tensor(a[3], w, "out");
      ldy = matrix(y, w, "out", T, H, type, dev);
    }
    check(g_enter(x.data_ptr(), ldx, code(x.scalar_type()), nm, y.data_ptr(), ldy, code(y.scalar_type()), (int)T,
                  (int)H, (moe_stream_t)place.stream),
          w);
    return THPVariable_Wrap(std::move(y));
  });
}

// leave(x, block, post, gate, gate_act, alpha, beta, next, out, y, stream)
PyObject* leave(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* w = "moe_block_leave";
    const at::Tensor& x = tensor(a[0], w, "x");
    const int64_t ldx = matrix(x, w, "x", -1, -1, std::nullopt, std::nullopt), T = x.size(0), H = x.size(1);
    const at::Device dev = x.device();
    const at::Tensor& b = tensor(a[1], w, "block");
    const int64_t ldb = matrix(b, w, "block", T, H, std::nullopt, dev);
    moe_norm_t descs[2];
    const moe_norm_t *post = norm(a[2], w, H, dev, descs[0]), *next = norm(a[7], w, H, dev, descs[1]);
    const void* gp = nullptr;
    int64_t gld = 0;
    int gstep = 0, gtype = MOE_DT_BF16;
    if (a[3] != Py_None) {
      const at::Tensor& g = tensor(a[3], w, "gate");
      gtype = code(g.scalar_type());
      if (!gtype || g.device() != dev) refuse(w, "gate", " is not bf16, fp16 or fp32 on x's device");
      const bool channel = g.dim() == 1 && g.size(0) == H, full = g.dim() == 2 && g.size(0) == T && g.size(1) == H;
      const bool token = g.dim() == 2 && g.size(0) == T && g.size(1) == 1;
      if (!channel && !full && !token) refuse(w, "gate", " is not [H], [T, 1] or [T, H]");
      gstep = channel || (full && H > 1);
      gld = channel ? 0 : g.stride(0);
      if (gld < 0 || (gstep && H > 1 && g.stride(g.dim() - 1) != 1)) refuse(w, "gate", " needs unit column stride");
      gp = g.data_ptr();
    }
    const Place place(x, a[10]);
    at::Tensor out, y;
    int64_t ldo = H, ldy = H;
    if (a[8] == Py_None) {
      out = fresh(T, H, x.scalar_type(), dev);
    } else {
      out = tensor(a[8], w, "out");
      ldo = matrix(out, w, "out", T, H, x.scalar_type(), dev);
    }
    if (next && a[9] == Py_None) {
      y = fresh(T, H, b.scalar_type(), dev);
    } else if (next) {
      y = tensor(a[9], w, "y");
      ldy = matrix(y, w, "y", T, H, b.scalar_type(), dev);
    }
    check(g_leave(x.data_ptr(), ldx, code(x.scalar_type()), b.data_ptr(), ldb, code(b.scalar_type()), post, gp, gld,
                  gstep, gtype, whole(a[4]), real(a[5]), real(a[6]), next, out.data_ptr(), ldo,
                  next ? y.data_ptr() : nullptr, ldy, (int)T, (int)H, (moe_stream_t)place.stream),
          w);
    PyObject* po = THPVariable_Wrap(std::move(out));
    if (!next || !po) return po;
    PyObject* py = THPVariable_Wrap(std::move(y));
    PyObject* both = py ? PyTuple_Pack(2, po, py) : nullptr;
    Py_DECREF(po);
    Py_XDECREF(py);
    return both;
  });
}

// route(logits, router address, top_k, bias, topk_idx, topk_w, stream)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* w = "moe_route_scored";
    const at::Tensor& l = tensor(a[0], w, "logits");
    const int64_t ld = matrix(l, w, "logits", -1, -1, std::nullopt, std::nullopt), T = l.size(0), E = l.size(1);
    const at::Device dev = l.device();
    const moe_router_t* r = (const moe_router_t*)PyLong_AsVoidPtr(a[1]);
    if (!r) throw Refused();
    const int k = whole(a[2]);
    if (k < 1 || k > 8) refuse(w, "top_k", " is not in 1 .. 8");
    const float* bias = (const float*)vector(a[3], w, "bias", E, at::kFloat, dev);
    const Place place(l, a[6]);
    at::Tensor idx, wt;
    for (int i = 0; i < 2; ++i) {
      at::Tensor& o = i ? wt : idx;
      const at::ScalarType type = i ? at::kFloat : at::kInt;
      if (a[4 + i] == Py_None) {
        o = fresh(T, k, type, dev);
        continue;
      }
      o = tensor(a[4 + i], w, i ? "topk_w" : "topk_idx");
      if (o.dim() != 2 || o.size(0) != T || o.size(1) != k || o.scalar_type() != type || o.device() != dev ||
          !o.is_contiguous())
        refuse(w, i ? "topk_w" : "topk_idx", " is not a contiguous [T, top_k] of its type on the logits' device");
    }
    check(g_route(r, l.data_ptr(), ld, code(l.scalar_type()), bias, (int)T, (int)E, k, (int32_t*)idx.data_ptr(),
                  (float*)wt.data_ptr(), (moe_stream_t)place.stream),
          w);
    PyObject *pi = THPVariable_Wrap(std::move(idx)), *pw = THPVariable_Wrap(std::move(wt));
    PyObject* both = pi && pw ? PyTuple_Pack(2, pi, pw) : nullptr;
    Py_XDECREF(pi);
    Py_XDECREF(pw);
    return both;
  });
}

// adapters(x, base, a, b, starts, slot, scale, rank, out, stream)
PyObject* adapters(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 10)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* w = "moe_adapters_add";
    const at::Tensor& x = tensor(a[0], w, "x");
    const int64_t ldx = matrix(x, w, "x", -1, -1, at::kBFloat16, std::nullopt), T = x.size(0), H = x.size(1);
    const at::Device dev = x.device();
    const at::Tensor &A = tensor(a[2], w, "a"), &B = tensor(a[3], w, "b");
    if (A.dim() != 3 || B.dim() != 3) refuse(w, "", "a and b are [n, r, H] and [n, N, r]");
    const int64_t na = A.size(0), r = A.size(1), N = B.size(1);
    if (A.size(2) != H || B.size(0) != na || B.size(2) != r || A.scalar_type() != at::kBFloat16 ||
        B.scalar_type() != at::kBFloat16 || A.device() != dev || B.device() != dev || !A.is_contiguous() ||
        !B.is_contiguous() || na > INT32_MAX || r > INT32_MAX || N > INT32_MAX)
      refuse(w, "", "a and b are not contiguous bf16 [n, r, H] and [n, N, r] on x's device");
    const at::Tensor& base = tensor(a[1], w, "base");
    const int64_t ldb = matrix(base, w, "base", T, N, at::kBFloat16, dev);
    const at::Tensor& slot = tensor(a[5], w, "slot");
    if (slot.dim() != 1 || slot.size(0) > INT32_MAX) refuse(w, "slot", " is not a vector");
    const int64_t R = slot.size(0);
    const void* st = vector(a[4], w, "starts", R + 1, at::kInt, dev);
    const void* sl = vector(a[5], w, "slot", R, at::kInt, dev);
    const void* sc = vector(a[6], w, "scale", na, at::kFloat, dev);
    const void* rk = vector(a[7], w, "rank", na, at::kInt, dev);
    const Place place(x, a[9]);
    at::Tensor out;
    int64_t ldo = N;
    if (a[8] == Py_None) {
      out = fresh(T, N, at::kBFloat16, dev);
    } else {
      out = tensor(a[8], w, "out");
      ldo = matrix(out, w, "out", T, N, at::kBFloat16, dev);
    }
    check(g_adapters(x.data_ptr(), pitch(x, ldx), base.data_ptr(), pitch(base, ldb), A.data_ptr(), B.data_ptr(),
                     (const float*)sc, (const int32_t*)rk, (const int32_t*)st, (const int32_t*)sl, out.data_ptr(),
                     pitch(out, ldo), (int)T, (int)R, (int)na, (int)r, (int)H, (int)N, (moe_stream_t)place.stream),
          w);
    return THPVariable_Wrap(std::move(out));
  });
}

// init(refuse, enter, leave, route, adapters): the refusal and the C functions' addresses
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 5)) return nullptr;
  Py_INCREF(a[0]);
  g_refuse = a[0];
  g_key = PyUnicode_InternFromString("_key");
  g_enter = (decltype(g_enter))PyLong_AsVoidPtr(a[1]);
  g_leave = (decltype(g_leave))PyLong_AsVoidPtr(a[2]);
  g_route = (decltype(g_route))PyLong_AsVoidPtr(a[3]);
  g_adapters = (decltype(g_adapters))PyLong_AsVoidPtr(a[4]);
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {{"init", (PyCFunction)(void*)init, METH_FASTCALL, nullptr},
                           {"enter", (PyCFunction)(void*)enter, METH_FASTCALL, nullptr},
                           {"leave", (PyCFunction)(void*)leave, METH_FASTCALL, nullptr},
                           {"route", (PyCFunction)(void*)route, METH_FASTCALL, nullptr},
                           {"adapters", (PyCFunction)(void*)adapters, METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_block_ext", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__block_ext(void) { return PyModule_Create(&g_module); }
