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
decltype(&moe_layer_few) g_few;
decltype(&moe_fp8_quantize) g_quantize;
decltype(&moe_fp8_linear) g_linear;
decltype(&moe_fp8_linear_workspace_size) g_linear_size;
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

// few(x, w_router, router address, desc address, packed, top_k, workspace, bias, out, topk_idx, topk_w, stream)
PyObject* few(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 12)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* w = "moe_layer_few";
    const moe_router_t* r = (const moe_router_t*)PyLong_AsVoidPtr(a[2]);
    const moe_packed_desc_t* d = (const moe_packed_desc_t*)PyLong_AsVoidPtr(a[3]);
    if (!r || !d) throw Refused();
    const at::Tensor& x = tensor(a[0], w, "x");
    const int64_t ldx = matrix(x, w, "x", -1, d->H, at::kBFloat16, std::nullopt), T = x.size(0);
    const at::Device dev = x.device();
    if (T > MOE_FEW_MAX_TOKENS) refuse(w, "x", " has more rows than the call takes (32)");
    const at::Tensor& wr = tensor(a[1], w, "w_router");
    const int64_t ldw = matrix(wr, w, "w_router", d->E, d->H, std::nullopt, dev);
    const at::Tensor &packed = tensor(a[4], w, "packed"), &ws = tensor(a[6], w, "workspace");
    if (packed.device() != dev || !packed.is_contiguous() || (uint64_t)packed.nbytes() < d->bytes)
      refuse(w, "packed", " is smaller than the descriptor says, not contiguous, or on another device");
    if (ws.device() != dev || !ws.is_contiguous()) refuse(w, "workspace", " is not contiguous or on another device");
    const int k = whole(a[5]);
    const float* bias = (const float*)vector(a[7], w, "bias", d->E, at::kFloat, dev);
    void* top[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i) {
      if (a[9 + i] == Py_None) continue;
      const char* name = i ? "topk_w" : "topk_idx";
      const at::Tensor& o = tensor(a[9 + i], w, name);
      if (o.dim() != 2 || o.size(0) != T || o.size(1) != k || o.scalar_type() != (i ? at::kFloat : at::kInt) || o.device() != dev ||
          !o.is_contiguous())
        refuse(w, name, " is not a contiguous [T, top_k] of its type on x's device");
      top[i] = o.data_ptr();
    }
    const Place place(x, a[11]);
    at::Tensor out;
    int64_t ldo = d->H;
    if (a[8] == Py_None) {
      out = fresh(T, d->H, at::kBFloat16, dev);
    } else {
      out = tensor(a[8], w, "out");
      ldo = matrix(out, w, "out", T, d->H, at::kBFloat16, dev);
    }
    check(g_few(x.data_ptr(), pitch(x, ldx), wr.data_ptr(), pitch(wr, ldw), code(wr.scalar_type()), r, bias, (int)T, d,
                packed.data_ptr(), k, out.data_ptr(), pitch(out, ldo), (int32_t*)top[0], (float*)top[1], ws.data_ptr(),
                ws.nbytes(), (moe_stream_t)place.stream),
          w);
    return THPVariable_Wrap(std::move(out));
  });
}

bool is_codes(const at::Tensor& t) { return t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte; }

// A [rows, cols] CUDA tensor of E4M3 codes with unit column stride; its row pitch.
int64_t codes(const at::Tensor& t, const char* where, const char* name, int64_t rows, int64_t cols, std::optional<at::Device> dev) {
  if (t.dim() != 2 || !t.is_cuda() || !is_codes(t)) refuse(where, name, " is not a 2-D CUDA tensor of E4M3 codes");
  if ((rows >= 0 && t.size(0) != rows) || (cols >= 0 && t.size(1) != cols)) refuse(where, name, " has another shape");
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) refuse(where, name, " has over 2^31 - 1 rows or columns");
  if (dev && t.device() != *dev) refuse(where, name, " is on another device");
  if ((t.stride(1) != 1 && t.size(1) > 1) || (t.size(0) > 1 && t.stride(0) < t.size(1)))
    refuse(where, name, " needs unit column stride and rows that do not overlap");
  return pitch(t, t.stride(0));
}

// Address of a contiguous fp32 [rows, cols].
float* scales(PyObject* o, const char* where, const char* name, int64_t rows, int64_t cols, at::Device dev) {
  const at::Tensor& t = tensor(o, where, name);
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || t.scalar_type() != at::kFloat || t.device() != dev || !t.is_contiguous())
    refuse(where, name, " is not a contiguous fp32 tensor of a scale per block");
  return (float*)t.data_ptr();
}

// quantize(x, codes, scale_inv, stream)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 4)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* w = "moe_fp8_quantize";
    const at::Tensor& x = tensor(a[0], w, "x");
    const int64_t ldx = matrix(x, w, "x", -1, -1, std::nullopt, std::nullopt), T = x.size(0), K = x.size(1), G = (K + 127) / 128;
    const at::Device dev = x.device();
    const Place place(x, a[3]);
    at::Tensor q, s;
    int64_t ldq = K;
    if (a[1] == Py_None) {
      q = fresh(T, K, at::kFloat8_e4m3fn, dev);
    } else {
      q = tensor(a[1], w, "codes");
      ldq = codes(q, w, "codes", T, K, dev);
    }
    if (a[2] == Py_None) {
      s = fresh(T, G, at::kFloat, dev);
    } else {
      s = tensor(a[2], w, "scale_inv");
      scales(a[2], w, "scale_inv", T, G, dev);
    }
    check(g_quantize(x.data_ptr(), ldx, code(x.scalar_type()), (uint8_t*)q.data_ptr(), ldq, (float*)s.data_ptr(), (int)T, (int)K,
                     (moe_stream_t)place.stream),
          w);
    PyObject *pq = THPVariable_Wrap(std::move(q)), *ps = THPVariable_Wrap(std::move(s));
    PyObject* both = pq && ps ? PyTuple_Pack(2, pq, ps) : nullptr;
    Py_XDECREF(pq);
    Py_XDECREF(ps);
    return both;
  });
}

// linear(x, x_scale, weight codes, weight scales, act, base, out, dtype, stream)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const char* w = "moe_fp8_linear";
    const at::Tensor &x = tensor(a[0], w, "x"), &wt = tensor(a[2], w, "weight");
    const bool coded = a[1] != Py_None;
    const int64_t ldx = coded ? codes(x, w, "x", -1, -1, std::nullopt) : matrix(x, w, "x", -1, -1, std::nullopt, std::nullopt);
    const int64_t T = x.size(0), K = x.size(1), N = wt.dim() == 2 ? wt.size(0) : 0, G = (K + 127) / 128;
    const at::Device dev = x.device();
    if (codes(wt, w, "weight", -1, K, dev) != K) refuse(w, "weight", " is not contiguous");
    const float* wsc = scales(a[3], w, "the weight's scale_inv", (N + 127) / 128, G, dev);
    const float* xsc = coded ? scales(a[1], w, "x_scale", T, G, dev) : nullptr;
    const int act = whole(a[4]);
    if (act == MOE_ACT_SILU_MUL && N % 2) refuse(w, "weight", " has an odd number of rows: no gates and ups");
    const int64_t cols = act == MOE_ACT_SILU_MUL ? N / 2 : N;
    std::optional<at::ScalarType> type;
    if (a[7] != Py_None) {
      if (!THPDtype_Check(a[7])) refuse(w, "dtype", " is not a torch.dtype");
      type = ((THPDtype*)a[7])->scalar_type;
      if (!code(*type)) refuse(w, "dtype", " is not bf16, fp16 or fp32");
    }
    const Place place(x, a[8]);
    at::Tensor out;
    int64_t ldo = cols, ldb = cols;
    if (a[6] != Py_None) {
      out = tensor(a[6], w, "out");
      ldo = matrix(out, w, "out", T, cols, type, dev);
    }
    const void* base = nullptr;
    if (a[5] != Py_None) {
      const at::Tensor& b = tensor(a[5], w, "base");
      if (out.defined()) type = out.scalar_type();
      ldb = matrix(b, w, "base", T, cols, type, dev);
      type = b.scalar_type();
      base = b.data_ptr();
    }
    if (!out.defined()) out = fresh(T, cols, type.value_or(coded ? at::kBFloat16 : x.scalar_type()), dev);
    const int xt = coded ? MOE_DT_E4M3 : code(x.scalar_type());
    size_t bytes = 0;
    check(g_linear_size(xt, (int)T, (int)K, (int)N, act, &bytes), w);
    at::Tensor ws;
    if (bytes) ws = at::Tensor(at::detail::empty_cuda({(int64_t)bytes}, at::kByte, dev, std::nullopt));
    check(g_linear(x.data_ptr(), ldx, xt, xsc, (const uint8_t*)wt.data_ptr(), wsc, act, base, ldb, out.data_ptr(), ldo,
                   code(out.scalar_type()), (int)T, (int)K, (int)N, bytes ? ws.data_ptr() : nullptr, bytes,
                   (moe_stream_t)place.stream),
          w);
    return THPVariable_Wrap(std::move(out));
  });
}

// init(refuse, enter, leave, route, adapters, few, quantize, linear, linear's workspace size): the refusal and the C
// functions' addresses
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 9)) return nullptr;
  Py_INCREF(a[0]);
  g_refuse = a[0];
  g_key = PyUnicode_InternFromString("_key");
  g_enter = (decltype(g_enter))PyLong_AsVoidPtr(a[1]);
  g_leave = (decltype(g_leave))PyLong_AsVoidPtr(a[2]);
  g_route = (decltype(g_route))PyLong_AsVoidPtr(a[3]);
  g_adapters = (decltype(g_adapters))PyLong_AsVoidPtr(a[4]);
  g_few = (decltype(g_few))PyLong_AsVoidPtr(a[5]);
  g_quantize = (decltype(g_quantize))PyLong_AsVoidPtr(a[6]);
  g_linear = (decltype(g_linear))PyLong_AsVoidPtr(a[7]);
  g_linear_size = (decltype(g_linear_size))PyLong_AsVoidPtr(a[8]);
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {{"init", (PyCFunction)(void*)init, METH_FASTCALL, nullptr},
                           {"enter", (PyCFunction)(void*)enter, METH_FASTCALL, nullptr},
                           {"leave", (PyCFunction)(void*)leave, METH_FASTCALL, nullptr},
                           {"route", (PyCFunction)(void*)route, METH_FASTCALL, nullptr},
                           {"adapters", (PyCFunction)(void*)adapters, METH_FASTCALL, nullptr},
                           {"few", (PyCFunction)(void*)few, METH_FASTCALL, nullptr},
                           {"quantize", (PyCFunction)(void*)quantize, METH_FASTCALL, nullptr},
                           {"linear", (PyCFunction)(void*)linear, METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_block_ext", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__block_ext(void) { return PyModule_Create(&g_module); }
