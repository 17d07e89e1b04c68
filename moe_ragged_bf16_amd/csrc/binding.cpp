// Python calls of the operators around the expert products: argument checks,
// outputs and workspaces from torch's allocator, and the C entry on the tensors'
// device and its current stream.  In C++ because a call is short: with the same
// checks in Python and ctypes, three tokens' dispatch took 7.5 us of host time, of
// which the launch is 3.4; here it takes 3.9 to 4.9 (plan 7.4 and 4.6 to 5.4, the 8-bit
// product 13.5 and 7.1 to 8.5).  One token's route, whose five outputs are allocated
// one by one, takes 7.4 to 8.1 (1.6 less when they shared a storage, which their
// owner could then not save or free one by one).
//
// The C entries are those of the library that the package has loaded; setup()
// takes their addresses.

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>
#include <vector>

#include "moe_ragged_bf16.h"

namespace {

using at::ScalarType;
using at::Tensor;

// The entries, in the order of kNames.
#define MDG_ENTRIES(X)                                                                                         \
  X(moe_route_fwd_workspace_bytes) X(moe_route_fwd) X(moe_route_bwd) X(moe_plan_workspace_bytes) X(moe_plan)   \
  X(moe_dispatch_fwd) X(moe_dispatch_bwd) X(moe_combine_fwd) X(moe_combine_bwd) X(grouped_fp8_quantize_rows)   \
  X(grouped_fp8_quantize_weight) X(grouped_fp8_gemm_fwd_workspace_bytes) X(grouped_fp8_gemm_fwd)

struct Entries {
#define X(name) decltype(&::name) name = nullptr;
  MDG_ENTRIES(X)
#undef X
} g;
PyObject* g_stream = nullptr;  // f(device index): the current stream's address
PyObject* g_check = nullptr;   // f(entry, status): raises

// A Python error is set.
struct Raised {};

template <class... A>
[[noreturn]] void refuse(PyObject* type, const char* format, A... a) {
  PyErr_Format(type, format, a...);
  throw Raised();
}

std::string type_name(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Double: return "torch.float64";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    case ScalarType::Bool: return "torch.bool";
    case ScalarType::Byte: return "torch.uint8";
    case ScalarType::Float8_e4m3fn: return "torch.float8_e4m3fn";
    case ScalarType::Float8_e8m0fnu: return "torch.float8_e8m0fnu";
    default: return c10::toString(t);
  }
}

std::string shape_name(at::IntArrayRef s) {
  std::string out = "(";
  for (size_t i = 0; i < s.size(); ++i) out += (i ? ", " : "") + std::to_string(s[i]);
  return out + (s.size() == 1 ? ",)" : ")");
}

const Tensor& any_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

void need_type(const Tensor& t, const char* name, ScalarType type) {
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type).c_str(), type_name(t.scalar_type()).c_str());
}

void need_dims(const Tensor& t, const char* name, int dims) {
  if (t.dim() != dims) refuse(PyExc_ValueError, "%s must be %d-D, got shape %s", name, dims, shape_name(t.sizes()).c_str());
}

void need_device(const Tensor& t, const char* name, const Tensor* like) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be on a ROCm device, got %s", name, t.device().str().c_str());
  if (like && t.device() != like->device()) refuse(PyExc_ValueError, "all tensors must be on the same device");
}

void need_layout(const Tensor& t, const char* name, int dims, const Tensor* like) {
  need_dims(t, name, dims);
  need_device(t, name, like);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
}

const Tensor& tensor(PyObject* o, const char* name, ScalarType type, int dims, const Tensor* like = nullptr) {
  const Tensor& t = any_tensor(o, name);
  need_type(t, name, type);
  need_layout(t, name, dims, like);
  return t;
}

int dtype_code(const Tensor& t, const char* name) {
  if (t.scalar_type() == ScalarType::BFloat16) return MDG_BF16;
  if (t.scalar_type() == ScalarType::Float) return MDG_FP32;
  refuse(PyExc_TypeError, "%s must be bfloat16 or float32, got %s", name, type_name(t.scalar_type()).c_str());
}

const Tensor& float_tensor(PyObject* o, const char* name, int dims, int* code) {
  const Tensor& t = any_tensor(o, name);
  *code = dtype_code(t, name);
  need_layout(t, name, dims, nullptr);
  return t;
}

void need_shape(const Tensor& t, const char* name, std::initializer_list<int64_t> shape) {
  const at::IntArrayRef s(shape);
  if (t.sizes() != s) refuse(PyExc_ValueError, "%s must have shape %s", name, shape_name(s).c_str());
}

void need_rows(const Tensor& t, const char* name, int64_t rows) {
  if (t.size(0) != rows)
    refuse(PyExc_ValueError, "%s must have %lld rows, got %lld", name, (long long)rows, (long long)t.size(0));
}

int64_t integer(PyObject* o, const char* name) {
  if (!PyLong_Check(o) || PyBool_Check(o)) refuse(PyExc_TypeError, "%s must be an int", name);
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

// An entry's 32-bit size: what does not fit stays too large for every check.
int32_t size32(int64_t v) { return v > INT32_MAX ? INT32_MAX : v < INT32_MIN ? INT32_MIN : (int32_t)v; }

bool boolean(PyObject* o, const char* name) {
  if (!PyBool_Check(o)) refuse(PyExc_TypeError, "%s must be a bool", name);
  return o == Py_True;
}

// A tensor with a storage of its own.
Tensor fresh(const Tensor& like, at::IntArrayRef shape, ScalarType type) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

Tensor scratch(const Tensor& like, size_t bytes) {
  return bytes ? fresh(like, {(int64_t)bytes}, ScalarType::Byte) : Tensor();
}

// An address as whatever pointer an entry takes.
struct Address {
  void* p = nullptr;
  template <class T>
  operator T*() const {
    return static_cast<T*>(p);
  }
};
Address ptr(const Tensor& t) { return Address{t.defined() ? t.data_ptr() : nullptr}; }

[[noreturn]] void raise_status(const char* entry, int st) {
  PyObject* r = PyObject_CallFunction(g_check, "si", entry, st);
  if (r) PyErr_Format(PyExc_RuntimeError, "%s: status %d", entry, st);
  Py_XDECREF(r);
  throw Raised();
}

// Calls an entry on t's device with its current stream as the last argument.
template <class F, class... A>
void call(const char* name, F entry, const Tensor& t, A... a) {
  const c10::DeviceGuard guard(t.device());
  PyObject* index = PyLong_FromLong(t.get_device());
  PyObject* s = index ? PyObject_CallOneArg(g_stream, index) : nullptr;
  Py_XDECREF(index);
  if (!s) throw Raised();
  void* stream = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (!stream && PyErr_Occurred()) throw Raised();
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = (int)entry(a..., stream);
  Py_END_ALLOW_THREADS
  if (st != MDG_OK) raise_status(name, st);
}

template <class... T>
PyObject* tuple(const T&... t) {
  PyObject* out = PyTuple_New(sizeof...(t));
  if (!out) throw Raised();
  Py_ssize_t i = 0;
  const bool ok = ((PyTuple_SET_ITEM(out, i, THPVariable_Wrap(t)), PyTuple_GET_ITEM(out, i++) != nullptr) && ...);
  if (!ok) {
    Py_DECREF(out);
    throw Raised();
  }
  return out;
}

// A method: its body with C++ exceptions turned into Python ones.
template <PyObject* (*BODY)(PyObject* const*), Py_ssize_t N>
PyObject* method(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return BODY(args);
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::bad_alloc&) {
    return PyErr_NoMemory();
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
    return nullptr;
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// ---------------------------------------------------------------------------
// routing, rows
// ---------------------------------------------------------------------------
// logits, top_k, normalize, token_mask or None -> weight, idx, counts, loss, balance
PyObject* route_fwd(PyObject* const* a) {
  int code;
  const Tensor& logits = float_tensor(a[0], "logits", 2, &code);
  const int64_t k = integer(a[1], "top_k"), T = logits.size(0), E = logits.size(1);
  const bool normalize = boolean(a[2], "normalize");
  if (k < 1 || k > E)
    refuse(PyExc_ValueError, "top_k must be between 1 and the number of experts %lld, got %lld", (long long)E, (long long)k);
  Address mask;
  if (a[3] != Py_None) {
    const Tensor& m = tensor(a[3], "token_mask", ScalarType::Bool, 1, &logits);
    if (m.size(0) != T) refuse(PyExc_ValueError, "token_mask must have %lld entries", (long long)T);
    mask = ptr(m);
  }
  const Tensor weight = fresh(logits, {T, k}, ScalarType::Float), idx = fresh(logits, {T, k}, ScalarType::Int);
  const Tensor counts = fresh(logits, {E}, ScalarType::Int), loss = fresh(logits, {}, ScalarType::Float);
  const Tensor balance = fresh(logits, {E}, ScalarType::Float);
  const size_t need = g.moe_route_fwd_workspace_bytes(T, size32(E));
  const Tensor ws = scratch(logits, need);
  call("moe_route_fwd", g.moe_route_fwd, logits, ptr(logits), code, mask, ptr(weight), ptr(idx), ptr(counts),
       ptr(loss), ptr(balance), T, size32(E), size32(k), (int)normalize, ptr(ws), need);
  return tuple(weight, idx, counts, loss, balance);
}

// dweight or None, dloss or None, logits, weight, idx, balance, normalize -> dlogits
PyObject* route_bwd(PyObject* const* a) {
  int code;
  const Tensor& logits = float_tensor(a[2], "logits", 2, &code);
  const int64_t T = logits.size(0), E = logits.size(1);
  const Tensor& weight = tensor(a[3], "route.weight", ScalarType::Float, 2, &logits);
  const Tensor& idx = tensor(a[4], "route.idx", ScalarType::Int, 2, &logits);
  const Tensor& balance = tensor(a[5], "route.balance", ScalarType::Float, 1, &logits);
  const int64_t k = idx.size(1);
  if (idx.size(0) != T || weight.sizes() != idx.sizes() || balance.size(0) != E)
    refuse(PyExc_ValueError, "route does not belong to logits of this shape");
  const bool normalize = boolean(a[6], "normalize");
  Address dw, dl;
  if (a[0] != Py_None) {
    const Tensor& d = tensor(a[0], "dweight", ScalarType::Float, 2, &logits);
    need_shape(d, "dweight", {T, k});
    dw = ptr(d);
  }
  if (a[1] != Py_None) dl = ptr(tensor(a[1], "dloss", ScalarType::Float, 0, &logits));
  const Tensor out = fresh(logits, {T, E}, logits.scalar_type());
  call("moe_route_bwd", g.moe_route_bwd, logits, ptr(logits), code, ptr(weight), ptr(idx), ptr(balance), dw, dl,
       ptr(out), T, size32(E), size32(k), (int)normalize);
  return THPVariable_Wrap(out);
}

// idx, num_experts -> offs, dest
PyObject* plan(PyObject* const* a) {
  const Tensor& idx = tensor(a[0], "idx", ScalarType::Int, 2);
  const int64_t E = integer(a[1], "num_experts"), T = idx.size(0), k = idx.size(1);
  if (k < 1 || E < 1)
    refuse(PyExc_ValueError, "idx needs at least one column and num_experts at least one expert");
  if (E > (1 << 20)) raise_status("moe_plan", MDG_EUNSUPPORTED);  // (as the entry would, before offs of that size)
  const Tensor offs = fresh(idx, {E}, ScalarType::Int), dest = fresh(idx, {T, k}, ScalarType::Int);
  const size_t need = g.moe_plan_workspace_bytes(T, size32(k), size32(E));
  const Tensor ws = scratch(idx, need);
  call("moe_plan", g.moe_plan, idx, ptr(idx), ptr(offs), ptr(dest), T, size32(k), size32(E), ptr(ws), need);
  return tuple(offs, dest);
}

struct Plan {
  const Tensor &offs, &dest;
  int64_t tokens, top_k, experts;
};
Plan need_plan(PyObject* offs, PyObject* dest, const Tensor& like) {
  const Tensor& o = tensor(offs, "plan.offs", ScalarType::Int, 1, &like);
  const Tensor& d = tensor(dest, "plan.dest", ScalarType::Int, 2, &like);
  return Plan{o, d, d.size(0), d.size(1), o.size(0)};
}

// x, offs, dest -> rows
PyObject* dispatch_fwd(PyObject* const* a) {
  int code;
  const Tensor& x = float_tensor(a[0], "x", 2, &code);
  const Plan p = need_plan(a[1], a[2], x);
  need_rows(x, "x", p.tokens);
  const int64_t H = x.size(1);
  const Tensor rows = fresh(x, {p.tokens * p.top_k, H}, x.scalar_type());
  call("moe_dispatch_fwd", g.moe_dispatch_fwd, x, ptr(x), ptr(p.dest), ptr(p.offs),
       ptr(rows), p.tokens, size32(p.top_k), size32(p.experts), H, code);
  return THPVariable_Wrap(rows);
}

// drows, offs, dest -> dx
PyObject* dispatch_bwd(PyObject* const* a) {
  int code;
  const Tensor& d = float_tensor(a[0], "drows", 2, &code);
  const Plan p = need_plan(a[1], a[2], d);
  need_rows(d, "drows", p.tokens * p.top_k);
  const int64_t H = d.size(1);
  const Tensor dx = fresh(d, {p.tokens, H}, d.scalar_type());
  call("moe_dispatch_bwd", g.moe_dispatch_bwd, d, ptr(d), ptr(p.dest), ptr(dx), p.tokens,
       size32(p.top_k), H, code);
  return THPVariable_Wrap(dx);
}

// y, weight, offs, dest -> out
PyObject* combine_fwd(PyObject* const* a) {
  int code;
  const Tensor& y = float_tensor(a[0], "y", 2, &code);
  const Plan p = need_plan(a[2], a[3], y);
  need_rows(y, "y", p.tokens * p.top_k);
  const Tensor& w = tensor(a[1], "weight", ScalarType::Float, 2, &y);
  need_shape(w, "weight", {p.tokens, p.top_k});
  const int64_t H = y.size(1);
  const Tensor out = fresh(y, {p.tokens, H}, y.scalar_type());
  call("moe_combine_fwd", g.moe_combine_fwd, y, ptr(y), ptr(w), ptr(p.dest), ptr(out),
       p.tokens, size32(p.top_k), H, code);
  return THPVariable_Wrap(out);
}

// dout, y, weight, offs, dest -> dy, dweight
PyObject* combine_bwd(PyObject* const* a) {
  int code;
  const Tensor& y = float_tensor(a[1], "y", 2, &code);
  const Plan p = need_plan(a[3], a[4], y);
  need_rows(y, "y", p.tokens * p.top_k);
  const Tensor& w = tensor(a[2], "weight", ScalarType::Float, 2, &y);
  need_shape(w, "weight", {p.tokens, p.top_k});
  const int64_t H = y.size(1);
  const Tensor& dout = tensor(a[0], "dout", y.scalar_type(), 2, &y);
  need_shape(dout, "dout", {p.tokens, H});
  const Tensor dy = fresh(y, {p.tokens * p.top_k, H}, y.scalar_type());
  const Tensor dweight = fresh(y, {p.tokens, p.top_k}, ScalarType::Float);
  call("moe_combine_bwd", g.moe_combine_bwd, y, ptr(dout), ptr(y), ptr(w), ptr(p.dest),
       ptr(p.offs), ptr(dy), ptr(dweight), p.tokens, size32(p.top_k), size32(p.experts), H,
       code);
  return tuple(dy, dweight);
}

// ---------------------------------------------------------------------------
// the product in 8 bits
// ---------------------------------------------------------------------------
constexpr ScalarType kE4M3 = ScalarType::Float8_e4m3fn, kE8M0 = ScalarType::Float8_e8m0fnu;

int64_t blocks(int64_t n) { return (n + 127) / 128; }
int64_t pitch_of(int64_t n) { return (n + 15) / 16 * 16; }

// 8-bit values in rows at a pitch of whole 16 bytes (contiguous where the row
// length is a multiple of 16).
Tensor fresh_q(const Tensor& like, at::IntArrayRef shape) {
  const int64_t n = shape.back(), pitch = pitch_of(n);
  if (n == pitch) return fresh(like, shape, kE4M3);
  std::vector<int64_t> padded(shape.begin(), shape.end());
  padded.back() = pitch;
  return fresh(like, padded, kE4M3).narrow(-1, 0, n);
}

// A tensor laid out as by fresh_q.
const Tensor& q_tensor(PyObject* o, const char* name, int dims, const Tensor* like = nullptr) {
  const Tensor& t = any_tensor(o, name);
  need_type(t, name, kE4M3);
  if (t.dim() != dims || t.size(-1) % 16 == 0) {
    need_layout(t, name, dims, like);
    return t;
  }
  need_device(t, name, like);
  const int64_t pitch = pitch_of(t.size(-1));
  int64_t want = 1, rows = 1;
  bool ok = true;
  for (int64_t i = dims - 1; i >= 0; --i) {
    ok = ok && (t.size(i) <= 1 || t.stride(i) == want);
    want *= i == dims - 1 ? pitch : t.size(i);
    if (i < dims - 1) rows *= t.size(i);
  }
  if (!ok || (int64_t)t.storage().nbytes() - t.storage_offset() < rows * pitch)
    refuse(PyExc_ValueError, "%s must have its rows at a pitch of %lld bytes, zeros behind the values", name,
           (long long)pitch);
  return t;
}

// x -> q, scale
PyObject* quantize_rows(PyObject* const* a) {
  int code;
  const Tensor& x = float_tensor(a[0], "x", 2, &code);
  const int64_t M = x.size(0), K = x.size(1);
  const Tensor q = fresh_q(x, {M, K}), scale = fresh(x, {(blocks(K) + 3) / 4, M, 4}, kE8M0);
  call("grouped_fp8_quantize_rows", g.grouped_fp8_quantize_rows, x, ptr(x), code, ptr(q), ptr(scale), M, K);
  return tuple(q, scale);
}

// w, transpose -> q, scale[, qt, scale_t]
PyObject* quantize_weight(PyObject* const* a) {
  const Tensor& w = any_tensor(a[0], "w");
  const int code = dtype_code(w, "w");
  const bool transpose = boolean(a[1], "transpose");
  need_layout(w, "w", 3, nullptr);
  const int64_t E = w.size(0), N = w.size(1), K = w.size(2), nb = blocks(N), kb = blocks(K);
  const Tensor q = fresh_q(w, {E, N, K}), scale = fresh(w, {E, nb, kb}, kE8M0);
  Tensor qt, scale_t;
  if (transpose) {
    qt = fresh_q(w, {E, K, N});
    scale_t = fresh(w, {E, kb, nb}, kE8M0);
  }
  call("grouped_fp8_quantize_weight", g.grouped_fp8_quantize_weight, w, ptr(w), code, ptr(q), ptr(scale), ptr(qt),
       ptr(scale_t), size32(E), N, K);
  return transpose ? tuple(q, scale, qt, scale_t) : tuple(q, scale);
}

// x, x_scale or None, wq, w_scale, offs, out or None, workspace or None -> y
PyObject* fp8_gemm_fwd(PyObject* const* a) {
  int code = MDG_E4M3;
  const bool quantized = a[1] != Py_None;
  const Tensor& x = quantized ? q_tensor(a[0], "x.q", 2) : float_tensor(a[0], "x", 2, &code);
  const int64_t M = x.size(0), K = x.size(1);
  Address xs;
  if (quantized) {
    const Tensor& s = tensor(a[1], "x.scale", kE8M0, 3, &x);
    if (s.sizes() != at::IntArrayRef({(blocks(K) + 3) / 4, M, 4}))
      refuse(PyExc_ValueError, "x.scale does not belong to x.q");
    xs = ptr(s);
  }
  const Tensor& w = q_tensor(a[2], "wq", 3, &x);
  const int64_t E = w.size(0), N = w.size(1);
  if (w.size(2) != K)
    refuse(PyExc_ValueError, "x has K=%lld but wq has K=%lld", (long long)K, (long long)w.size(2));
  const Tensor& ws_ = tensor(a[3], "w_scale", kE8M0, 3, &x);
  need_shape(ws_, "w_scale", {E, blocks(N), blocks(K)});
  const Tensor& offs = any_tensor(a[4], "offs");
  if (offs.scalar_type() != ScalarType::Int || offs.dim() != 1 || !offs.is_cuda())
    refuse(PyExc_TypeError, "offs must be a 1-D int32 device tensor");
  if (!offs.is_contiguous()) refuse(PyExc_ValueError, "offs must be contiguous");
  need_device(offs, "offs", &x);
  if (offs.size(0) != E && offs.size(0) != E + 1)
    refuse(PyExc_ValueError, "offs has %lld entries; expected E=%lld (offs) or E+1 (m_indptr)",
           (long long)offs.size(0), (long long)E);
  const int32_t* op = ptr(offs);
  op += offs.size(0) - E;  // (skips m_indptr's leading zero)
  const bool given = a[5] != Py_None;
  Tensor out;
  if (given) {
    out = tensor(a[5], "out", ScalarType::BFloat16, 2, &x);
    need_shape(out, "out", {M, N});
  } else {
    out = fresh(x, {M, N}, ScalarType::BFloat16);
  }
  size_t need = g.grouped_fp8_gemm_fwd_workspace_bytes(M, N, K, size32(E), code);
  Tensor ws;
  if (a[6] == Py_None) {
    ws = scratch(x, need);
  } else {
    ws = any_tensor(a[6], "workspace");
    if (ws.scalar_type() != ScalarType::Byte || !ws.is_contiguous())
      refuse(PyExc_ValueError, "workspace must be a contiguous uint8 tensor");
    if ((size_t)ws.numel() < need)
      refuse(PyExc_ValueError, "workspace too small: %lld < %lld bytes", (long long)ws.numel(), (long long)need);
    need_device(ws, "workspace", &x);
    need = (size_t)ws.numel();
  }
  call("grouped_fp8_gemm_fwd", g.grouped_fp8_gemm_fwd, x, ptr(x), code, xs, ptr(w), ptr(ws_), op, ptr(out), M, N, K,
       size32(E), ptr(ws), need);
  if (!given) return THPVariable_Wrap(out);
  if (!out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
  Py_INCREF(a[5]);
  return a[5];
}

// addresses of the entries by name, f(device index) -> stream, f(entry, status)
PyObject* setup(PyObject* const* a) {
  if (!PyDict_Check(a[0])) refuse(PyExc_TypeError, "addresses must be a dict");
  Entries e;
#define X(name)                                                          \
  {                                                                      \
    PyObject* v = PyDict_GetItemString(a[0], #name);                     \
    if (!v) refuse(PyExc_KeyError, "%s", #name);                         \
    void* p = PyLong_AsVoidPtr(v);                                       \
    if (!p) refuse(PyExc_ValueError, "%s has no address", #name);        \
    e.name = reinterpret_cast<decltype(e.name)>(p);                      \
  }
  MDG_ENTRIES(X)
#undef X
  g = e;
  Py_INCREF(a[1]);
  Py_INCREF(a[2]);
  Py_XSETREF(g_stream, a[1]);
  Py_XSETREF(g_check, a[2]);
  Py_RETURN_NONE;
}

// the names setup() takes
PyObject* entries(PyObject* const*) {
  PyObject* out = PyList_New(0);
#define X(name)                                          \
  if (out) {                                             \
    PyObject* s = PyUnicode_FromString(#name);           \
    if (!s || PyList_Append(out, s) != 0) Py_CLEAR(out); \
    Py_XDECREF(s);                                       \
  }
  MDG_ENTRIES(X)
#undef X
  if (!out) throw Raised();
  return out;
}

#define METHOD(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&method<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(setup, 3),         METHOD(entries, 0),        METHOD(route_fwd, 4),
                         METHOD(route_bwd, 7),     METHOD(plan, 2),           METHOD(dispatch_fwd, 3),
                         METHOD(dispatch_bwd, 3),  METHOD(combine_fwd, 4),    METHOD(combine_bwd, 5),
                         METHOD(quantize_rows, 1), METHOD(quantize_weight, 2), METHOD(fp8_gemm_fwd, 7),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
