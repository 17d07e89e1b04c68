// Python calls of the operators around the expert products: argument checks,
// outputs and workspaces from torch's allocator, and the C entry on the tensors'
// device and its current stream.  In C++ because a call is short: with the same
// checks in Python and ctypes, three tokens' dispatch took 7.5 us of host time, of
// which the launch is 3.4; here it takes 3.9 to 4.9 (plan 7.4 and 4.6 to 5.4, the 8-bit
// product 13.5 and 7.1 to 8.5).  One token's route, whose five outputs are allocated
// one by one, takes 7.4 to 8.1 (1.6 less when they shared a storage, which their
// owner could then not save or free one by one).  A call of the gated product takes 5 to 7,
// a block norm 5.3, clipping of 4 tensors 8.5 and of 300 16; the gated feed-forward's forward and
// backward pass, eight entries, 117 (238 with a Python call for each).
//
// The C entries are those of the library that the package has loaded; setup()
// takes their addresses.

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
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
  X(grouped_fp8_quantize_weight) X(grouped_fp8_gemm_fwd_workspace_bytes) X(grouped_fp8_gemm_fwd)               \
  X(grouped_gated_gemm_fwd_workspace_bytes) X(grouped_gated_gemm_fwd)                                          \
  X(grouped_gated_gemm_dgrad_workspace_bytes) X(grouped_gated_gemm_dgrad) X(block_norm_fwd) X(block_norm_bwd)   \
  X(block_norm_bwd_workspace_bytes) X(grad_norm_workspace_bytes) X(grad_norm) X(grad_clip)                     \
  X(grouped_det_gemm_fwd_workspace_bytes) X(grouped_det_gemm_fwd) X(grouped_det_gemm_dgrad_workspace_bytes)    \
  X(grouped_det_gemm_dgrad) X(grouped_det_gemm_wgrad_workspace_bytes) X(grouped_det_gemm_wgrad)                \
  X(grouped_det_gemm_zero_pad_rows)

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

// A workspace query on t's device (what a call needs can depend on it).
template <class F, class... A>
size_t query(const Tensor& t, F entry, A... a) {
  const c10::DeviceGuard guard(t.device());
  return entry(a...);
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

// (None for a tensor that is not there)
template <class... T>
PyObject* tuple(const T&... t) {
  PyObject* out = PyTuple_New(sizeof...(t));
  if (!out) throw Raised();
  Py_ssize_t i = 0;
  const auto wrap = [](const Tensor& x) { return x.defined() ? THPVariable_Wrap(x) : (Py_INCREF(Py_None), Py_None); };
  const bool ok = ((PyTuple_SET_ITEM(out, i, wrap(t)), PyTuple_GET_ITEM(out, i++) != nullptr) && ...);
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

// The E cumulative end offsets of a tensor in either form.
const int32_t* need_offs(PyObject* o, int64_t E, const Tensor& like) {
  const Tensor& offs = any_tensor(o, "offs");
  if (offs.scalar_type() != ScalarType::Int || offs.dim() != 1 || !offs.is_cuda())
    refuse(PyExc_TypeError, "offs must be a 1-D int32 device tensor");
  if (!offs.is_contiguous()) refuse(PyExc_ValueError, "offs must be contiguous");
  need_device(offs, "offs", &like);
  if (offs.size(0) != E && offs.size(0) != E + 1)
    refuse(PyExc_ValueError, "offs has %lld entries; expected E=%lld (offs) or E+1 (m_indptr)",
           (long long)offs.size(0), (long long)E);
  const int32_t* p = ptr(offs);
  return p + (offs.size(0) - E);  // (skips m_indptr's leading zero)
}

// The caller's workspace (checked; *need becomes its size) or a fresh one.
Tensor need_workspace(PyObject* o, size_t* need, const Tensor& like) {
  if (o == Py_None) return scratch(like, *need);
  const Tensor& ws = any_tensor(o, "workspace");
  if (ws.scalar_type() != ScalarType::Byte || !ws.is_contiguous())
    refuse(PyExc_ValueError, "workspace must be a contiguous uint8 tensor");
  if ((size_t)ws.numel() < *need)
    refuse(PyExc_ValueError, "workspace too small: %lld < %lld bytes", (long long)ws.numel(), (long long)*need);
  need_device(ws, "workspace", &like);
  *need = (size_t)ws.numel();
  return ws;
}

// The caller's bf16 output of this shape or a fresh one; wrote() is what a call returns
// for it.
Tensor need_out(PyObject* o, const Tensor& like, std::initializer_list<int64_t> shape) {
  if (o == Py_None) return fresh(like, shape, ScalarType::BFloat16);
  const Tensor& out = tensor(o, "out", ScalarType::BFloat16, (int)shape.size(), &like);
  need_shape(out, "out", shape);
  return out;
}
PyObject* wrote(PyObject* o, const Tensor& out) {
  if (o == Py_None) return THPVariable_Wrap(out);
  if (!out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
  Py_INCREF(o);
  return o;
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
  const int32_t* op = need_offs(a[4], E, x);
  const Tensor out = need_out(a[5], x, {M, N});
  size_t need = g.grouped_fp8_gemm_fwd_workspace_bytes(M, N, K, size32(E), code);
  const Tensor ws = need_workspace(a[6], &need, x);
  call("grouped_fp8_gemm_fwd", g.grouped_fp8_gemm_fwd, x, ptr(x), code, xs, ptr(w), ptr(ws_), op, ptr(out), M, N, K,
       size32(E), ptr(ws), need);
  return wrote(a[5], out);
}

// ---------------------------------------------------------------------------
// the gated feed-forward
// ---------------------------------------------------------------------------
// h (and gate_up) of operands that are known to fit; `out`, `ws_given`: the caller's, or None.
Tensor gated_h(const Tensor& x, const Tensor& w, const int32_t* offs, int act, bool keep, Tensor* kept,
               PyObject* out = Py_None, PyObject* ws_given = Py_None) {
  const int64_t M = x.size(0), K = x.size(1), E = w.size(0), F = w.size(1) / 2;
  const Tensor h = need_out(out, x, {M, F});
  if (keep) *kept = fresh(x, {M, 2 * F}, ScalarType::BFloat16);
  size_t need = query(x, g.grouped_gated_gemm_fwd_workspace_bytes, M, F, K, size32(E));
  const Tensor ws = need_workspace(ws_given, &need, x);
  call("grouped_gated_gemm_fwd", g.grouped_gated_gemm_fwd, x, ptr(x), ptr(w), offs, ptr(h), ptr(*kept), act, M, F, K,
       size32(E), ptr(ws), need);
  return h;
}
Tensor gated_d(const Tensor& dy, const Tensor& w, const Tensor& gate_up, const int32_t* offs, int act, Tensor out,
               PyObject* ws_given = Py_None) {
  const int64_t M = dy.size(0), N = dy.size(1), E = w.size(0), F = w.size(2);
  if (!out.defined()) out = fresh(dy, {M, 2 * F}, ScalarType::BFloat16);
  size_t need = query(dy, g.grouped_gated_gemm_dgrad_workspace_bytes, M, N, F, size32(E));
  const Tensor ws = need_workspace(ws_given, &need, dy);
  call("grouped_gated_gemm_dgrad", g.grouped_gated_gemm_dgrad, dy, ptr(dy), ptr(w), ptr(gate_up), offs, ptr(out), act,
       M, N, F, size32(E), ptr(ws), need);
  return out;
}

// x, w, offs, activation's code, keep, out or None, workspace or None -> h, gate_up (None unless kept)
PyObject* gated_fwd(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x", ScalarType::BFloat16, 2);
  const Tensor& w = tensor(a[1], "w", ScalarType::BFloat16, 3, &x);
  if (w.size(2) != x.size(1))
    refuse(PyExc_ValueError, "x has K=%lld but w has K=%lld", (long long)x.size(1), (long long)w.size(2));
  if (w.size(1) % 2) refuse(PyExc_ValueError, "w must have an even number of rows (gate and up), got %lld", (long long)w.size(1));
  const int32_t* offs = need_offs(a[2], w.size(0), x);
  const int act = (int)integer(a[3], "activation");
  const bool keep = boolean(a[4], "keep");
  Tensor kept;
  const Tensor out = gated_h(x, w, offs, act, keep, &kept, a[5], a[6]);
  PyObject* r = tuple(out, kept);
  if (a[5] != Py_None) {  // (the caller's own object)
    PyObject* h = wrote(a[5], out);
    PyObject* old = PyTuple_GET_ITEM(r, 0);
    PyTuple_SET_ITEM(r, 0, h);
    Py_DECREF(old);
  }
  return r;
}

// dy, w_down, gate_up, offs, activation's code, out or None, workspace or None -> dgate_up
PyObject* gated_dgrad(PyObject* const* a) {
  const Tensor& dy = tensor(a[0], "dy", ScalarType::BFloat16, 2);
  const Tensor& w = tensor(a[1], "w_down", ScalarType::BFloat16, 3, &dy);
  const int64_t M = dy.size(0), F = w.size(2);
  if (w.size(1) != dy.size(1))
    refuse(PyExc_ValueError, "dy has N=%lld but w_down has N=%lld", (long long)dy.size(1), (long long)w.size(1));
  const Tensor& gate_up = tensor(a[2], "gate_up", ScalarType::BFloat16, 2, &dy);
  need_shape(gate_up, "gate_up", {M, 2 * F});
  const int32_t* offs = need_offs(a[3], w.size(0), dy);
  const int act = (int)integer(a[4], "activation");
  const Tensor out = need_out(a[5], dy, {M, 2 * F});
  gated_d(dy, w, gate_up, offs, act, out, a[6]);
  return wrote(a[5], out);
}

// The products of the block's other steps, on operands that are known to fit.
Tensor det_fwd(const Tensor& x, const Tensor& w, const int32_t* offs) {
  const int64_t M = x.size(0), E = w.size(0), N = w.size(1), K = w.size(2);
  const Tensor y = fresh(x, {M, N}, ScalarType::BFloat16);
  const size_t need = g.grouped_det_gemm_fwd_workspace_bytes(M, N, K, size32(E));
  const Tensor ws = scratch(x, need);
  call("grouped_det_gemm_fwd", g.grouped_det_gemm_fwd, x, ptr(x), ptr(w), offs, ptr(y), M, N, K, size32(E), ptr(ws), need);
  return y;
}
Tensor det_dgrad(const Tensor& d, const Tensor& w, const int32_t* offs) {
  const int64_t M = d.size(0), E = w.size(0), N = w.size(1), K = w.size(2);
  const Tensor dx = fresh(d, {M, K}, ScalarType::BFloat16);
  const size_t need = g.grouped_det_gemm_dgrad_workspace_bytes(M, N, K, size32(E));
  const Tensor ws = scratch(d, need);
  call("grouped_det_gemm_dgrad", g.grouped_det_gemm_dgrad, d, ptr(d), ptr(w), offs, ptr(dx), M, N, K, size32(E), ptr(ws),
       need);
  return dx;
}
Tensor det_wgrad(const Tensor& d, const Tensor& x, int64_t E, const int32_t* offs) {
  const int64_t M = d.size(0), N = d.size(1), K = x.size(1);
  const Tensor dw = fresh(d, {E, N, K}, ScalarType::BFloat16);
  const size_t need = g.grouped_det_gemm_wgrad_workspace_bytes(M, N, K, size32(E));
  const Tensor ws = scratch(d, need);
  call("grouped_det_gemm_wgrad", g.grouped_det_gemm_wgrad, d, ptr(d), ptr(x), offs, ptr(dw), (int)MDG_BF16, 0, M, N, K,
       size32(E), ptr(ws), need);
  return dw;
}
void zero_rows(const Tensor& t, int64_t E, const int32_t* offs) {
  call("grouped_det_gemm_zero_pad_rows", g.grouped_det_gemm_zero_pad_rows, t, ptr(t), offs, t.size(0), t.size(1) * 2,
       size32(E));
}

// x, w, w_down, offs, activation's code, what is kept (1: gate_up, 2: h)
// -> y (zeros in rows of no group), h, gate_up (None unless kept)
PyObject* ffn_fwd(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x", ScalarType::BFloat16, 2);
  const Tensor& w = tensor(a[1], "w_gate_up", ScalarType::BFloat16, 3, &x);
  const Tensor& w2 = tensor(a[2], "w_down", ScalarType::BFloat16, 3, &x);
  const int64_t E = w.size(0), F = w2.size(2);
  if (w.size(2) != x.size(1))
    refuse(PyExc_ValueError, "x has K=%lld but w_gate_up has K=%lld", (long long)x.size(1), (long long)w.size(2));
  if (w2.size(0) != E || w.size(1) != 2 * F)
    refuse(PyExc_ValueError, "w_gate_up %s and w_down %s do not belong together: [E, 2 F, K] and [E, N, F]",
           shape_name(w.sizes()).c_str(), shape_name(w2.sizes()).c_str());
  const int32_t* offs = need_offs(a[3], E, x);
  const int act = (int)integer(a[4], "activation");
  const int64_t keep = integer(a[5], "keep");
  Tensor kept;
  const Tensor h = gated_h(x, w, offs, act, keep & 1, &kept);
  const Tensor y = det_fwd(h, w2, offs);
  zero_rows(y, E, offs);
  return tuple(y, (keep & 2) ? h : Tensor(), kept);
}

// dy, w_down, gate_up, offs, activation's code, x, w, h, experts, what is wanted (1: dx, 2: dw, 4: dw_down; 8:
// dgate_up) -> dx (zeros in rows of no group), dw, dw_down, dgate_up.  What nothing wanted reads may be None: w_down and
// gate_up but for 1, 2 and 8, w but for 1, x but for 2, h but for 4.
PyObject* ffn_bwd(PyObject* const* a) {
  const Tensor& dy = tensor(a[0], "the output gradient", ScalarType::BFloat16, 2);
  const int64_t M = dy.size(0), E = integer(a[8], "experts"), want = integer(a[9], "need");
  const int32_t* offs = need_offs(a[3], E, dy);
  const int act = (int)integer(a[4], "activation");
  Tensor d, dx, dw, dw2;
  if (want & 11) {
    const Tensor& w2 = tensor(a[1], "w_down", ScalarType::BFloat16, 3, &dy);
    const int64_t F = w2.size(2);
    need_shape(w2, "w_down", {E, dy.size(1), F});
    const Tensor& gate_up = tensor(a[2], "gate_up", ScalarType::BFloat16, 2, &dy);
    need_shape(gate_up, "gate_up", {M, 2 * F});
    d = gated_d(dy, w2, gate_up, offs, act, Tensor());
  }
  if (want & 1) {
    const Tensor& w = tensor(a[6], "w_gate_up", ScalarType::BFloat16, 3, &dy);
    need_shape(w, "w_gate_up", {E, d.size(1), w.size(2)});
    dx = det_dgrad(d, w, offs);
    zero_rows(dx, E, offs);
  }
  if (want & 2) {
    const Tensor& x = tensor(a[5], "x", ScalarType::BFloat16, 2, &dy);
    need_rows(x, "x", M);
    dw = det_wgrad(d, x, E, offs);
  }
  if (want & 4) {
    const Tensor& h = tensor(a[7], "h", ScalarType::BFloat16, 2, &dy);
    need_rows(h, "h", M);
    dw2 = det_wgrad(dy, h, E, offs);
  }
  return tuple(dx, dw, dw2, (want & 8) ? d : Tensor());
}

// ---------------------------------------------------------------------------
// the norms around a block
// ---------------------------------------------------------------------------
float real(PyObject* o, const char* name) {
  const double v = PyFloat_Check(o) ? PyFloat_AS_DOUBLE(o) : PyLong_Check(o) && !PyBool_Check(o) ? PyLong_AsDouble(o) : NAN;
  if (PyErr_Occurred()) throw Raised();
  if (std::isnan(v)) refuse(PyExc_TypeError, "%s must be a number", name);
  return (float)v;
}

// A tensor of the type and shape of the rows it goes with, or nothing.
Tensor optional_rows(PyObject* o, const char* name, const Tensor& like) {
  if (o == Py_None) return Tensor();
  const Tensor& t = tensor(o, name, like.scalar_type(), 2, &like);
  if (t.sizes() != like.sizes()) refuse(PyExc_ValueError, "%s must have shape %s", name, shape_name(like.sizes()).c_str());
  return t;
}
Tensor optional_of_tokens(PyObject* o, const char* name, const Tensor& like) {
  if (o == Py_None) return Tensor();
  const Tensor& t = tensor(o, name, ScalarType::Float, 1, &like);
  need_shape(t, name, {like.size(0)});
  return t;
}

struct NormWeights {
  Tensor weight, post_weight;
  int code = MDG_FP32;
};
NormWeights need_norm_weights(PyObject* weight, PyObject* post_weight, const Tensor& like) {
  NormWeights w;
  int code[2];
  if (weight != Py_None) {
    w.weight = float_tensor(weight, "weight", 1, &code[0]);
    need_device(w.weight, "weight", &like);
    need_shape(w.weight, "weight", {like.size(1)});
    w.code = code[0];
  }
  if (post_weight != Py_None) {
    w.post_weight = float_tensor(post_weight, "post_weight", 1, &code[1]);
    need_device(w.post_weight, "post_weight", &like);
    need_shape(w.post_weight, "post_weight", {like.size(1)});
    if (w.weight.defined() && code[0] != code[1])
      refuse(PyExc_TypeError, "weight and post_weight must be of one type");
    w.code = code[1];
  }
  return w;
}

// residual, y, weight, post_weight, gate (each but the first may be None), scale, eps -> out, normed, rstd, post_rstd
PyObject* norm_fwd(PyObject* const* a) {
  int code;
  const Tensor& r = float_tensor(a[0], "residual", 2, &code);
  const Tensor y = optional_rows(a[1], "y", r);
  const NormWeights w = need_norm_weights(a[2], a[3], r);
  const Tensor gate = optional_of_tokens(a[4], "gate", r);
  const float scale = real(a[5], "scale"), eps = real(a[6], "eps");
  if (!y.defined() && (w.post_weight.defined() || gate.defined()))
    refuse(PyExc_ValueError, "post_weight and gate go with y");
  if (!y.defined() && !w.weight.defined()) refuse(PyExc_ValueError, "without y a weight is needed");
  const int64_t T = r.size(0), H = r.size(1);
  Tensor out, normed, rstd, post_rstd;
  if (y.defined()) out = fresh(r, {T, H}, r.scalar_type());
  if (w.weight.defined()) {
    normed = fresh(r, {T, H}, r.scalar_type());
    rstd = fresh(r, {T}, ScalarType::Float);
  }
  if (w.post_weight.defined()) post_rstd = fresh(r, {T}, ScalarType::Float);
  call("block_norm_fwd", g.block_norm_fwd, r, ptr(r), ptr(y), ptr(w.weight), ptr(w.post_weight), ptr(gate), ptr(out),
       ptr(normed), ptr(rstd), ptr(post_rstd), T, H, code, w.code, scale, eps);
  PyObject* got = tuple(out, normed, rstd, post_rstd);
  if (!out.defined()) {  // (the residual itself)
    PyObject* none = PyTuple_GET_ITEM(got, 0);
    Py_INCREF(a[0]);
    PyTuple_SET_ITEM(got, 0, a[0]);
    Py_DECREF(none);
  }
  return got;
}

// dout, dnormed, out (may be None without a weight), rstd, post_rstd, y, weight, post_weight, gate, scale, what is wanted (bits)
// -> dresidual, dy, dweight, dpost_weight, dgate
PyObject* norm_bwd(PyObject* const* a) {
  int code;
  const bool with_out = a[2] != Py_None;
  const Tensor& like = with_out ? float_tensor(a[2], "norm.out", 2, &code) : float_tensor(a[0], "dout", 2, &code);
  const Tensor out = with_out ? like : Tensor();
  const Tensor dout = optional_rows(a[0], "dout", like), dnormed = optional_rows(a[1], "dnormed", like);
  if (!dout.defined() && !dnormed.defined()) refuse(PyExc_ValueError, "dout or dnormed is needed");
  const Tensor rstd = optional_of_tokens(a[3], "norm.rstd", like), post_rstd = optional_of_tokens(a[4], "norm.post_rstd", like);
  const Tensor y = optional_rows(a[5], "y", like);
  const NormWeights w = need_norm_weights(a[6], a[7], like);
  const Tensor gate = optional_of_tokens(a[8], "gate", like);
  const float scale = real(a[9], "scale");
  const int64_t need = integer(a[10], "need"), T = like.size(0), H = like.size(1);
  if (!with_out && w.weight.defined()) refuse(PyExc_ValueError, "norm.out goes with a weight");
  if (dnormed.defined() && !w.weight.defined()) refuse(PyExc_ValueError, "dnormed goes with a weight");
  if (w.weight.defined() != rstd.defined() || w.post_weight.defined() != post_rstd.defined())
    refuse(PyExc_ValueError, "norm does not belong to these weights");
  if ((w.post_weight.defined() || gate.defined()) && !y.defined()) refuse(PyExc_ValueError, "post_weight and gate go with y");
  const ScalarType wt = w.code == MDG_FP32 ? ScalarType::Float : ScalarType::BFloat16;
  Tensor dr, dy, dw, dp, dg;
  if (need & 1) dr = fresh(like, {T, H}, like.scalar_type());
  if (need & 2) dy = fresh(like, {T, H}, like.scalar_type());
  if (need & 4) dw = fresh(like, {H}, wt);
  if (need & 8) dp = fresh(like, {H}, wt);
  if (need & 16) dg = fresh(like, {T}, ScalarType::Float);
  const size_t bytes = (need & 12) ? g.block_norm_bwd_workspace_bytes(T, H) : 0;
  const Tensor ws = scratch(like, bytes);
  call("block_norm_bwd", g.block_norm_bwd, like, ptr(dout), ptr(dnormed), ptr(out), ptr(y), ptr(w.weight),
       ptr(w.post_weight), ptr(gate), ptr(rstd), ptr(post_rstd), ptr(dr), ptr(dy), ptr(dw), ptr(dp), ptr(dg), T, H, code,
       w.code, scale, ptr(ws), bytes);
  return tuple(dr, dy, dw, dp, dg);
}

// ---------------------------------------------------------------------------
// the gradients' norm and clipping
// ---------------------------------------------------------------------------
struct Items {  // a sequence's items, held while the call runs (a list could change meanwhile)
  PyObject* items;
  Items(PyObject* o, const char* name) {
    if (THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a sequence of tensors, not one tensor", name);
    items = PySequence_Tuple(o);
    if (!items) throw Raised();
  }
  Items(const Items&) = delete;
  ~Items() { Py_DECREF(items); }
  Py_ssize_t size() const { return PyTuple_GET_SIZE(items); }
  PyObject* operator[](Py_ssize_t i) const { return PyTuple_GET_ITEM(items, i); }
};

const Tensor& need_gradient(PyObject* o, const char* name, const Tensor* like, int* code) {
  const Tensor& t = any_tensor(o, name);
  *code = dtype_code(t, name);
  if (t.layout() != at::kStrided) refuse(PyExc_ValueError, "%s must be dense", name);
  need_device(t, name, like);
  if (!t.is_non_overlapping_and_dense()) refuse(PyExc_ValueError, "%s must have no gaps or overlaps between its elements", name);
  return t;
}

std::vector<mdg_gradient> need_gradients(const Items& grads) {
  if (grads.size() == 0) refuse(PyExc_ValueError, "no gradients");
  std::vector<mdg_gradient> list((size_t)grads.size());
  const Tensor* like = nullptr;
  for (Py_ssize_t i = 0; i < grads.size(); ++i) {
    int code;
    const Tensor& t = need_gradient(grads[i], "a gradient", like, &code);
    if (!like) like = &t;
    list[i] = mdg_gradient{t.data_ptr(), t.data_ptr(), t.numel(), code, 0};
  }
  return list;
}

// grads -> norm
PyObject* grad_norm(PyObject* const* a) {
  const Items grads(a[0], "grads");
  const std::vector<mdg_gradient> list = need_gradients(grads);
  const Tensor& first = THPVariable_Unpack(grads[0]);
  const Tensor norm = fresh(first, {}, ScalarType::Float);
  const size_t need = g.grad_norm_workspace_bytes((int64_t)list.size());
  const Tensor ws = scratch(first, need);
  call("grad_norm", g.grad_norm, first, list.data(), (int64_t)list.size(), (float*)ptr(norm), (void*)ptr(ws), need);
  return THPVariable_Wrap(norm);
}

// grads, max_norm, norm or None, out or None -> norm
PyObject* clip_grads(PyObject* const* a) {
  const Items grads(a[0], "grads");
  std::vector<mdg_gradient> list = need_gradients(grads);
  const Tensor& first = THPVariable_Unpack(grads[0]);
  const float max_norm = real(a[1], "max_norm");
  if (max_norm < 0.0f) refuse(PyExc_ValueError, "max_norm must not be negative");
  const bool given = a[2] != Py_None;
  Tensor norm;
  if (given) norm = tensor(a[2], "norm", ScalarType::Float, 0, &first);
  const Items outs(a[3] == Py_None ? grads.items : a[3], "out");
  if (a[3] != Py_None) {
    if (outs.size() != grads.size())
      refuse(PyExc_ValueError, "out has %zd tensors, grads has %zd", outs.size(), grads.size());
    for (Py_ssize_t i = 0; i < outs.size(); ++i) {
      int code;
      const Tensor &t = need_gradient(outs[i], "an output", &first, &code), &x = THPVariable_Unpack(grads[i]);
      if (t.scalar_type() != x.scalar_type() || t.sizes() != x.sizes() || t.strides() != x.strides())
        refuse(PyExc_ValueError, "out[%zd] must have its gradient's type, shape and strides", i);
      list[i].out = t.data_ptr();
    }
  }
  if (!given) norm = fresh(first, {}, ScalarType::Float);
  const size_t need = given ? 0 : g.grad_norm_workspace_bytes((int64_t)list.size());
  const Tensor ws = scratch(first, need);
  call("grad_clip", g.grad_clip, first, list.data(), (int64_t)list.size(), max_norm, given ? (float*)ptr(norm) : nullptr,
       given ? nullptr : (float*)ptr(norm), (void*)ptr(ws), need);
  for (Py_ssize_t i = 0; i < outs.size(); ++i) {
    const Tensor& t = THPVariable_Unpack(outs[i]);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }
  if (!given) return THPVariable_Wrap(norm);
  Py_INCREF(a[2]);
  return a[2];
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
                         METHOD(gated_fwd, 7),     METHOD(gated_dgrad, 7),    METHOD(norm_fwd, 7),
                         METHOD(norm_bwd, 11),     METHOD(grad_norm, 1),      METHOD(clip_grads, 4),
                         METHOD(ffn_fwd, 6),       METHOD(ffn_bwd, 10),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
