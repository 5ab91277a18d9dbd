// attn_bind.cpp -- Python extension module _attn_native: checks the tensors of
// an attention call or of one of a hybrid's other operators, fills its descriptor
// and calls the C ABI (include/gdn_attn.h, include/gdn_hybrid.h).  Argument
// marshalling only.
//
// A decode step's calls are so short that the host's share decides how fast
// they follow each other; the same checks made from Python cost 5 us a call.
// The module is bound to no library: every call is given the address of the C
// function, so that attn.py decides which one runs.  It returns the status;
// what cannot be marshalled raises ValueError.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#define __HIP_PLATFORM_AMD__ 1
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <exception>
#include <initializer_list>
#include <string>

#include "gdn_hybrid.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refused : std::exception {
  std::string text;
  explicit Refused(std::string t) : text(std::move(t)) {}
  const char* what() const noexcept override { return text.c_str(); }
};

std::string type_name(ScalarType t) {
  switch (t) {
    case ScalarType::Float: return "torch.float32";
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Float8_e4m3fn: return "torch.float8_e4m3fn";
    case ScalarType::Byte: return "torch.uint8";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    default: return c10::toString(t);
  }
}

std::string shape_name(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// The tensor `name`, on device dev, of this type and shape.
const Tensor& like(PyObject* o, const char* name, int dev, at::IntArrayRef shape, ScalarType type) {
  const Tensor& t = tensor(o, name);
  const std::string n(name);
  if (!t.is_cuda()) throw Refused(n + " must be a device tensor");
  if (t.get_device() != dev) throw Refused(n + " must be on the same device as the other tensors");
  if (t.scalar_type() != type)
    throw Refused(n + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
  if (t.sizes() != shape)
    throw Refused(n + " has shape " + shape_name(t.sizes()) + ", expected " + shape_name(shape));
  return t;
}

// The address of a contiguous tensor (None: NULL).
void* dense(PyObject* o, const char* name, int dev, at::IntArrayRef shape, ScalarType type) {
  if (o == Py_None) return nullptr;
  const Tensor& t = like(o, name, dev, shape, type);
  if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
  return t.data_ptr();
}

// The address and row stride (elements) of a [rows, H, d] tensor whose rows are
// dense; a column block of a wider buffer is fine.
void* heads(PyObject* o, const char* name, int dev, int64_t rows, int64_t H, int64_t d,
            ScalarType type, int64_t* ld) {
  const Tensor& t = like(o, name, dev, {rows, H, d}, type);
  const auto s = t.strides();
  if ((s[2] != 1 || (s[1] != d && H > 1)) && rows * H > 0)
    throw Refused(std::string(name) + " must have dense rows of " + std::to_string(H) + " x " +
                  std::to_string(d) + " elements");
  *ld = rows > 1 ? s[0] : H * d;
  return t.data_ptr();
}

// The [rows, heads, head size] tensor that sets device and type of a call.
const Tensor& first(PyObject* o, const char* name) {
  const Tensor& t = tensor(o, name);
  const std::string n(name);
  if (!t.is_cuda()) throw Refused(n + " must be a device tensor");
  if (t.scalar_type() != ScalarType::Float && t.scalar_type() != ScalarType::BFloat16)
    throw Refused(n + " must be float32 or bfloat16");
  if (t.dim() != 3) throw Refused(n + " must have 3 dimensions (rows, heads, head size)");
  return t;
}

int32_t io_of(ScalarType t) { return t == ScalarType::Float ? GDN_F32 : GDN_BF16; }

int32_t narrow(int64_t x, const char* what) {
  if (x > INT32_MAX) throw Refused(std::string(what) + " is too large");
  return (int32_t)x;
}

// rope_dim and the frequencies' address.
int32_t rope_of(PyObject* o, int dev, const float** f) {
  *f = nullptr;
  if (o == Py_None) return 0;
  const Tensor& t = tensor(o, "inv_freq");
  if (t.dim() != 1) throw Refused("inv_freq must be a 1-d tensor of rope_dim / 2 frequencies");
  const void* p = dense(o, "inv_freq", dev, t.sizes(), ScalarType::Float);
  if (t.numel() == 0) return 0;
  *f = static_cast<const float*>(p);
  return narrow(2 * t.numel(), "inv_freq");
}

// The sequences of a packed (offsets) or equal-length batch.
int64_t packed(PyObject* cu, PyObject* n, int dev, const int64_t** offsets) {
  *offsets = nullptr;
  int64_t want = -1;
  if (n != Py_None) {
    want = PyLong_AsLongLong(n);
    if (want == -1 && PyErr_Occurred()) { PyErr_Clear(); throw Refused("N must be an integer"); }
  }
  if (cu == Py_None) return n == Py_None ? 1 : want;
  const Tensor& t = tensor(cu, "cu_seqlens");
  if (t.dim() != 1 || t.numel() < 1)
    throw Refused("cu_seqlens must be a 1-d tensor of N + 1 offsets");
  if (n != Py_None && want + 1 != t.numel())
    throw Refused("cu_seqlens has " + std::to_string(t.numel()) + " offsets, expected N + 1 = " +
                  std::to_string(want + 1));
  *offsets = static_cast<const int64_t*>(dense(cu, "cu_seqlens", dev, t.sizes(), ScalarType::Long));
  return t.numel() - 1;
}

struct Cache {
  int64_t pages, N, width;
  int32_t Hk, P, d;
  void *k, *v;
  float *ks, *vs;
  const int32_t* table;
  const int64_t* lens;
};
// a: k_cache, v_cache, k_scale, v_scale, page_table, seq_lens
Cache cache_of(PyObject* const* a, int dev) {
  const Tensor& k = tensor(a[0], "k_cache");
  if (k.dim() != 4) throw Refused("k_cache must be [num_pages, H_k, page_size, d]");
  const Tensor& t = tensor(a[4], "page_table");
  if (t.dim() != 2) throw Refused("page_table must be [N, max_pages]");
  const auto s = k.sizes(), ts = t.sizes();
  Cache c;
  c.pages = s[0];
  c.Hk = narrow(s[1], "H_k");
  c.P = narrow(s[2], "page_size");
  c.d = narrow(s[3], "d");
  c.N = ts[0];
  c.width = ts[1];
  c.k = dense(a[0], "k_cache", dev, s, ScalarType::Float8_e4m3fn);
  c.v = dense(a[1], "v_cache", dev, s, ScalarType::Float8_e4m3fn);
  c.ks = static_cast<float*>(dense(a[2], "k_scale", dev, {s[0], s[1]}, ScalarType::Float));
  c.vs = static_cast<float*>(dense(a[3], "v_scale", dev, {s[0], s[1]}, ScalarType::Float));
  c.table = static_cast<const int32_t*>(dense(a[4], "page_table", dev, ts, ScalarType::Int));
  c.lens = static_cast<const int64_t*>(dense(a[5], "seq_lens", dev, {ts[0]}, ScalarType::Long));
  return c;
}

double number(PyObject* o, const char* name) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be a number");
  }
  return x;
}
int64_t integer(PyObject* o, const char* name) {
  const int64_t x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be an integer of 64 bits");
  }
  return x;
}
float scale_of(PyObject* o, int64_t d) {
  return o == Py_None ? (float)(1.0 / std::sqrt((double)d)) : (float)number(o, "scale");
}

template <typename Fn>
Fn function(PyObject* o) { return reinterpret_cast<Fn>(PyLong_AsVoidPtr(o)); }
void* handle(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) { PyErr_Clear(); throw Refused("stream is no handle of a stream"); }
  return p;
}
bool truth(PyObject* o, const char* name) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) { PyErr_Clear(); throw Refused(std::string(name) + " must be true or false"); }
  return x != 0;
}

// Runs `call` with dev as the current device.
template <typename F>
PyObject* on_device(int dev, F call) {
  int now = dev;
  (void)hipGetDevice(&now);
  gdn_status st;
  if (now == dev) {
    st = call();
  } else {
    if (hipSetDevice(dev) != hipSuccess) return PyLong_FromLong(GDN_ERR_HIP);
    st = call();
    (void)hipSetDevice(now);
  }
  return PyLong_FromLong((long)st);
}

// An exception of torch's own, as its allocations raise them.
void raise_torch(const char* name, const char* text) {
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* type = torch ? PyObject_GetAttrString(torch, name) : nullptr;
  if (type) PyErr_SetString(type, text);    // (otherwise the import has raised)
  Py_XDECREF(type);
  Py_XDECREF(torch);
}

// Turns what a body throws into a Python error.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const c10::OutOfMemoryError& e) {
    raise_torch("OutOfMemoryError", e.what());
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
}

// (fn, q_raw, k_raw, positions, inv_freq, q_weight, k_weight, interleaved, rope_scale, eps, q, k, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const bool has_q = a[1] != Py_None, has_k = a[2] != Py_None;
    if (!has_q && !has_k) throw Refused("q_raw or k_raw must be given");
    const Tensor& one = has_q ? first(a[1], "q_raw") : first(a[2], "k_raw");
    const int dev = (int)one.get_device();
    const ScalarType io = one.scalar_type();
    const int64_t rows = one.size(0), d = one.size(2);
    gdn_qk_desc desc{};
    desc.rows = rows;
    desc.d = narrow(d, "d");
    desc.io_dtype = io_of(io);
    const void *q_in = nullptr, *k_in = nullptr;
    void *q = nullptr, *k = nullptr;
    if (has_q) {
      desc.H_q = narrow(one.size(1), "H_q");
      q_in = heads(a[1], "q_raw", dev, rows, desc.H_q, d, io, &desc.ld_q);
      q = dense(a[10], "q", dev, {rows, desc.H_q, d}, io);
    } else if (a[10] != Py_None) {
      throw Refused("q without q_raw");
    }
    if (has_k) {
      const Tensor& t = first(a[2], "k_raw");
      desc.H_k = narrow(t.size(1), "H_k");
      k_in = heads(a[2], "k_raw", dev, rows, desc.H_k, d, io, &desc.ld_k);
      k = dense(a[11], "k", dev, {rows, desc.H_k, d}, io);
    } else if (a[11] != Py_None) {
      throw Refused("k without k_raw");
    }
    if (a[4] != Py_None && a[3] == Py_None) throw Refused("rotation needs positions");
    const float* freqs;
    desc.rope_dim = rope_of(a[4], dev, &freqs);
    const void* pos = dense(a[3], "positions", dev, {rows}, ScalarType::Long);
    const void* qw = dense(a[5], "q_weight", dev, {d}, ScalarType::Float);
    const void* kw = dense(a[6], "k_weight", dev, {d}, ScalarType::Float);
    desc.rope_mode = truth(a[7], "interleaved") ? GDN_ROPE_INTERLEAVED : GDN_ROPE_HALF;
    desc.rope_scale = (float)number(a[8], "rope_scale");
    desc.eps = (float)number(a[9], "eps");
    const auto fn = function<decltype(&gdn_qk_norm_rope)>(a[0]);
    void* stream = handle(a[12]);
    return on_device(dev, [&] {
      return fn(&desc, q_in, k_in, static_cast<const float*>(qw), static_cast<const float*>(kw),
                desc.rope_dim ? static_cast<const int64_t*>(pos) : nullptr, freqs, q, k,
                stream);
    });
  });
}

// (fn, k_raw, v_raw, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, cu_seqlens, inv_freq, k_weight,
//  interleaved, rope_scale, eps, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const Tensor& k = first(a[1], "k_raw");
    const int dev = (int)k.get_device();
    const ScalarType io = k.scalar_type();
    const Cache c = cache_of(a + 3, dev);
    gdn_kv_append_desc desc{};
    desc.N = c.N;
    desc.total_T = k.size(0);
    desc.num_pages = c.pages;
    desc.max_pages = c.width;
    desc.H_k = c.Hk;
    desc.d = c.d;
    desc.page_size = c.P;
    desc.io_dtype = io_of(io);
    const void* k_in = heads(a[1], "k_raw", dev, desc.total_T, c.Hk, c.d, io, &desc.ld_k);
    const void* v_in = heads(a[2], "v_raw", dev, desc.total_T, c.Hk, c.d, io, &desc.ld_v);
    const int64_t* cu;
    if (a[9] != Py_None && packed(a[9], Py_None, dev, &cu) != c.N)
      throw Refused("cu_seqlens has " + std::to_string(tensor(a[9], "cu_seqlens").numel()) +
                    " offsets, expected N + 1 = " + std::to_string(c.N + 1));
    if (a[9] == Py_None) cu = nullptr;
    const float* freqs;
    desc.rope_dim = rope_of(a[10], dev, &freqs);
    const void* kw = dense(a[11], "k_weight", dev, {c.d}, ScalarType::Float);
    desc.rope_mode = truth(a[12], "interleaved") ? GDN_ROPE_INTERLEAVED : GDN_ROPE_HALF;
    desc.rope_scale = (float)number(a[13], "rope_scale");
    desc.eps = (float)number(a[14], "eps");
    const auto fn = function<decltype(&gdn_kv_append)>(a[0]);
    void* stream = handle(a[15]);
    return on_device(dev, [&] {
      return fn(&desc, cu, c.lens, c.table, k_in, v_in, static_cast<const float*>(kw), freqs, c.k,
                c.v, c.ks, c.vs, stream);
    });
  });
}

// (fn, q, k, v, cu_seqlens, N, window, scale, o, stream)
PyObject* attn_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Tensor& q = first(a[1], "q");
    const int dev = (int)q.get_device();
    const ScalarType io = q.scalar_type();
    const int64_t T = q.size(0), d = q.size(2);
    gdn_attn_prefill_desc desc{};
    desc.total_T = T;
    desc.H_q = narrow(q.size(1), "H_q");
    desc.H_k = narrow(first(a[2], "k").size(1), "H_k");
    desc.d = narrow(d, "d");
    desc.io_dtype = io_of(io);
    const void* q_in = heads(a[1], "q", dev, T, desc.H_q, d, io, &desc.ld_q);
    const void* k_in = heads(a[2], "k", dev, T, desc.H_k, d, io, &desc.ld_k);
    const void* v_in = heads(a[3], "v", dev, T, desc.H_k, d, io, &desc.ld_v);
    const int64_t* cu;
    desc.N = packed(a[4], a[5], dev, &cu);
    desc.window = integer(a[6], "window");
    desc.scale = scale_of(a[7], d);
    void* o = dense(a[8], "o", dev, {T, desc.H_q, d}, io);
    const auto fn = function<decltype(&gdn_attn_prefill)>(a[0]);
    void* stream = handle(a[9]);
    return on_device(dev, [&] { return fn(&desc, cu, q_in, k_in, v_in, o, stream); });
  });
}

// (fn, size_fn, q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, window, scale, o, workspace, stream);
// a workspace that is needed and not given: minus its bytes
PyObject* attn_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const Tensor& q = first(a[2], "q");
    const int dev = (int)q.get_device();
    const ScalarType io = q.scalar_type();
    const Cache c = cache_of(a + 3, dev);
    gdn_attn_decode_desc desc{};
    desc.N = c.N;
    desc.num_pages = c.pages;
    desc.max_pages = c.width;
    desc.window = integer(a[9], "window");
    desc.H_q = narrow(q.size(1), "H_q");
    desc.H_k = c.Hk;
    desc.d = c.d;
    desc.page_size = c.P;
    desc.io_dtype = io_of(io);
    desc.scale = scale_of(a[10], c.d);
    const void* q_in = dense(a[2], "q", dev, {c.N, desc.H_q, c.d}, io);
    void* o = dense(a[11], "o", dev, {c.N, desc.H_q, c.d}, io);
    const size_t need = function<decltype(&gdn_attn_decode_workspace_size)>(a[1])(&desc);
    void* ws = nullptr;
    size_t bytes = 0;
    if (need) {
      if (a[12] == Py_None) return PyLong_FromLongLong(-(long long)need);
      const Tensor& t = tensor(a[12], "workspace");
      if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
        throw Refused("workspace must be a contiguous tensor on the device of the others");
      ws = t.data_ptr();
      bytes = t.nbytes();
    }
    const auto fn = function<decltype(&gdn_attn_decode)>(a[0]);
    void* stream = handle(a[13]);
    return on_device(dev, [&] {
      return fn(&desc, q_in, c.k, c.v, c.ks, c.vs, c.table, c.lens, o, ws, bytes, stream);
    });
  });
}

// Outputs and workspaces that are not given are allocated here, for the current stream of
// the device: from Python that costs as much again as the rest of a call.
Tensor make(int dev, at::IntArrayRef shape, ScalarType type) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)dev)));
}
// A contiguous output: the one given, or a new one in `made`.
void* out_dense(PyObject* o, const char* name, int dev, at::IntArrayRef shape, ScalarType type, Tensor* made) {
  if (o != Py_None) return dense(o, name, dev, shape, type);
  *made = make(dev, shape, type);
  return made->data_ptr();
}
void* out_heads(PyObject* o, const char* name, int dev, int64_t rows, int64_t H, int64_t d, ScalarType type,
                int64_t* ld, Tensor* made) {
  if (o != Py_None) return heads(o, name, dev, rows, H, d, type, ld);
  *made = make(dev, {rows, H, d}, type);
  *ld = H * d;
  return made->data_ptr();
}
// A new reference to what stands for an output: given, made or None.
PyObject* given_or(PyObject* o, const Tensor& made) {
  if (made.defined()) return THPVariable_Wrap(made);
  Py_INCREF(o);
  return o;
}
// (status, outputs ...)
template <size_t N>
PyObject* answer(PyObject* status, PyObject* const (&given)[N], const Tensor (&made)[N]) {
  if (!status) return nullptr;
  PyObject* r = PyTuple_New(N + 1);
  if (!r) { Py_DECREF(status); return nullptr; }
  PyTuple_SET_ITEM(r, 0, status);
  for (size_t i = 0; i < N; ++i) PyTuple_SET_ITEM(r, i + 1, given_or(given[i], made[i]));
  return r;
}

int64_t stats_words(int64_t T, int64_t Hq, ScalarType io, int64_t d) {
  return T * Hq * (io == ScalarType::BFloat16 ? 2 + d / 4 : 2);
}

// (fn, q, k, v, cu_seqlens, N, window, scale, o, stats, stream) -> (status, o, stats)
PyObject* attn_prefill_save(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Tensor& q = first(a[1], "q");
    const int dev = (int)q.get_device();
    const ScalarType io = q.scalar_type();
    const int64_t T = q.size(0), d = q.size(2);
    gdn_attn_prefill_desc desc{};
    desc.total_T = T;
    desc.H_q = narrow(q.size(1), "H_q");
    desc.H_k = narrow(first(a[2], "k").size(1), "H_k");
    desc.d = narrow(d, "d");
    desc.io_dtype = io_of(io);
    const void* q_in = heads(a[1], "q", dev, T, desc.H_q, d, io, &desc.ld_q);
    const void* k_in = heads(a[2], "k", dev, T, desc.H_k, d, io, &desc.ld_k);
    const void* v_in = heads(a[3], "v", dev, T, desc.H_k, d, io, &desc.ld_v);
    const int64_t* cu;
    desc.N = packed(a[4], a[5], dev, &cu);
    desc.window = integer(a[6], "window");
    desc.scale = scale_of(a[7], d);
    Tensor made[2];
    void* o = out_dense(a[8], "o", dev, {T, desc.H_q, d}, io, &made[0]);
    void* stats = out_dense(a[9], "stats", dev, {stats_words(T, desc.H_q, io, d)}, ScalarType::Float, &made[1]);
    const auto fn = function<decltype(&gdn_attn_prefill_save)>(a[0]);
    void* stream = handle(a[10]);
    PyObject* const given[2] = {a[8], a[9]};
    return answer(on_device(dev, [&] {
      return fn(&desc, cu, q_in, k_in, v_in, o, static_cast<float*>(stats), stream);
    }), given, made);
  });
}

// The workspace's address and bytes where `need` is not 0.
void* workspace_of(PyObject* o, int dev, size_t need, size_t* bytes, Tensor* made) {
  *bytes = 0;
  if (!need) return nullptr;
  if (o == Py_None) {
    *made = make(dev, {(int64_t)need}, ScalarType::Byte);
    *bytes = need;
    return made->data_ptr();
  }
  const Tensor& t = tensor(o, "workspace");
  if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
    throw Refused("workspace must be a contiguous tensor on the device of the others");
  *bytes = t.nbytes();
  return t.data_ptr();
}

// The type of an operand that may be fp32 beside bf16.
ScalarType second_type(const Tensor& t, const char* name) {
  const ScalarType s = t.scalar_type();
  if (s != ScalarType::Float && s != ScalarType::BFloat16)
    throw Refused(std::string(name) + " must be float32 or bfloat16");
  return s;
}

// (fn, size_fn, q, k, v, o, d_o, stats, cu_seqlens, N, window, scale, dq, dk, dv, grad_dtype is float32, workspace,
//  stream) -> (status, dq, dk, dv)
PyObject* attn_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 18, [&]() -> PyObject* {
    const Tensor& q = first(a[2], "q");
    const int dev = (int)q.get_device();
    const ScalarType io = q.scalar_type();
    const int64_t T = q.size(0), d = q.size(2);
    gdn_attn_bwd_desc desc{};
    desc.total_T = T;
    desc.H_q = narrow(q.size(1), "H_q");
    desc.H_k = narrow(first(a[3], "k").size(1), "H_k");
    desc.d = narrow(d, "d");
    desc.io_dtype = io_of(io);
    const void* q_in = heads(a[2], "q", dev, T, desc.H_q, d, io, &desc.ld_q);
    const void* k_in = heads(a[3], "k", dev, T, desc.H_k, d, io, &desc.ld_k);
    const void* v_in = heads(a[4], "v", dev, T, desc.H_k, d, io, &desc.ld_v);
    const void* o = dense(a[5], "o", dev, {T, desc.H_q, d}, io);
    const void* d_o = dense(a[6], "d_o", dev, {T, desc.H_q, d}, io);
    const void* stats = dense(a[7], "stats", dev, {stats_words(T, desc.H_q, io, d)}, ScalarType::Float);
    const int64_t* cu;
    desc.N = packed(a[8], a[9], dev, &cu);
    desc.window = integer(a[10], "window");
    desc.scale = scale_of(a[11], d);
    const ScalarType grad = truth(a[15], "grad_dtype") ? ScalarType::Float : ScalarType::BFloat16;
    desc.grad_dtype = io_of(grad);
    Tensor made[3], scratch;
    void* dq = out_heads(a[12], "dq", dev, T, desc.H_q, d, grad, &desc.ld_dq, &made[0]);
    void* dk = out_heads(a[13], "dk", dev, T, desc.H_k, d, grad, &desc.ld_dk, &made[1]);
    void* dv = out_heads(a[14], "dv", dev, T, desc.H_k, d, grad, &desc.ld_dv, &made[2]);
    const size_t need = function<decltype(&gdn_attn_backward_workspace_size)>(a[1])(&desc);
    size_t bytes;
    void* ws = workspace_of(a[16], dev, need, &bytes, &scratch);
    const auto fn = function<decltype(&gdn_attn_backward)>(a[0]);
    void* stream = handle(a[17]);
    PyObject* const given[3] = {a[12], a[13], a[14]};
    return answer(on_device(dev, [&] {
      return fn(&desc, cu, q_in, k_in, v_in, o, d_o, static_cast<const float*>(stats), ws, bytes,
                dq, dk, dv, stream);
    }), given, made);
  });
}

// (fn, size_fn, dq, dk, q_raw, k_raw, positions, inv_freq, q_weight, k_weight, interleaved, rope_scale, eps, dq_raw,
//  dk_raw, dq_weight, dk_weight, workspace, stream) -> (status, dq_raw, dk_raw, dq_weight, dk_weight)
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 19, [&]() -> PyObject* {
    const bool has_q = a[2] != Py_None, has_k = a[3] != Py_None;
    if (!has_q && !has_k) throw Refused("dq or dk must be given");
    const Tensor& one = has_q ? first(a[2], "dq") : first(a[3], "dk");
    const int dev = (int)one.get_device();
    const ScalarType grad = one.scalar_type();
    const int64_t rows = one.size(0), d = one.size(2);
    gdn_qk_bwd_desc desc{};
    desc.rows = rows;
    desc.d = narrow(d, "d");
    desc.grad_dtype = desc.io_dtype = io_of(grad);
    ScalarType io = grad;
    if (has_q && a[4] != Py_None) io = second_type(tensor(a[4], "q_raw"), "q_raw");
    else if (has_k && a[5] != Py_None) io = second_type(tensor(a[5], "k_raw"), "k_raw");
    desc.io_dtype = io_of(io);
    const void* up[2] = {nullptr, nullptr};
    const void* raw[2] = {nullptr, nullptr};
    void* out[2] = {nullptr, nullptr};
    const char* names[2][3] = {{"dq", "q_raw", "dq_raw"}, {"dk", "k_raw", "dk_raw"}};
    Tensor made[4], scratch;
    for (int i = 0; i < 2; ++i) {
      int32_t& H = i ? desc.H_k : desc.H_q;
      int64_t &ld = i ? desc.ld_k : desc.ld_q, &ldo = i ? desc.ld_dk : desc.ld_dq;
      if (a[2 + i] == Py_None) {
        if (a[4 + i] != Py_None || a[13 + i] != Py_None)
          throw Refused(std::string(names[i][1]) + " or " + names[i][2] + " without " + names[i][0]);
        continue;
      }
      H = narrow(first(a[2 + i], names[i][0]).size(1), "H");
      up[i] = dense(a[2 + i], names[i][0], dev, {rows, H, d}, grad);
      ld = (int64_t)H * d;
      if (a[4 + i] != Py_None) raw[i] = heads(a[4 + i], names[i][1], dev, rows, H, d, io, &ld);
      out[i] = out_heads(a[13 + i], names[i][2], dev, rows, H, d, grad, &ldo, &made[i]);
    }
    if (a[7] != Py_None && a[6] == Py_None) throw Refused("rotation needs positions");
    const float* freqs;
    desc.rope_dim = rope_of(a[7], dev, &freqs);
    const void* pos = dense(a[6], "positions", dev, {rows}, ScalarType::Long);
    const void* qw = dense(a[8], "q_weight", dev, {d}, ScalarType::Float);
    const void* kw = dense(a[9], "k_weight", dev, {d}, ScalarType::Float);
    desc.rope_mode = truth(a[10], "interleaved") ? GDN_ROPE_INTERLEAVED : GDN_ROPE_HALF;
    desc.rope_scale = (float)number(a[11], "rope_scale");
    desc.eps = (float)number(a[12], "eps");
    void* dqw = qw ? out_dense(a[15], "dq_weight", dev, {d}, ScalarType::Float, &made[2])
                   : dense(a[15], "dq_weight", dev, {d}, ScalarType::Float);
    void* dkw = kw ? out_dense(a[16], "dk_weight", dev, {d}, ScalarType::Float, &made[3])
                   : dense(a[16], "dk_weight", dev, {d}, ScalarType::Float);
    const size_t need = dqw || dkw
        ? function<decltype(&gdn_qk_norm_rope_backward_workspace_size)>(a[1])(&desc) : 0;
    size_t bytes;
    void* ws = workspace_of(a[17], dev, need, &bytes, &scratch);
    const auto fn = function<decltype(&gdn_qk_norm_rope_backward)>(a[0]);
    void* stream = handle(a[18]);
    PyObject* const given[4] = {a[13], a[14], a[15], a[16]};
    return answer(on_device(dev, [&] {
      return fn(&desc, up[0], up[1], raw[0], raw[1], static_cast<const float*>(qw),
                static_cast<const float*>(kw),
                desc.rope_dim ? static_cast<const int64_t*>(pos) : nullptr, freqs, ws, bytes, out[0],
                out[1], static_cast<float*>(dqw), static_cast<float*>(dkw), stream);
    }), given, made);
  });
}

// The [rows, C] tensor `name` on device dev (any if < 0) with dense rows, its type and row stride.
void* rows_of(PyObject* o, const char* name, int dev, int64_t rows, int64_t C, ScalarType type,
              int64_t* ld) {
  const Tensor& t = like(o, name, dev, {rows, C}, type);
  if (t.stride(1) != 1 && rows * C > 0 && C > 1)
    throw Refused(std::string(name) + " must have dense rows of " + std::to_string(C) + " elements");
  *ld = rows > 1 ? t.stride(0) : C;
  return t.data_ptr();
}
const Tensor& first_rows(PyObject* o, const char* name) {
  const Tensor& t = tensor(o, name);
  if (!t.is_cuda()) throw Refused(std::string(name) + " must be a device tensor");
  second_type(t, name);
  if (t.dim() != 2) throw Refused(std::string(name) + " must have 2 dimensions (rows, channels)");
  return t;
}

// (fn, x, res, weight, eps, group (None: y like x), res_out, y, y_scale, stream) -> (status, y, y_scale, res_out)
PyObject* add_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Tensor& x = first_rows(a[1], "x");
    const int dev = (int)x.get_device();
    const ScalarType io = x.scalar_type();
    const int64_t rows = x.size(0), C = x.size(1);
    gdn_add_norm_desc desc{};
    desc.rows = rows;
    desc.C = narrow(C, "C");
    desc.io_dtype = desc.res_dtype = io_of(io);
    desc.eps = (float)number(a[4], "eps");
    desc.group = -1;
    if (a[5] != Py_None) {
      const int64_t g = integer(a[5], "group");
      if (g < 0 || (g > 0 && C % g != 0))
        throw Refused("group must be None, 0 or a divisor of the row's channels");
      desc.group = narrow(g, "group");
    }
    const void* x_in = rows_of(a[1], "x", dev, rows, C, io, &desc.ld_x);
    ScalarType rt = io;
    if (a[2] != Py_None) rt = second_type(tensor(a[2], "res"), "res");
    else if (a[6] != Py_None) rt = second_type(tensor(a[6], "res_out"), "res_out");
    desc.res_dtype = io_of(rt);
    const void* res = dense(a[2], "res", dev, {rows, C}, rt);
    const void* weight = dense(a[3], "weight", dev, {C}, ScalarType::Float);
    Tensor made[3];
    void* res_out = res ? out_dense(a[6], "res_out", dev, {rows, C}, rt, &made[2])
                        : dense(a[6], "res_out", dev, {rows, C}, rt);
    const bool codes = desc.group >= 0;
    void* y = out_dense(a[7], "y", dev, {rows, C}, codes ? ScalarType::Float8_e4m3fn : io, &made[0]);
    void* scale = nullptr;
    if (codes) {
      scale = out_dense(a[8], "y_scale", dev, {rows, desc.group ? C / desc.group : 1}, ScalarType::Float, &made[1]);
    } else if (a[8] != Py_None) {
      throw Refused("y_scale without group");
    }
    const auto fn = function<decltype(&gdn_add_norm)>(a[0]);
    void* stream = handle(a[9]);
    PyObject* const given[3] = {a[7], a[8], a[6]};
    return answer(on_device(dev, [&] {
      return fn(&desc, x_in, res, static_cast<const float*>(weight), res_out, y,
                static_cast<float*>(scale), stream);
    }), given, made);
  });
}

// (fn, size_fn, dy, r, weight, d_res_out, eps, dx, d_res, d_weight, workspace, stream) -> (status, dx, d_res,
//  d_weight); dx is d_res where it is not given and the types are one
PyObject* add_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const Tensor& dy = first_rows(a[2], "dy");
    const int dev = (int)dy.get_device();
    const ScalarType io = dy.scalar_type();
    const int64_t rows = dy.size(0), C = dy.size(1);
    const ScalarType rt = second_type(tensor(a[3], "r"), "r");
    gdn_add_norm_bwd_desc desc{};
    desc.rows = rows;
    desc.C = narrow(C, "C");
    desc.ld_dx = C;
    desc.io_dtype = io_of(io);
    desc.res_dtype = io_of(rt);
    desc.eps = (float)number(a[6], "eps");
    const void* up = dense(a[2], "dy", dev, {rows, C}, io);
    const void* r = dense(a[3], "r", dev, {rows, C}, rt);
    const void* weight = dense(a[4], "weight", dev, {C}, ScalarType::Float);
    const void* dro = dense(a[5], "d_res_out", dev, {rows, C}, rt);
    Tensor made[3], scratch;
    const bool one = a[7] == Py_None && io == rt;
    void* d_res = out_dense(a[8], "d_res", dev, {rows, C}, rt, &made[1]);
    void* dx = nullptr;
    if (!one)
      dx = a[7] == Py_None ? out_dense(a[7], "dx", dev, {rows, C}, io, &made[0])
                           : rows_of(a[7], "dx", dev, rows, C, io, &desc.ld_dx);
    void* dw = weight ? out_dense(a[9], "d_weight", dev, {C}, ScalarType::Float, &made[2])
                      : dense(a[9], "d_weight", dev, {C}, ScalarType::Float);
    const size_t need = dw ? function<decltype(&gdn_add_norm_backward_workspace_size)>(a[1])(&desc) : 0;
    size_t bytes;
    void* ws = workspace_of(a[10], dev, need, &bytes, &scratch);
    const auto fn = function<decltype(&gdn_add_norm_backward)>(a[0]);
    void* stream = handle(a[11]);
    PyObject* const given[3] = {one ? a[8] : a[7], a[8], a[9]};
    if (one) made[0] = made[1];
    return answer(on_device(dev, [&] {
      return fn(&desc, up, r, static_cast<const float*>(weight), dro, ws, bytes, dx, d_res,
                static_cast<float*>(dw), stream);
    }), given, made);
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)),
                     METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<qk_norm_rope>("qk_norm_rope"), method<kv_append>("kv_append"),
                           method<attn_prefill>("attn_prefill"),
                           method<attn_decode>("attn_decode"),
                           method<attn_prefill_save>("attn_prefill_save"),
                           method<attn_backward>("attn_backward"),
                           method<qk_norm_rope_backward>("qk_norm_rope_backward"),
                           method<add_norm>("add_norm"),
                           method<add_norm_backward>("add_norm_backward"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_attn_native", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_native(void) {
  PyObject* m = PyModule_Create(&g_module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
