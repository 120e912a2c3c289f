// marshal.cpp — argument checks and marshalling of the serving-side entry points, for Python.
//
// These calls run many times per generated token and take a few microseconds of GPU time at
// serving's small sizes; looking at a dozen tensors from Python took longer than that.  Each
// function here takes its arguments by position, checks the tensors (device, type, shape,
// strides), and calls the C ABI on the given stream.  It returns the status code, or raises the
// binding's error for a tensor that does not fit.
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "dspark.h"

namespace {

PyObject* g_error = nullptr;  // the binding's exception class

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
[[noreturn]] void refuse(const std::string& what) { throw Refused(what); }

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kInt: return "torch.int32";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

const at::Tensor& cuda(PyObject* o, const char* name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  return THPVariable_Unpack(o);
}
void typed(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type) refuse(std::string(name) + " must be " + name_of(type) + ", got " + name_of(t.scalar_type()));
}
// The address of a contiguous CUDA tensor of `type` and n elements (n < 0: any number).
template <typename T = void>
T* flat(PyObject* o, const char* name, at::ScalarType type, int64_t n) {
  const at::Tensor& t = cuda(o, name);
  typed(t, name, type);
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  if (n >= 0 && t.numel() != n)
    refuse(std::string(name) + " must hold " + std::to_string(n) + " values, got " + std::to_string(t.numel()));
  return static_cast<T*>(const_cast<void*>(t.const_data_ptr()));
}
template <typename T = void>
T* flat_or_null(PyObject* o, const char* name, at::ScalarType type, int64_t n) {
  return o == Py_None ? nullptr : flat<T>(o, name, type, n);
}
int to_int(int64_t v, const char* name) {
  if (v > INT32_MAX || v < INT32_MIN) refuse(std::string(name) + " is out of range");
  return (int)v;
}
int integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::exception();
  return to_int(v, name);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw std::exception();
  return v;
}
void* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw std::exception();
  return p;
}

// A 2-D CUDA tensor with contiguous rows, any distance apart.
struct Rows {
  void* p;
  int n, m;
  int64_t stride;
  at::ScalarType type;
};
Rows rows(PyObject* o, const char* name) {
  const at::Tensor& t = cuda(o, name);
  if (t.dim() != 2) refuse(std::string(name) + " must be 2-D");
  const int64_t n = t.size(0), m = t.size(1);
  if (m > 1 && t.stride(1) != 1) refuse("the rows of " + std::string(name) + " must be contiguous");
  int64_t stride = t.stride(0);
  if (n <= 1) stride = m;  // the stride of one row means nothing
  else if (stride < m) refuse("the rows of " + std::string(name) + " overlap");
  return {const_cast<void*>(t.const_data_ptr()), to_int(n, name), to_int(m, name), stride, t.scalar_type()};
}
int logit_type(at::ScalarType t) {
  if (t == at::kFloat) return DSPARK_F32;
  if (t == at::kBFloat16) return DSPARK_BF16;
  if (t == at::kHalf) return DSPARK_F16;
  refuse(std::string("logits must be float32, bfloat16 or float16, got ") + name_of(t));
}
int cache_type(at::ScalarType t) {
  if (t == at::kBFloat16) return DSPARK_BF16;
  if (t == at::kHalf) return DSPARK_F16;
  if (t == at::kFloat8_e4m3fn) return DSPARK_E4M3;
  refuse("the pools must share a type: bfloat16, float16 or float8_e4m3fn");
}

struct Workspace {
  void* p;
  size_t bytes;
};
Workspace workspace(PyObject* o) {
  const at::Tensor& t = cuda(o, "ws");
  if (!t.is_contiguous()) refuse("ws must be contiguous");
  return {const_cast<void*>(t.const_data_ptr()), (size_t)t.numel() * t.element_size()};
}

// The tables of a cache: page_table, seq_len, ref_count.
struct Tables {
  int R, num_pages, width;
  int64_t stride;
  int32_t *table, *len, *ref;
};
Rows page_table(PyObject* o) {
  const Rows t = rows(o, "page_table");
  if (t.type != at::kInt) refuse(std::string("page_table must be torch.int32, got ") + name_of(t.type));
  return t;
}
Tables tables(PyObject* const* a) {
  const Rows t = page_table(a[0]);
  int32_t* ref = flat<int32_t>(a[2], "ref_count", at::kInt, -1);
  return {t.n, to_int(THPVariable_Unpack(a[2]).numel(), "ref_count"), t.m, t.stride, static_cast<int32_t*>(t.p),
          flat<int32_t>(a[1], "seq_len", at::kInt, t.n), ref};
}

// Two pools [num_pages, Hkv, page_size, D] with contiguous rows and the same strides (0 where a
// dimension has one entry, whose stride means nothing).
struct Pools {
  int64_t size[4], stride[3];
  int type;
  void *k, *v;
};
Pools pools(PyObject* ko, PyObject* vo) {
  const at::Tensor &k = cuda(ko, "k_pool"), &v = cuda(vo, "v_pool");
  Pools p;
  p.type = cache_type(k.scalar_type());
  if (v.scalar_type() != k.scalar_type()) refuse("the pools must share a type: bfloat16, float16 or float8_e4m3fn");
  if (k.dim() != 4 || v.sizes() != k.sizes() || k.stride(3) != 1 || v.stride(3) != 1)
    refuse("the pools must share a shape [num_pages, Hkv, page_size, D] with contiguous rows");
  for (int i = 0; i < 4; ++i) p.size[i] = k.size(i);
  for (int i = 0; i < 3; ++i) {
    p.stride[i] = p.size[i] > 1 ? k.stride(i) : 0;
    if (p.size[i] > 1 && v.stride(i) != k.stride(i)) refuse("the pools must share their strides");
  }
  p.k = const_cast<void*>(k.const_data_ptr());
  p.v = const_cast<void*>(v.const_data_ptr());
  return p;
}
// A CUDA tensor [T, heads, D] of 16-bit floats with contiguous rows.
struct TokenRows {
  void* p;
  int64_t T, heads, token, head;
  at::ScalarType type;
};
TokenRows token_rows(PyObject* o, const char* name, int64_t heads, int64_t D) {
  const at::Tensor& t = cuda(o, name);
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kHalf)
    refuse(std::string(name) + " must be bfloat16 or float16, got " + name_of(t.scalar_type()));
  if (t.dim() != 3 || (heads >= 0 && t.size(1) != heads) || t.size(2) != D || t.stride(2) != 1)
    refuse(std::string(name) + " must be [T, " + (heads < 0 ? "heads" : std::to_string(heads)) + ", " + std::to_string(D) +
           "] with contiguous rows");
  return {const_cast<void*>(t.const_data_ptr()), t.size(0), t.size(1), t.size(0) > 1 ? t.stride(0) : 0,
          t.size(1) > 1 ? t.stride(1) : 0, t.scalar_type()};
}

// (logits, tokens, temperature, top_k, logprob, entropy, lse, top_ids, top_logprobs, stream)
int token_logprobs(PyObject* const* a) {
  const Rows x = rows(a[0], "logits");
  const int dt = logit_type(x.type), K = integer(a[3], "top_k");
  const bool top = K > 0;
  return dspark_token_logprobs(x.n, x.m, x.stride, dt, x.p, flat<int32_t>(a[1], "tokens", at::kInt, x.n), (float)number(a[2]),
                               K, flat<float>(a[4], "logprob", at::kFloat, x.n),
                               flat<float>(a[5], "entropy", at::kFloat, x.n), flat<float>(a[6], "lse", at::kFloat, x.n),
                               top ? flat<int32_t>(a[7], "top_ids", at::kInt, (int64_t)x.n * K) : nullptr,
                               top ? flat<float>(a[8], "top_logprobs", at::kFloat, (int64_t)x.n * K) : nullptr, address(a[9]));
}

// (logits, tokens, lse, entropy, grad_logprob, grad_entropy, temperature, out, stream)
int token_logprobs_backward(PyObject* const* a) {
  const Rows x = rows(a[0], "logits"), y = rows(a[7], "out");
  const int dt = logit_type(x.type);
  if (y.type != x.type || y.n != x.n || y.m != x.m) refuse("out must have the logits' shape and type");
  return dspark_token_logprobs_backward(
      x.n, x.m, x.stride, y.stride, dt, x.p, flat<int32_t>(a[1], "tokens", at::kInt, x.n), (float)number(a[6]),
      flat<float>(a[2], "lse", at::kFloat, x.n), flat<float>(a[3], "entropy", at::kFloat, x.n),
      flat<float>(a[4], "grad_logprob", at::kFloat, x.n), flat_or_null<float>(a[5], "grad_entropy", at::kFloat, x.n), y.p,
      address(a[8]));
}

// (page_table, seq_len, ref_count, src, dst, page_size, ws, stream)
int cache_fork(PyObject* const* a) {
  const Tables t = tables(a);
  const int64_t F = cuda(a[3], "src").numel();
  const Workspace w = workspace(a[6]);
  return dspark_cache_fork(to_int(F, "src"), t.R, t.num_pages, integer(a[5], "page_size"), t.width, t.stride, t.table, t.len,
                           t.ref, flat<int32_t>(a[3], "src", at::kInt, F), flat<int32_t>(a[4], "dst", at::kInt, F), w.p,
                           w.bytes, address(a[7]));
}

// (page_table, seq_len, ref_count, n_new, page_size, n_pools, pools, page_bytes, granted, copies, ws, stream)
int cache_reserve(PyObject* const* a) {
  const Tables t = tables(a);
  const Workspace w = workspace(a[10]);
  return dspark_cache_reserve(t.R, t.num_pages, integer(a[4], "page_size"), t.width, t.stride, t.table, t.len, t.ref,
                              flat<int32_t>(a[3], "n_new", at::kInt, t.R), flat<int32_t>(a[8], "granted", at::kInt, t.R),
                              flat<int32_t>(a[9], "copies", at::kInt, 2 * (int64_t)t.R), integer(a[5], "n_pools"),
                              static_cast<void* const*>(address(a[6])), (size_t)PyLong_AsSize_t(a[7]), w.p, w.bytes,
                              address(a[11]));
}

// (k, v, k_pool, v_pool, page_table, seq_len, q_start, granted, k_scale, v_scale, ws, stream)
int cache_write(PyObject* const* a) {
  const Pools p = pools(a[2], a[3]);
  const int64_t H = p.size[1], D = p.size[3];
  const TokenRows k = token_rows(a[0], "k", H, D), v = token_rows(a[1], "v", H, D);
  if (k.type != v.type || k.T != v.T || k.token != v.token || k.head != v.head)
    refuse("k and v must share their type, shape and strides");
  const Rows t = page_table(a[4]);
  const Workspace w = workspace(a[10]);
  return dspark_cache_write(to_int(k.T, "k"), t.n, to_int(H, "Hkv"), to_int(D, "D"), to_int(p.size[0], "num_pages"),
                            to_int(p.size[2], "page_size"), t.m, cache_type(k.type), p.type, k.p, v.p, k.token, k.head, p.k,
                            p.v, p.stride[0], p.stride[1], p.stride[2], static_cast<int32_t*>(t.p), t.stride,
                            flat<int32_t>(a[5], "seq_len", at::kInt, t.n),
                            flat<int32_t>(a[6], "q_start", at::kInt, (int64_t)t.n + 1),
                            flat_or_null<int32_t>(a[7], "granted", at::kInt, t.n),
                            flat_or_null<float>(a[8], "k_scale", at::kFloat, H),
                            flat_or_null<float>(a[9], "v_scale", at::kFloat, H), w.p, w.bytes, address(a[11]));
}

// (page_table, seq_len, ref_count, new_len, page_size, ws, stream)
int cache_truncate(PyObject* const* a) {
  const Tables t = tables(a);
  const Workspace w = workspace(a[5]);
  return dspark_cache_truncate(t.R, t.num_pages, integer(a[4], "page_size"), t.width, t.stride, t.table, t.len, t.ref,
                               flat<int32_t>(a[3], "new_len", at::kInt, t.R), w.p, w.bytes, address(a[6]));
}

// (page_table, seq_len, ref_count, page_size, n_pools, pools, page_bytes, out, ws, stream)
int cache_compact(PyObject* const* a) {
  const Tables t = tables(a);
  const Workspace w = workspace(a[8]);
  return dspark_cache_compact(t.R, t.num_pages, integer(a[3], "page_size"), t.width, t.stride, t.table, t.len, t.ref,
                              flat<int32_t>(a[7], "out", at::kInt, 1), integer(a[4], "n_pools"),
                              static_cast<void* const*>(address(a[5])), (size_t)PyLong_AsSize_t(a[6]), w.p, w.bytes,
                              address(a[9]));
}

// (q, k_pool, v_pool, page_table, seq_len, q_start, max_q, scale, k_scale, v_scale, window, out, lse, ws, stream,
//  granted)
int paged_attention(PyObject* const* a) {
  const Pools p = pools(a[1], a[2]);
  const int64_t H = p.size[1], D = p.size[3];
  const TokenRows q = token_rows(a[0], "q", -1, D);
  const Rows t = page_table(a[3]);
  const Workspace w = workspace(a[13]);
  return dspark_paged_attention_granted(
      to_int(q.T, "q"), t.n, to_int(q.heads, "Hq"), to_int(H, "Hkv"), to_int(D, "D"), to_int(p.size[0], "num_pages"),
      to_int(p.size[2], "page_size"), t.m, integer(a[6], "max_q"), cache_type(q.type), p.type, q.p, q.token, q.head, p.k, p.v,
      p.stride[0], p.stride[1], p.stride[2], static_cast<int32_t*>(t.p), t.stride,
      flat<int32_t>(a[4], "seq_len", at::kInt, t.n), flat<int32_t>(a[5], "q_start", at::kInt, (int64_t)t.n + 1),
      flat_or_null<int32_t>(a[15], "granted", at::kInt, t.n), (float)number(a[7]), flat_or_null<float>(a[8], "k_scale", at::kFloat, H),
      flat_or_null<float>(a[9], "v_scale", at::kFloat, H), integer(a[10], "window"),
      flat(a[11], "out", q.type, q.T * q.heads * D), flat_or_null<float>(a[12], "lse", at::kFloat, q.T * q.heads), w.p, w.bytes,
      address(a[14]));
}

// A Python function of N positional arguments around F.
template <int (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are wanted, got %zd", N, n);
    return nullptr;
  }
  try {
    const int status = F(args);
    return PyErr_Occurred() ? nullptr : PyLong_FromLong(status);
  } catch (const Refused& e) {
    PyErr_SetString(g_error != nullptr ? g_error : PyExc_RuntimeError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
template <int (*F)(PyObject* const*), int N>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<F, N>)), METH_FASTCALL, nullptr};
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"set_error", set_error, METH_O, nullptr},
    method<token_logprobs, 10>("token_logprobs"),
    method<token_logprobs_backward, 9>("token_logprobs_backward"),
    method<cache_fork, 8>("cache_fork"),
    method<cache_reserve, 12>("cache_reserve"),
    method<cache_write, 12>("cache_write"),
    method<cache_truncate, 7>("cache_truncate"),
    method<cache_compact, 10>("cache_compact"),
    method<paged_attention, 16>("paged_attention"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&g_module); }
