// Marshalling of the serving calls: torch tensors -> the C ABI of include/lcp.h.
// A decode step makes several calls of a few microseconds of GPU time; reading
// tensors through Python attributes and ctypes took longer than the kernels
// (us a call on the host: lcp_rope 7.6, append 8.1, attend with its outputs 10.2; here
// 4.2, 4.6 and 6.1, where a torch elementwise call takes 4.3). Shapes, types, layouts and devices are
// checked here and raise ValueError or TypeError; everything else is the library's own
// validation, whose status is returned.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/core/Stream.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>

#include "../../include/lcp.h"

namespace {

// Raised as ValueError.
struct Bad {
  const char* what;
};

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Bad{what};
  return THPVariable_Unpack(o);
}

// Optional arguments: None is a null pointer.
const at::Tensor* maybe(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }

// The index of the GPU that all of a call's tensors (and its cache) are on.
int on_gpu(std::initializer_list<const at::Tensor*> all, int cache = -2) {
  int gpu = -2;
  for (const at::Tensor* t : all) {
    if (!t) continue;
    if (!t->is_cuda() || cache == -1) throw Bad{"tensors must be on the GPU"};
    const int at = t->get_device();
    if ((gpu != -2 && at != gpu) || (cache >= 0 && at != cache)) throw Bad{"tensors must be on one GPU"};
    gpu = at;
  }
  return gpu;
}

lcp_dtype dtype_of(const at::Tensor& t) { return t.scalar_type() == at::kFloat ? LCP_F32 : LCP_BF16; }

long long whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Bad{nullptr};
  return v;
}

int small(PyObject* o) {
  const long long v = whole(o);
  if (v < INT32_MIN || v > INT32_MAX) throw Bad{"a size does not fit 32 bits"};
  return (int)v;
}

int flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Bad{nullptr};
  return v;
}

// The package's function from a stream argument (None: the current stream) to a
// handle; called once the arguments are known to be good.
PyObject* handle_of = nullptr;

// The stream's handle for tensors on a GPU, which has to be the current one.
void* stream_of(PyObject* o, int gpu) {
  const c10::impl::VirtualGuardImpl device(c10::DeviceType::CUDA);
  const c10::Device now = device.getDevice();
  if (now.index() != gpu) throw Bad{"tensors must be on the current GPU"};
  if (o == Py_None && device.getStream(now).id() == 0) return nullptr;      // the default stream: no call into Python
  PyObject* h = handle_of ? PyObject_CallFunctionObjArgs(handle_of, o, nullptr) : nullptr;
  if (!h) throw Bad{handle_of ? nullptr : "use_streams has not been called"};
  void* s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (!s && PyErr_Occurred()) throw Bad{nullptr};
  return s;
}

// An index array of n entries.
const int32_t* index_of(const at::Tensor& t, int64_t n, const char* what) {
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous()) throw Bad{what};
  return static_cast<const int32_t*>(t.data_ptr());
}

// Head rows [T, heads, D], any strides, channels contiguous.
lcp_heads heads_of(const at::Tensor& x, const at::Tensor* y, int64_t T, int64_t D, at::ScalarType dt, const char* what) {
  if (x.dim() != 3 || x.size(0) != T || x.size(2) != D || x.scalar_type() != dt || x.stride(2) != 1 ||
      x.size(1) > INT32_MAX)
    throw Bad{what};
  lcp_heads h{x.data_ptr(), nullptr, (int)x.size(1), x.stride(0), x.stride(1), 0, 0};
  if (y) {
    if (y->sizes() != x.sizes() || y->scalar_type() != dt || y->stride(2) != 1)
      throw Bad{"an output must have its input's shape and dtype and contiguous channels"};
    h.y = y->data_ptr();
    h.y_token = y->stride(0);
    h.y_head = y->stride(1);
  }
  return h;
}

struct Table {
  const float* p = nullptr;
  int max_pos = 0, rot = 0;
};
Table table_of(const at::Tensor& t) {
  if (t.dim() != 3 || t.size(2) != 2 || t.scalar_type() != at::kFloat || !t.is_contiguous() || t.size(0) > INT32_MAX ||
      t.size(1) > INT32_MAX / 2)
    throw Bad{"table must be contiguous float32 [max_pos, rot_dim / 2, 2]"};
  return Table{static_cast<const float*>(t.data_ptr()), (int)t.size(0), (int)(2 * t.size(1))};
}

// The struct in a bytes-like object, and the index of its GPU (-1: none, -2: the
// object does not know).
template <typename T>
struct Held {
  Py_buffer b{};
  int gpu = -2;
  Held(PyObject* o, const char* what) {
    static PyObject* const name = PyUnicode_InternFromString("gpu");
    if (PyObject* g = PyObject_GetAttr(o, name)) {
      gpu = (int)PyLong_AsLong(g);
      Py_DECREF(g);
    }
    PyErr_Clear();
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Bad{nullptr};
    if (b.len != (Py_ssize_t)sizeof(T)) {
      PyBuffer_Release(&b);
      throw Bad{what};
    }
  }
  Held(const Held&) = delete;
  ~Held() { PyBuffer_Release(&b); }
  const T* operator->() const { return static_cast<const T*>(b.buf); }
  const T* get() const { return static_cast<const T*>(b.buf); }
};
struct Cache : Held<lcp_kv_cache> {
  explicit Cache(PyObject* o) : Held(o, "cache must be an lcp_kv_cache") {}
};

// Runs f, which may throw, for a method with n arguments.
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t n, F f) {
  HANDLE_TH_ERRORS
  if (given != n) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Bad& e) {
    if (e.what) PyErr_SetString(PyExc_ValueError, e.what);
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// rope(q, q_out, table, pos, k, k_out, interleaved, inverse, stream) -> status
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q must be a tensor"), &qo = tensor(a[1], "q_out must be a tensor");
    const at::Tensor *k = maybe(a[4], "k must be a tensor"), *ko = maybe(a[5], "k_out must be a tensor");
    if (q.dim() != 3) throw Bad{"q must be [T, heads, D]"};
    const at::ScalarType dt = q.scalar_type();
    if (dt != at::kFloat && dt != at::kBFloat16) {
      PyErr_SetString(PyExc_TypeError, "unsupported dtype: float32 or bfloat16");
      return nullptr;
    }
    const int64_t T = q.size(0), D = q.size(2);
    if (T > INT32_MAX || D > INT32_MAX) throw Bad{"q is too large"};
    const lcp_heads hq = heads_of(q, &qo, T, D, dt, "q must be [T, heads, D] with contiguous channels");
    lcp_heads hk{};
    if (k) {
      if (!ko) throw Bad{"k needs an output"};
      hk = heads_of(*k, ko, T, D, dt, "k must have q's tokens, channels and dtype, and contiguous channels");
    }
    const at::Tensor &tab = tensor(a[2], "table must be a tensor"), &at_pos = tensor(a[3], "pos must be a tensor");
    const Table t = table_of(tab);
    const int32_t* pos = index_of(at_pos, T, "pos must be contiguous int32 [T]");
    const int inter = flag(a[6]), inverse = flag(a[7]);
    const int gpu = on_gpu({&q, &qo, k, ko, &tab, &at_pos});
    void* s = stream_of(a[8], gpu);
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = lcp_rope(&hq, k ? &hk : nullptr, dtype_of(q), (int)T, (int)D, t.p, t.max_pos, pos, t.rot, inter, inverse, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(code);
  });
}

// cache(k, v, k_scale, v_scale) -> bytes of an lcp_kv_cache
PyObject* cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    const at::Tensor &k = tensor(a[0], "k must be a tensor"), &v = tensor(a[1], "v must be a tensor");
    lcp_kv_cache c{};
    switch (k.scalar_type()) {
      case at::kBFloat16: c.format = LCP_KV_BF16; break;
      case at::kFloat8_e4m3fn: c.format = LCP_KV_E4M3; break;
      case at::kChar: c.format = LCP_KV_INT8; break;
      default:
        PyErr_SetString(PyExc_TypeError, "unsupported cache dtype: bfloat16, float8_e4m3fn or int8");
        return nullptr;
    }
    if (k.dim() != 4 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type() || !k.is_contiguous() ||
        !v.is_contiguous())
      throw Bad{"k and v must be contiguous [pages, heads, page_size, D] of one dtype"};
    for (int i = 0; i < 4; ++i)
      if (k.size(i) > INT32_MAX) throw Bad{"the cache is too large"};
    if (v.device() != k.device()) throw Bad{"the cache must be on one device"};
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.pages = (int)k.size(0);
    c.heads = (int)k.size(1);
    c.page_size = (int)k.size(2);
    c.D = (int)k.size(3);
    if (c.format != LCP_KV_BF16) {
      const at::Tensor *s[2] = {maybe(a[2], "k_scale must be a tensor"), maybe(a[3], "v_scale must be a tensor")};
      for (const at::Tensor* t : s)
        if (!t || t->scalar_type() != at::kFloat || t->sizes() != k.sizes().slice(0, 3) || !t->is_contiguous())
          throw Bad{"8-bit caches need contiguous float32 scales [pages, heads, page_size]"};
        else if (t->device() != k.device()) throw Bad{"the cache must be on one device"};
      c.k_scale = static_cast<float*>(s[0]->data_ptr());
      c.v_scale = static_cast<float*>(s[1]->data_ptr());
    }
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&c), sizeof c);
  });
}

// append(cache, k, v, slots, q, q_out, table, pos, interleaved, stream) -> status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Cache c(a[0]);
    const at::Tensor &k = tensor(a[1], "k must be a tensor"), &v = tensor(a[2], "v must be a tensor");
    const at::Tensor *q = maybe(a[4], "q must be a tensor"), *qo = maybe(a[5], "q_out must be a tensor");
    const at::Tensor* tab = maybe(a[6], "table must be a tensor");
    if (k.dim() != 3 || k.size(0) > INT32_MAX) throw Bad{"k must be [T, heads, D]"};
    const int64_t T = k.size(0);
    const lcp_heads hk = heads_of(k, nullptr, T, c->D, at::kBFloat16, "k must be bfloat16 [T, heads, D]");
    const lcp_heads hv = heads_of(v, nullptr, T, c->D, at::kBFloat16, "v must be bfloat16 with k's tokens and channels");
    lcp_heads hq{};
    if (q) {
      if (!qo || !tab) throw Bad{"q needs an output and a table"};
      hq = heads_of(*q, qo, T, c->D, at::kBFloat16, "q must be bfloat16 with k's tokens and channels");
    }
    Table t;
    const int32_t* pos = nullptr;
    if (tab) {
      t = table_of(*tab);
      pos = index_of(tensor(a[7], "a table needs pos"), T, "pos must be contiguous int32 [T]");
    }
    const at::Tensor& at_slots = tensor(a[3], "slots must be a tensor");
    const int32_t* slots = index_of(at_slots, T, "slots must be contiguous int32 [T]");
    const int inter = flag(a[8]);
    const int gpu = on_gpu({&k, &v, q, qo, tab, tab ? &THPVariable_Unpack(a[7]) : nullptr, &at_slots}, c.gpu);
    void* s = stream_of(a[9], gpu);
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = lcp_kv_append(c.get(), q ? &hq : nullptr, &hk, &hv, (int)T, slots, t.p, t.max_pos, pos, t.rot, inter, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(code);
  });
}

// read(cache, slots, k_out, v_out, stream) -> (status, k_out, v_out); outputs
// that are None are made here, bfloat16
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const Cache c(a[0]);
    const at::Tensor& slots = tensor(a[1], "slots must be a tensor");
    if (slots.dim() != 1 || slots.size(0) > INT32_MAX) throw Bad{"slots must be contiguous int32 [T]"};
    const int64_t T = slots.size(0);
    const int64_t shape[3] = {T, c->heads, c->D};
    const at::Tensor* given[2] = {maybe(a[2], "k_out must be a tensor"), maybe(a[3], "v_out must be a tensor")};
    at::Tensor out[2];
    const at::ScalarType dt = given[0] ? given[0]->scalar_type() : given[1] ? given[1]->scalar_type() : at::kBFloat16;
    if (dt != at::kFloat && dt != at::kBFloat16) {
      PyErr_SetString(PyExc_TypeError, "unsupported dtype: float32 or bfloat16");
      return nullptr;
    }
    for (const at::Tensor* t : given)
      if (t && (t->sizes() != at::IntArrayRef(shape, 3) || t->scalar_type() != dt || !t->is_contiguous()))
        throw Bad{"k_out and v_out must be contiguous [T, heads, D] of one dtype"};
    const int32_t* index = index_of(slots, T, "slots must be contiguous int32 [T]");
    const int gpu = on_gpu({&slots, given[0], given[1]}, c.gpu);
    for (int i = 0; i < 2; ++i)
      out[i] = given[i] ? *given[i] : at::empty(at::IntArrayRef(shape, 3), slots.options().dtype(dt));
    void* s = stream_of(a[4], gpu);
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = lcp_kv_read(c.get(), index, (int)T, out[0].data_ptr(), out[1].data_ptr(), dtype_of(out[0]), s);
    Py_END_ALLOW_THREADS
    return Py_BuildValue("iNN", code, THPVariable_Wrap(out[0]), THPVariable_Wrap(out[1]));
  });
}

// attend(cache, q, pages, lens, max_len, out, lse, ws, scale, window, make, stream)
// -> (status, out, lse). make: what is None among out (bfloat16), lse and a needed
// ws is made here; else lse is not written and ws is passed as it is. max_len and
// scale may be None: what the pages can hold, D^-1/2.
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const Cache c(a[0]);
    const at::Tensor &q = tensor(a[1], "q must be a tensor"), &pages = tensor(a[2], "pages must be a tensor");
    const at::Tensor *out = maybe(a[5], "out must be a tensor"), *lse = maybe(a[6], "lse must be a tensor"),
                     *ws = maybe(a[7], "ws must be a tensor");
    if (q.dim() != 3 || q.scalar_type() != at::kBFloat16 || q.size(2) != c->D || q.stride(2) != 1 ||
        (q.size(1) > 1 && q.stride(1) != c->D) || q.size(0) > INT32_MAX || q.size(1) > INT32_MAX)
      throw Bad{"q must be bfloat16 [B, heads, D] with adjacent heads"};
    const int B = (int)q.size(0), hq = (int)q.size(1), D = (int)q.size(2);
    if (pages.dim() != 2 || pages.size(0) != B || pages.scalar_type() != at::kInt || !pages.is_contiguous() ||
        pages.size(1) > INT32_MAX)
      throw Bad{"pages must be contiguous int32 [B, max_pages]"};
    const int P = (int)pages.size(1);
    const at::ScalarType dt = out ? out->scalar_type() : at::kBFloat16;
    if (dt != at::kFloat && dt != at::kBFloat16) {
      PyErr_SetString(PyExc_TypeError, "unsupported dtype: float32 or bfloat16");
      return nullptr;
    }
    if (out && (out->sizes() != q.sizes() || !out->is_contiguous()))
      throw Bad{"out must be contiguous and have q's shape"};
    const int64_t rows[2] = {B, hq};
    if (lse && (lse->sizes() != at::IntArrayRef(rows, 2) || lse->scalar_type() != at::kFloat || !lse->is_contiguous()))
      throw Bad{"lse must be contiguous float32 [B, heads]"};
    if (ws && !ws->is_contiguous()) throw Bad{"ws must be contiguous"};
    const at::Tensor& lens = tensor(a[3], "lens must be a tensor");
    if (lens.scalar_type() != at::kInt || lens.dim() != 1 || lens.size(0) != B || !lens.is_contiguous())
      throw Bad{"lens must be contiguous int32 [B]"};
    long long most = a[4] == Py_None ? (long long)P * c->page_size : whole(a[4]);
    if (most > INT32_MAX) throw Bad{"max_len does not fit 32 bits"};
    const int max_len = most < 0 ? -1 : (int)most, window = small(a[9]);
    const double scale = a[8] == Py_None ? 1.0 / std::sqrt((double)D) : PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    const bool make = flag(a[10]);
    if (!make && !out) throw Bad{"out must be a tensor"};
    size_t need = 0;
    int code = lcp_attn_decode_workspace_bytes(c.get(), B, hq, max_len, window, &need);
    at::Tensor o, l, w;
    if (code == LCP_OK) {
      const int gpu = on_gpu({&q, &pages, &lens, out, lse, ws}, c.gpu);
      if (out) o = *out;
      else o = at::empty(q.sizes(), q.options());
      if (lse) l = *lse;
      else if (make) l = at::empty(at::IntArrayRef(rows, 2), q.options().dtype(at::kFloat));
      if (ws) w = *ws;
      else if (make && need) w = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
      const int64_t row = B > 1 ? q.stride(0) : (int64_t)hq * D;
      void* s = stream_of(a[11], gpu);
      Py_BEGIN_ALLOW_THREADS
      code = lcp_attn_decode(c.get(), q.data_ptr(), row, B, hq, static_cast<const int32_t*>(pages.data_ptr()), P,
                             static_cast<const int32_t*>(lens.data_ptr()), max_len, (float)scale, window, o.data_ptr(),
                             dt == at::kFloat ? LCP_F32 : LCP_BF16, l.defined() ? static_cast<float*>(l.data_ptr()) : nullptr,
                             w.defined() ? w.data_ptr() : nullptr, w.defined() ? w.nbytes() : 0, s);
      Py_END_ALLOW_THREADS
    }
    return Py_BuildValue("iNN", code, THPVariable_Wrap(o), THPVariable_Wrap(l));
  });
}

// ---- a decoder block's operators around its deployed products ----------------------

// The lcp_dtype of a tensor among the given ones.
lcp_dtype type_of(at::ScalarType t, const char* what, bool e4m3 = false) {
  if (t == at::kFloat) return LCP_F32;
  if (t == at::kBFloat16) return LCP_BF16;
  if (e4m3 && t == at::kFloat8_e4m3fn) return LCP_E4M3;
  PyErr_SetString(PyExc_TypeError, what);
  throw Bad{nullptr};
}
constexpr const char* kTwoTypes = "unsupported dtype: float32 or bfloat16";
constexpr const char* kThreeTypes = "unsupported dtype: float32, bfloat16 or float8_e4m3fn";

// A matrix [T, C] with contiguous rows.
void check_rows(const at::Tensor& t, int64_t T, int64_t C, const char* what) {
  if (t.dim() != 2 || t.size(0) != T || t.size(1) != C || (C > 1 && t.stride(1) != 1)) throw Bad{what};
}

// These calls are no part of autograd's graph: what they make of tensors that ask for a gradient has none, which
// the caller (of the Python function above this one) is told.
void warn_of_no_graph(std::initializer_list<const at::Tensor*> inputs, const char* what) {
  if (!c10::GradMode::is_enabled()) return;
  for (const at::Tensor* t : inputs)
    if (t && t->requires_grad()) {
      if (PyErr_WarnEx(PyExc_UserWarning, what, 2) < 0) throw Bad{nullptr};
      return;
    }
}

// rms_norm(x, weight, residual, perm, y, scale, sum, y_type, eps, make, stream) ->
// (status, y, scale, sum). y_type: an lcp_dtype, or -1 for x's; with make, what is
// None among y, scale (e4m3) and sum (with a residual) is made here.
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x must be a tensor"), &w = tensor(a[1], "weight must be a tensor");
    const at::Tensor *res = maybe(a[2], "residual must be a tensor"), *perm = maybe(a[3], "perm must be a tensor"),
                     *y = maybe(a[4], "out must be a tensor"), *scale = maybe(a[5], "scale must be a tensor"),
                     *sum = maybe(a[6], "sum_out must be a tensor");
    if (x.dim() != 2 || x.size(0) > INT32_MAX || x.size(1) > INT32_MAX) throw Bad{"x must be [T, C]"};
    const int64_t T = x.size(0), C = x.size(1);
    const at::ScalarType xt = x.scalar_type();
    lcp_norm f{};
    f.dt = type_of(xt, kTwoTypes);
    f.weight_dt = type_of(w.scalar_type(), kTwoTypes);
    check_rows(x, T, C, "x must be [T, C] with contiguous rows");
    if (w.dim() != 1 || w.size(0) != C || !w.is_contiguous()) throw Bad{"weight must be contiguous [C]"};
    for (const at::Tensor* t : {res, sum})
      if (t) {
        check_rows(*t, T, C, "residual and sum_out must have x's shape and contiguous rows");
        if (t->scalar_type() != xt) throw Bad{"residual and sum_out must have x's dtype"};
      }
    const int asked = small(a[7]);
    const bool make = flag(a[9]);
    if (asked < -1 || asked > LCP_E4M3) throw Bad{"no such dtype"};
    f.y_dt = y ? type_of(y->scalar_type(), kThreeTypes, true) : asked < 0 ? f.dt : (lcp_dtype)asked;
    if (y) {
      check_rows(*y, T, C, "out must have x's shape and contiguous rows");
      if (asked >= 0 && f.y_dt != asked) throw Bad{"out has another dtype"};
    } else if (!make) {
      throw Bad{"out must be a tensor"};
    }
    const bool e4m3 = f.y_dt == LCP_E4M3;
    if (scale && (!e4m3 || scale->scalar_type() != at::kFloat || scale->dim() != 1 || scale->size(0) != T ||
                  !scale->is_contiguous()))
      throw Bad{"scale must be contiguous float32 [T], and is of 8-bit outputs only"};
    if (e4m3 && !scale && !make) throw Bad{"an 8-bit output needs scale"};
    if (perm) {
      if (perm->scalar_type() != at::kInt || perm->dim() != 2 || !perm->is_contiguous() || perm->numel() != C)
        throw Bad{"perm must be contiguous int32 [C / B, B]"};
      f.perm = static_cast<const int32_t*>(perm->data_ptr());
      f.B = (int)perm->size(1);
    }
    f.eps = (float)PyFloat_AsDouble(a[8]);
    if (f.eps == -1.f && PyErr_Occurred()) return nullptr;
    const int gpu = on_gpu({&x, &w, res, perm, y, scale, sum});
    warn_of_no_graph({&x, &w, res},
                     "lcp_rms_norm is not part of autograd's graph: its outputs have no gradient (RMSNorm.backward and "
                     "lcp_rms_norm_bwd compute it); detach its inputs or call it under torch.no_grad()");
    at::Tensor o, sc, su;
    if (y) o = *y;
    else o = at::empty({T, C}, x.options().dtype(e4m3 ? at::kFloat8_e4m3fn : f.y_dt == LCP_F32 ? at::kFloat : at::kBFloat16));
    if (scale) sc = *scale;
    else if (e4m3) sc = at::empty({T}, x.options().dtype(at::kFloat));
    if (sum) su = *sum;
    else if (res && make) su = at::empty({T, C}, x.options());
    f.x = x.data_ptr();
    f.x_row = x.stride(0);
    f.weight = w.data_ptr();
    if (res) { f.residual = res->data_ptr(); f.residual_row = res->stride(0); }
    if (su.defined()) { f.sum = su.data_ptr(); f.sum_row = su.stride(0); }
    f.y = o.data_ptr();
    f.y_row = o.stride(0);
    if (sc.defined()) f.scale = static_cast<float*>(sc.data_ptr());
    f.T = (int)T;
    f.C = (int)C;
    void* s = stream_of(a[10], gpu);
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = lcp_rms_norm(&f, s);
    Py_END_ALLOW_THREADS
    return Py_BuildValue("iNNN", code, THPVariable_Wrap(o), THPVariable_Wrap(sc), THPVariable_Wrap(su));
  });
}

// rms_norm_bwd(h, weight, dy, dsum, dx, dweight, ws, eps, make, stream) -> (status, dx, dweight)
PyObject* rms_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor &h = tensor(a[0], "h must be a tensor"), &w = tensor(a[1], "weight must be a tensor"),
                     &dy = tensor(a[2], "dy must be a tensor");
    const at::Tensor *dsum = maybe(a[3], "dsum must be a tensor"), *dx = maybe(a[4], "dx must be a tensor"),
                     *dw = maybe(a[5], "dweight must be a tensor"), *ws = maybe(a[6], "ws must be a tensor");
    if (h.dim() != 2 || h.size(0) > INT32_MAX || h.size(1) > INT32_MAX) throw Bad{"h must be [T, C]"};
    const int64_t T = h.size(0), C = h.size(1);
    const lcp_dtype dt = type_of(h.scalar_type(), kTwoTypes), wt = type_of(w.scalar_type(), kTwoTypes);
    for (const at::Tensor* t : {&h, &dy, dsum, dx})
      if (t) {
        check_rows(*t, T, C, "h, dy, dsum and dx must be [T, C] with contiguous rows");
        if (t->scalar_type() != h.scalar_type()) throw Bad{"h, dy, dsum and dx must have one dtype"};
      }
    for (const at::Tensor* t : {&w, dw})
      if (t && (t->dim() != 1 || t->size(0) != C || !t->is_contiguous() || t->scalar_type() != w.scalar_type()))
        throw Bad{"weight and dweight must be contiguous [C] of one dtype"};
    if (ws && !ws->is_contiguous()) throw Bad{"ws must be contiguous"};
    const double eps = PyFloat_AsDouble(a[7]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    const bool make = flag(a[8]);
    if (!make && (!dx || !dw)) throw Bad{"dx and dweight must be tensors"};
    size_t need = 0;
    int code = lcp_rms_norm_bwd_workspace_bytes((int)T, (int)C, &need);
    at::Tensor x, g, b;
    if (code == LCP_OK) {
      const int gpu = on_gpu({&h, &w, &dy, dsum, dx, dw, ws});
      if (dx) x = *dx;
      else x = at::empty({T, C}, h.options());
      if (dw) g = *dw;
      else g = at::empty({C}, w.options());
      if (ws) b = *ws;
      else if (make) b = at::empty({(int64_t)need}, h.options().dtype(at::kByte));
      void* s = stream_of(a[9], gpu);
      Py_BEGIN_ALLOW_THREADS
      code = lcp_rms_norm_bwd(h.data_ptr(), h.stride(0), dy.data_ptr(), dy.stride(0), dsum ? dsum->data_ptr() : nullptr,
                              dsum ? dsum->stride(0) : 0, w.data_ptr(), dt, wt, (int)T, (int)C, (float)eps, x.data_ptr(),
                              x.stride(0), g.data_ptr(), b.defined() ? b.data_ptr() : nullptr,
                              b.defined() ? b.nbytes() : 0, s);
      Py_END_ALLOW_THREADS
    }
    return Py_BuildValue("iNN", code, THPVariable_Wrap(x), THPVariable_Wrap(g));
  });
}

// packed(vals, meta, wscale, cout, cin) -> bytes of an lcp_packed
PyObject* packed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const at::Tensor &vals = tensor(a[0], "vals must be a tensor"), &meta = tensor(a[1], "meta must be a tensor");
    const at::Tensor* ws = maybe(a[2], "scale must be a tensor");
    lcp_packed p{};
    p.cout = small(a[3]);
    p.cin = small(a[4]);
    p.dt = ws ? LCP_E4M3 : LCP_BF16;
    size_t vb = 0, mb = 0;
    const int code = ws ? lcp_sparse_pack_e4m3_bytes(p.cout, p.cin, &vb, &mb) : lcp_sparse_pack_bytes(p.cout, p.cin, &vb, &mb);
    if (code != LCP_OK) throw Bad{"a packed layer needs cout and cin that are positive multiples of 32"};
    if (!vals.is_contiguous() || !meta.is_contiguous() || vals.nbytes() != vb || meta.nbytes() != mb)
      throw Bad{"vals and meta must be contiguous and as large as lcp_sparse_pack_bytes says for their type"};
    if (ws && (ws->scalar_type() != at::kFloat || ws->dim() != 1 || ws->size(0) != p.cout || !ws->is_contiguous()))
      throw Bad{"scale must be contiguous float32 [cout]"};
    if (meta.device() != vals.device() || (ws && ws->device() != vals.device()))
      throw Bad{"a packed layer must be on one device"};
    p.vals = vals.data_ptr();
    p.meta = static_cast<const uint32_t*>(meta.data_ptr());
    p.wscale = ws ? static_cast<const float*>(ws->data_ptr()) : nullptr;
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&p), sizeof p);
  });
}

// linear(packed, x, x_scale, bias, gate, residual, y, ws, act, y_type, make, stream) ->
// (status, y). y_type: an lcp_dtype, or -1 for y's or bfloat16.
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const Held<lcp_packed> p(a[0], "packed must be an lcp_packed");
    const at::Tensor& x = tensor(a[1], "x must be a tensor");
    const at::Tensor *xs = maybe(a[2], "scale must be a tensor"), *bias = maybe(a[3], "bias must be a tensor"),
                     *gate = maybe(a[4], "gate must be a tensor"), *res = maybe(a[5], "residual must be a tensor"),
                     *y = maybe(a[6], "out must be a tensor"), *ws = maybe(a[7], "ws must be a tensor");
    if (x.dim() != 2 || x.size(0) > INT32_MAX) throw Bad{"x must be [T, cin]"};
    const int64_t T = x.size(0), cout = p->cout;
    const bool e4m3 = p->dt == LCP_E4M3;
    if (x.scalar_type() != (e4m3 ? at::kFloat8_e4m3fn : at::kBFloat16)) {
      PyErr_SetString(PyExc_TypeError, e4m3 ? "x must be float8_e4m3fn as the layer is" : "x must be bfloat16 as the layer is");
      return nullptr;
    }
    check_rows(x, T, p->cin, "x must be [T, cin] with contiguous rows");
    if (e4m3 != (xs != nullptr)) throw Bad{"scale belongs to 8-bit inputs, and they need it"};
    if (xs && (xs->scalar_type() != at::kFloat || xs->dim() != 1 || xs->size(0) != T || !xs->is_contiguous()))
      throw Bad{"scale must be contiguous float32 [T]"};
    if (bias && (bias->scalar_type() != at::kBFloat16 || bias->dim() != 1 || bias->size(0) != cout || !bias->is_contiguous()))
      throw Bad{"bias must be contiguous bfloat16 [cout]"};
    lcp_epilogue e{};
    e.act = small(a[8]);
    if (bias) e.bias = bias->data_ptr();
    if (gate) {
      if (gate->scalar_type() != at::kBFloat16) throw Bad{"gate must be bfloat16"};
      check_rows(*gate, T, cout, "gate must be [T, cout] with contiguous rows");
      e.gate = gate->data_ptr();
      e.gate_row = gate->stride(0);
    }
    if (res) {
      e.residual_dt = type_of(res->scalar_type(), kTwoTypes);
      check_rows(*res, T, cout, "residual must be [T, cout] with contiguous rows");
      e.residual = res->data_ptr();
      e.residual_row = res->stride(0);
    }
    const int asked = small(a[9]);
    const bool make = flag(a[10]);
    if (asked != -1 && asked != LCP_F32 && asked != LCP_BF16) throw Bad{"out must be float32 or bfloat16"};
    const lcp_dtype yt = y ? type_of(y->scalar_type(), kTwoTypes) : asked < 0 ? LCP_BF16 : (lcp_dtype)asked;
    if (y) {
      check_rows(*y, T, cout, "out must be [T, cout] with contiguous rows");
      if (asked >= 0 && yt != asked) throw Bad{"out has another dtype"};
    } else if (!make) {
      throw Bad{"out must be a tensor"};
    }
    if (ws && !ws->is_contiguous()) throw Bad{"ws must be contiguous"};
    size_t need = 0;
    int code = lcp_sparse_linear_workspace_bytes(p.get(), (int)T, &need);
    at::Tensor o, b;
    if (code == LCP_OK) {
      const int gpu = on_gpu({&x, xs, bias, gate, res, y, ws}, p.gpu);
      warn_of_no_graph({&x, xs, bias, gate, res},
                       "lcp_sparse_linear has no gradient and is not part of autograd's graph; detach its inputs or call "
                       "it under torch.no_grad()");
      if (y) o = *y;
      else o = at::empty({T, cout}, x.options().dtype(yt == LCP_F32 ? at::kFloat : at::kBFloat16));
      if (ws) b = *ws;
      else if (make && need) b = at::empty({(int64_t)need}, x.options().dtype(at::kByte));
      void* s = stream_of(a[11], gpu);
      Py_BEGIN_ALLOW_THREADS
      code = lcp_sparse_linear(p.get(), x.data_ptr(), x.stride(0), xs ? static_cast<const float*>(xs->data_ptr()) : nullptr,
                               (int)T, &e, o.data_ptr(), o.stride(0), yt, b.defined() ? b.data_ptr() : nullptr,
                               b.defined() ? b.nbytes() : 0, s);
      Py_END_ALLOW_THREADS
    }
    return Py_BuildValue("iN", code, THPVariable_Wrap(o));
  });
}

// use_streams(function)
PyObject* use_streams(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 1, [&]() -> PyObject* {
    Py_INCREF(a[0]);
    Py_XSETREF(handle_of, a[0]);
    Py_RETURN_NONE;
  });
}

PyMethodDef methods[] = {
    {"use_streams", (PyCFunction)(void*)use_streams, METH_FASTCALL, nullptr},
    {"rope", (PyCFunction)(void*)rope, METH_FASTCALL, nullptr},
    {"cache", (PyCFunction)(void*)cache, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void*)append, METH_FASTCALL, nullptr},
    {"read", (PyCFunction)(void*)read, METH_FASTCALL, nullptr},
    {"attend", (PyCFunction)(void*)attend, METH_FASTCALL, nullptr},
    {"rms_norm", (PyCFunction)(void*)rms_norm, METH_FASTCALL, nullptr},
    {"rms_norm_bwd", (PyCFunction)(void*)rms_norm_bwd, METH_FASTCALL, nullptr},
    {"packed", (PyCFunction)(void*)packed, METH_FASTCALL, nullptr},
    {"linear", (PyCFunction)(void*)linear, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__serve(void) { return PyModule_Create(&module); }
