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

// The lcp_kv_cache in a bytes-like object, and the index of its GPU (-1: none, -2:
// the object does not know).
struct Cache {
  Py_buffer b{};
  int gpu = -2;
  explicit Cache(PyObject* o) {
    static PyObject* const name = PyUnicode_InternFromString("gpu");
    if (PyObject* g = PyObject_GetAttr(o, name)) {
      gpu = (int)PyLong_AsLong(g);
      Py_DECREF(g);
    }
    PyErr_Clear();
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Bad{nullptr};
    if (b.len != (Py_ssize_t)sizeof(lcp_kv_cache)) {
      PyBuffer_Release(&b);
      throw Bad{"cache must be an lcp_kv_cache"};
    }
  }
  Cache(const Cache&) = delete;
  ~Cache() { PyBuffer_Release(&b); }
  const lcp_kv_cache* operator->() const { return static_cast<const lcp_kv_cache*>(b.buf); }
  const lcp_kv_cache* get() const { return static_cast<const lcp_kv_cache*>(b.buf); }
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
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__serve(void) { return PyModule_Create(&module); }
