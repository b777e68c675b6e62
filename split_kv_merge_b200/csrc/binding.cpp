// Python binding of the serving operators (rotary positions, cache append, block-scaled cache
// attention, packed prompt attention): argument checks, outputs and workspaces from torch's
// allocator, one call of the C ABI each.  Their smallest calls take the GPU a few microseconds, as long
// as the interpreter takes for the checks alone, so these run here on torch's own tensor objects.
// serving.py holds the functions' documented signatures and hands the arguments on in a fixed order.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <optional>
#include <string>

#include "../../include/splitkv.h"

namespace {

PyObject* g_skv_error = nullptr;  // SkvError(code, where)

struct Bad {
  std::string what;
};
struct Raised {};  // a Python error is set
[[noreturn]] void bad(std::string what) { throw Bad{std::move(what)}; }

std::string shape_of(const at::Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}

const at::Tensor* optional_tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
  const at::Tensor* t = optional_tensor(o, name);
  if (t == nullptr) bad(std::string(name) + " must be a tensor");
  return *t;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int32_t int32(PyObject* o) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) bad("an integer argument is out of range");
  return (int32_t)v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v;
}

int cuda_index(const at::Tensor& t) {
  if (!t.is_cuda()) bad("tensors must be on a CUDA device");
  return t.get_device();
}
void on_device(const at::Tensor& t, const char* name, int dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    bad(std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(dev));
}
// Address of a contiguous int32 vector of n entries (n < 0: any).
const int32_t* index(const at::Tensor& t, const char* name, int64_t n, int dev) {
  if (t.scalar_type() != at::kInt || t.dim() != 1 || (n >= 0 && t.size(0) != n) || !t.is_contiguous())
    bad(std::string(name) + " must be a contiguous int32 vector" + (n < 0 ? "" : " of " + std::to_string(n) + " entries"));
  on_device(t, name, dev);
  return static_cast<const int32_t*>(t.data_ptr());
}
const int32_t* optional_index(PyObject* o, const char* name, int64_t n, int dev) {
  const at::Tensor* t = optional_tensor(o, name);
  return t == nullptr ? nullptr : index(*t, name, n, dev);
}
// A [rows, heads, dim] tensor with contiguous heads: its head count, and (token, head) strides.
int32_t rows(const at::Tensor& t, const char* name, at::ScalarType dtype, int64_t n, int64_t dim, int dev,
             int64_t (&stride)[2]) {
  on_device(t, name, dev);
  if (t.dim() != 3 || t.scalar_type() != dtype || t.size(0) != n || t.size(2) != dim ||
      (t.stride(2) != 1 && t.numel() != 0))
    bad(std::string(name) + " must be " + c10::toString(dtype) + " [" + std::to_string(n) + ", heads, " +
        std::to_string(dim) + "] with contiguous heads, got " + c10::toString(t.scalar_type()) + " " + shape_of(t));
  if (t.size(1) > INT32_MAX || n > INT32_MAX) bad(std::string(name) + " is too large");
  stride[0] = t.stride(0);
  stride[1] = t.stride(1);
  return (int32_t)t.size(1);
}

// A tensor that a call has written: autograd refuses a backward pass that kept its old values.
void written(const at::Tensor* t) {
  if (t != nullptr && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// The tensors' device made current for a call (nothing to do when it is), and its stream.
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  explicit OnDevice(int dev) {
    if (c10::cuda::current_device() != dev) guard.set_index((c10::DeviceIndex)dev);
  }
};
skv_stream_t stream_of(int dev) {
  return reinterpret_cast<skv_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
}

// Frequencies of a rotation: a float64 buffer, or None.
class Frequencies {
 public:
  Frequencies(PyObject* o, int32_t dim) {
    if (o == Py_None || dim <= 0) return;
    if (PyObject_GetBuffer(o, &view_, PyBUF_C_CONTIGUOUS) != 0) throw Raised{};
    held_ = true;
    if (view_.itemsize != 8 || view_.len != (Py_ssize_t)(dim / 2) * 8) {
      PyBuffer_Release(&view_);
      bad("inv_freq must hold rope_dim / 2 = " + std::to_string(dim / 2) + " frequencies");
    }
  }
  ~Frequencies() {
    if (held_) PyBuffer_Release(&view_);
  }
  const double* get() const { return held_ ? static_cast<const double*>(view_.buf) : nullptr; }

 private:
  Py_buffer view_;
  bool held_ = false;
};

skv_rope rope_of(int32_t dim, PyObject* layout, PyObject* theta, const Frequencies& f, PyObject* mscale) {
  skv_rope r;
  r.dim = dim;
  r.layout = int32(layout);
  r.theta = real(theta);
  r.inv_freq_h = f.get();
  r.mscale = (float)real(mscale);
  return r;
}

template <typename Call>
void run(const char* where, Call call) {
  skv_status st;
  Py_BEGIN_ALLOW_THREADS st = call();
  Py_END_ALLOW_THREADS if (st == SKV_OK) return;
  PyObject* e = PyObject_CallFunction(g_skv_error, "is", (int)st, where);
  if (e != nullptr) {
    PyErr_SetObject(g_skv_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

// Python's side of an entry: argument count, C++ errors as Python's.
template <typename Body>
PyObject* entry(Py_ssize_t given, Py_ssize_t wanted, Body body) {
  try {
    if (given != wanted) bad("wrong number of arguments");
    return body();
  } catch (const Raised&) {
  } catch (const Bad& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (...) {  // torch's own errors under torch's own names
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

PyObject* none() { Py_RETURN_NONE; }
// `given` where the caller passed the output, else the new tensor (undefined: None)
PyObject* out(PyObject* given, const at::Tensor& made) {
  if (given != Py_None) return Py_NewRef(given);
  return made.defined() ? THPVariable_Wrap(made) : none();
}
PyObject* tuple(PyObject* a, PyObject* b, PyObject* c = nullptr) {
  PyObject* t = PyTuple_New(c == nullptr ? 2 : 3);
  if (t == nullptr || a == nullptr || b == nullptr) {
    Py_XDECREF(t);
    Py_XDECREF(a);
    Py_XDECREF(b);
    Py_XDECREF(c);
    return nullptr;
  }
  PyTuple_SET_ITEM(t, 0, a);
  PyTuple_SET_ITEM(t, 1, b);
  if (c != nullptr) PyTuple_SET_ITEM(t, 2, c);
  return t;
}

// (q, k, positions, rope_dim, theta, layout, inv_freq, mscale, inverse, q_out, k_out) -> (q_out, k_out)
PyObject* rope_apply(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 11, [&]() -> PyObject* {
    const at::Tensor *q = optional_tensor(a[0], "q"), *k = optional_tensor(a[1], "k");
    const at::Tensor *qo = optional_tensor(a[9], "q_out"), *ko = optional_tensor(a[10], "k_out");
    const at::Tensor* x = q != nullptr ? q : k;
    if (x == nullptr || x->dim() != 3) bad("q or k is needed, [tokens, heads, head_dim]");
    const at::ScalarType dtype = x->scalar_type();
    if (dtype != at::kBFloat16 && dtype != at::kFloat) bad("q and k must be bfloat16 or float32");
    if ((qo != nullptr && q == nullptr) || (ko != nullptr && k == nullptr)) bad("an output without its input");
    const int dev = cuda_index(*x);
    OnDevice on(dev);
    const int64_t tokens = x->size(0), dim = x->size(2);
    if (dim > INT32_MAX) bad("head_dim is too large");
    skv_rope_params p;
    std::memset(&p, 0, sizeof(p));
    at::Tensor made[2];
    const at::Tensor* in[2] = {q, k};
    const at::Tensor* given[2] = {qo, ko};
    const char* names[4] = {"q", "k", "q_out", "k_out"};
    int32_t heads[2] = {0, 0};
    int64_t in_st[2][2] = {{0, 0}, {0, 0}}, out_st[2][2] = {{0, 0}, {0, 0}};
    const void* src[2] = {nullptr, nullptr};
    void* dst[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i) {
      if (in[i] == nullptr) continue;
      heads[i] = rows(*in[i], names[i], dtype, tokens, dim, dev, in_st[i]);
      src[i] = in[i]->data_ptr();
      if (given[i] == nullptr) made[i] = at::empty(in[i]->sizes(), in[i]->options());
      const at::Tensor& o = given[i] != nullptr ? *given[i] : made[i];
      if (rows(o, names[2 + i], dtype, tokens, dim, dev, out_st[i]) != heads[i])
        bad(std::string(names[2 + i]) + " must have the shape of " + names[i]);
      dst[i] = o.data_ptr();
    }
    p.q = src[0];
    p.k = src[1];
    p.q_out = dst[0];
    p.k_out = dst[1];
    std::memcpy(p.q_stride, in_st[0], 16);
    std::memcpy(p.k_stride, in_st[1], 16);
    std::memcpy(p.q_out_stride, out_st[0], 16);
    std::memcpy(p.k_out_stride, out_st[1], 16);
    p.positions = index(tensor(a[2], "positions"), "positions", tokens, dev);
    p.num_tokens = (int32_t)tokens;
    p.num_q_heads = heads[0];
    p.num_k_heads = heads[1];
    p.head_dim = (int32_t)dim;
    p.dtype = dtype == at::kFloat ? SKV_F32 : SKV_BF16;
    p.inverse = truth(a[8]);
    const int32_t rope_dim = a[3] == Py_None ? (int32_t)dim : int32(a[3]);
    const Frequencies f(a[6], rope_dim);
    p.rope = rope_of(rope_dim, a[5], a[4], f, a[7]);
    const skv_stream_t s = stream_of(dev);
    run("skv_rope_apply", [&] { return skv_rope_apply(&p, s); });
    written(qo);
    written(ko);
    return tuple(out(a[9], made[0]), out(a[10], made[1]));
  });
}

int32_t cache_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return SKV_BF16;
    case at::kFloat8_e4m3fn:
    case at::kByte: return SKV_E4M3;
    case at::kChar: return SKV_I8;
    default: return -1;
  }
}

struct Caches {
  int32_t code, pages, page, hk, dim;
  void *k, *v;
  int64_t ks[3], vs[3];
};
Caches caches_of(const at::Tensor& k, const at::Tensor& v, int64_t dim, PyObject* num_pages, int dev) {
  Caches c;
  c.code = cache_code(k);
  if (c.code < 0 || v.scalar_type() != k.scalar_type())
    bad("caches must both be bfloat16, float8_e4m3fn or int8");
  if (k.dim() != 4 || v.sizes() != k.sizes()) bad("the caches must both be [num_pages, P, Hk, D]");
  on_device(k, "k_cache", dev);
  on_device(v, "v_cache", dev);
  if (k.size(3) != dim || k.stride(3) != 1 || v.stride(3) != 1)
    bad("the caches must be [num_pages, P, Hk, " + std::to_string(dim) + "] with contiguous heads");
  if (k.size(0) > INT32_MAX || k.size(1) > INT32_MAX || k.size(2) > INT32_MAX) bad("the caches are too large");
  c.pages = num_pages == Py_None ? (int32_t)k.size(0) : int32(num_pages);
  if (c.pages < 0 || c.pages > k.size(0)) bad("num_pages is more than the cache holds");
  c.page = (int32_t)k.size(1);
  c.hk = (int32_t)k.size(2);
  c.dim = (int32_t)dim;
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  for (int i = 0; i < 3; ++i) {
    c.ks[i] = k.stride(i);
    c.vs[i] = v.stride(i);
  }
  return c;
}

// Scale tensors [num_pages, blocks per page, Hk]: tokens that share a scale, and their strides.
int32_t scales_of(const at::Tensor* k, const at::Tensor* v, const Caches& c, int dev, int64_t (&ks)[3], int64_t (&vs)[3]) {
  if (k == nullptr || v == nullptr) bad("k_scale and v_scale come together");
  on_device(*k, "k_scale", dev);
  on_device(*v, "v_scale", dev);
  if (k->dim() != 3 || v->sizes() != k->sizes() || k->scalar_type() != at::kFloat || v->scalar_type() != at::kFloat ||
      k->size(0) < c.pages || k->size(2) != c.hk || k->size(1) < 1 || c.page % k->size(1) != 0)
    bad("k_scale and v_scale must be float32 [num_pages, blocks per page, " + std::to_string(c.hk) +
        "] with whole blocks of tokens");
  for (int i = 0; i < 3; ++i) {
    ks[i] = k->stride(i);
    vs[i] = v->stride(i);
  }
  return (int32_t)(c.page / k->size(1));
}

// (k, v, k_cache, v_cache, append_indptr, kv_indptr, kv_indices, kv_last_page_len, k_scale, v_scale, kv_scale, q, q_out,
//  positions, rope_dim, theta, layout, inv_freq, mscale, num_pages, status) -> q_out
PyObject* paged_kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 21, [&]() -> PyObject* {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    if (k.dim() != 3) bad("k and v are [rows, Hk, D]");
    const int dev = cuda_index(k);
    OnDevice on(dev);
    const int64_t num = k.size(0), dim = k.size(2);
    skv_append_params p;
    std::memset(&p, 0, sizeof(p));
    const int32_t hk = rows(k, "k", at::kBFloat16, num, dim, dev, p.k_row_stride);
    const int32_t hv = rows(v, "v", at::kBFloat16, num, dim, dev, p.v_row_stride);
    const at::Tensor &k_cache = tensor(a[2], "k_cache"), &v_cache = tensor(a[3], "v_cache");
    const Caches c = caches_of(k_cache, v_cache, dim, a[19], dev);
    if (hk != c.hk || hv != c.hk) bad("k, v and the caches must have the same heads");
    p.k = k.data_ptr();
    p.v = v.data_ptr();
    p.k_cache = c.k;
    p.v_cache = c.v;
    std::memcpy(p.k_stride, c.ks, 24);
    std::memcpy(p.v_stride, c.vs, 24);
    p.kv_dtype = c.code;
    p.kv_scale = (float)real(a[10]);
    const at::Tensor *kscale = optional_tensor(a[8], "k_scale"), *vscale = optional_tensor(a[9], "v_scale");
    if (kscale != nullptr || vscale != nullptr) {
      p.block_tokens = scales_of(kscale, vscale, c, dev, p.k_scale_stride, p.v_scale_stride);
      p.k_scale = static_cast<float*>(kscale->data_ptr());
      p.v_scale = static_cast<float*>(vscale->data_ptr());
    }
    const at::Tensor& ip = tensor(a[4], "append_indptr");
    const int64_t batch = ip.numel() - 1;
    if (batch < 0 || batch > INT32_MAX) bad("append_indptr must be a contiguous int32 vector");
    p.append_indptr = index(ip, "append_indptr", batch + 1, dev);
    p.kv_indptr = index(tensor(a[5], "kv_indptr"), "kv_indptr", batch + 1, dev);
    p.kv_indices = index(tensor(a[6], "kv_indices"), "kv_indices", -1, dev);
    p.kv_last_page_len = index(tensor(a[7], "kv_last_page_len"), "kv_last_page_len", batch, dev);
    // torch gives empty tensors no storage; no page id of a request without pages is read
    if (p.kv_indices == nullptr) p.kv_indices = p.kv_indptr;
    p.positions = optional_index(a[13], "positions", num, dev);
    p.batch = (int32_t)batch;
    p.num_rows = (int32_t)num;
    p.num_pages = c.pages;
    p.page_size = c.page;
    p.num_kv_heads = c.hk;
    p.head_dim = c.dim;
    const int32_t rope_dim = int32(a[14]);
    const Frequencies f(a[17], rope_dim);
    p.rope = rope_of(rope_dim, a[16], a[15], f, a[18]);
    const at::Tensor *q = optional_tensor(a[11], "q"), *qo = optional_tensor(a[12], "q_out");
    at::Tensor made;
    if (q != nullptr) {
      p.num_q_heads = rows(*q, "q", at::kBFloat16, num, dim, dev, p.q_stride);
      if (qo == nullptr) made = at::empty(q->sizes(), q->options());
      const at::Tensor& o = qo != nullptr ? *qo : made;
      if (rows(o, "q_out", at::kBFloat16, num, dim, dev, p.q_out_stride) != p.num_q_heads)
        bad("q_out must have the shape of q");
      p.q = q->data_ptr();
      p.q_out = o.data_ptr();
    } else if (qo != nullptr) {
      bad("q_out without q");
    }
    p.status = const_cast<int32_t*>(optional_index(a[20], "status", -1, dev));
    const skv_stream_t s = stream_of(dev);
    run("skv_paged_kv_append", [&] { return skv_paged_kv_append(&p, s); });
    written(&k_cache);
    written(&v_cache);
    written(kscale);
    written(vscale);
    written(qo);
    return out(a[12], made);
  });
}

// Outputs of an attention call: `given` or new ones, [total_q, Hq, D] of F32 / BF16 and [total_q, Hq].
struct Outputs {
  at::Tensor o, lse;  // made here
  void* o_ptr;
  float* lse_ptr;
  int32_t o_code;
};
Outputs outputs_of(const at::Tensor& q, PyObject* o_given, PyObject* lse_given, int32_t o_code, int dev) {
  Outputs r;
  const at::Tensor *o = optional_tensor(o_given, "o_out"), *lse = optional_tensor(lse_given, "lse_out");
  if (o == nullptr) {
    r.o = at::empty(q.sizes(), q.options().dtype(o_code == SKV_BF16 ? at::kBFloat16 : at::kFloat));
    o = &r.o;
  } else {
    on_device(*o, "o_out", dev);
    if (o->sizes() != q.sizes() || !o->is_contiguous()) bad("o_out must be contiguous " + shape_of(q));
    if (o->scalar_type() != at::kFloat && o->scalar_type() != at::kBFloat16) bad("outputs are float32 or bfloat16");
    o_code = o->scalar_type() == at::kFloat ? SKV_F32 : SKV_BF16;
  }
  if (lse == nullptr) {
    r.lse = at::empty({q.size(0), q.size(1)}, q.options().dtype(at::kFloat));
    lse = &r.lse;
  } else {
    on_device(*lse, "lse_out", dev);
    if (lse->dim() != 2 || lse->size(0) != q.size(0) || lse->size(1) != q.size(1) || !lse->is_contiguous() ||
        lse->scalar_type() != at::kFloat)
      bad("lse_out must be contiguous float32 [total_q, Hq]");
  }
  r.o_ptr = o->data_ptr();
  r.lse_ptr = static_cast<float*>(lse->data_ptr());
  r.o_code = o_code;
  return r;
}
// One buffer for the plan's split partials: o_part, then lse_part.
at::Tensor workspace_of(const at::Tensor& q, const skv_plan_info& info, float** o_part, float** lse_part) {
  *o_part = *lse_part = nullptr;
  if (info.num_partial_rows == 0) return at::Tensor();
  const int64_t heads = (int64_t)info.num_partial_rows * q.size(1);
  at::Tensor ws = at::empty({heads * (q.size(2) + 1)}, q.options().dtype(at::kFloat));
  *o_part = static_cast<float*>(ws.data_ptr());
  *lse_part = *o_part + heads * q.size(2);
  return ws;
}

// (q, k_cache, v_cache, k_scale, v_scale, kv_indptr, kv_indices, kv_last_page_len, plan, plan info's address, sm_scale,
//  o code, o_out, lse_out, num_pages, status) -> (o, lse, workspace)
PyObject* paged_attention_scaled(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 16, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    if (q.dim() != 3) bad("q is [total_q, Hq, D]");
    const int dev = cuda_index(q);
    OnDevice on(dev);
    if (q.scalar_type() != at::kBFloat16 || !q.is_contiguous()) bad("q must be contiguous bfloat16");
    if (q.size(0) > INT32_MAX || q.size(1) > INT32_MAX || q.size(2) > INT32_MAX) bad("q is too large");
    const Caches c = caches_of(tensor(a[1], "k_cache"), tensor(a[2], "v_cache"), q.size(2), a[14], dev);
    if (c.code == SKV_BF16) bad("caches must both be float8_e4m3fn or int8");
    skv_paged_scaled_params sp;
    std::memset(&sp, 0, sizeof(sp));
    const at::Tensor *ks = optional_tensor(a[3], "k_scale"), *vs = optional_tensor(a[4], "v_scale");
    sp.block_tokens = scales_of(ks, vs, c, dev, sp.k_scale_stride, sp.v_scale_stride);
    sp.k_scale = static_cast<const float*>(ks->data_ptr());
    sp.v_scale = static_cast<const float*>(vs->data_ptr());
    skv_paged_params& p = sp.base;
    const at::Tensor& ip = tensor(a[5], "kv_indptr");
    const int64_t batch = ip.numel() - 1;
    if (batch < 0 || batch > INT32_MAX) bad("kv_indptr must be a contiguous int32 vector");
    p.kv_indptr = index(ip, "kv_indptr", batch + 1, dev);
    p.kv_indices = index(tensor(a[6], "kv_indices"), "kv_indices", -1, dev);
    p.kv_last_page_len = index(tensor(a[7], "kv_last_page_len"), "kv_last_page_len", batch, dev);
    if (p.kv_indices == nullptr) p.kv_indices = p.kv_indptr;  // no page of any request
    if (p.kv_last_page_len == nullptr) p.kv_last_page_len = p.kv_indptr;
    const int32_t* plan = index(tensor(a[8], "plan"), "plan", -1, dev);
    const skv_plan_info* info = reinterpret_cast<const skv_plan_info*>((uintptr_t)integer(a[9]));
    p.q = q.data_ptr();
    p.k_cache = c.k;
    p.v_cache = c.v;
    std::memcpy(p.k_stride, c.ks, 24);
    std::memcpy(p.v_stride, c.vs, 24);
    p.batch = (int32_t)batch;
    p.total_q = (int32_t)q.size(0);
    p.num_pages = c.pages;
    p.page_size = c.page;
    p.num_qo_heads = (int32_t)q.size(1);
    p.num_kv_heads = c.hk;
    p.head_dim = c.dim;
    p.sm_scale = a[10] == Py_None ? (float)(1.0 / std::sqrt((double)c.dim)) : (float)real(a[10]);
    const Outputs r = outputs_of(q, a[12], a[13], int32(a[11]), dev);
    const at::Tensor ws = workspace_of(q, *info, &p.o_part, &p.lse_part);
    p.o = r.o_ptr;
    p.o_dtype = r.o_code;
    p.lse = r.lse_ptr;
    p.status = const_cast<int32_t*>(optional_index(a[15], "status", -1, dev));
    p.kv_dtype = c.code;
    p.kv_scale = 1.f;
    const skv_stream_t s = stream_of(dev);
    run("skv_paged_attn_scaled_fwd", [&] { return skv_paged_attn_scaled_fwd(&sp, plan, info, s); });
    written(optional_tensor(a[12], "o_out"));
    written(optional_tensor(a[13], "lse_out"));
    return tuple(out(a[12], r.o), out(a[13], r.lse), out(Py_None, ws));
  });
}

// (q, k, v, plan, plan info's address, sm_scale, o code, o_out, lse_out, status) -> (o, lse, workspace)
PyObject* prompt_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 10, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    if (q.dim() != 3 || k.dim() != 3) bad("q is [total_q, Hq, D], k and v are [total_kv, Hk, D]");
    const int dev = cuda_index(q);
    OnDevice on(dev);
    skv_prompt_params p;
    std::memset(&p, 0, sizeof(p));
    const int64_t dim = q.size(2);
    p.num_qo_heads = rows(q, "q", at::kBFloat16, q.size(0), dim, dev, p.q_stride);
    p.num_kv_heads = rows(k, "k", at::kBFloat16, k.size(0), dim, dev, p.k_stride);
    if (rows(v, "v", at::kBFloat16, k.size(0), dim, dev, p.v_stride) != p.num_kv_heads)
      bad("k and v must have the same heads");
    p.q = q.data_ptr();
    p.k = k.data_ptr();
    p.v = v.data_ptr();
    p.total_q = (int32_t)q.size(0);
    p.total_kv = (int32_t)k.size(0);
    p.head_dim = (int32_t)dim;
    p.sm_scale = a[5] == Py_None ? (float)(1.0 / std::sqrt((double)dim)) : (float)real(a[5]);
    const int32_t* plan = index(tensor(a[3], "plan"), "plan", -1, dev);
    const skv_plan_info* info = reinterpret_cast<const skv_plan_info*>((uintptr_t)integer(a[4]));
    const Outputs r = outputs_of(q, a[7], a[8], int32(a[6]), dev);
    const at::Tensor ws = workspace_of(q, *info, &p.o_part, &p.lse_part);
    p.o = r.o_ptr;
    p.o_dtype = r.o_code;
    p.lse = r.lse_ptr;
    p.status = const_cast<int32_t*>(optional_index(a[9], "status", -1, dev));
    const skv_stream_t s = stream_of(dev);
    run("skv_prompt_attn_fwd", [&] { return skv_prompt_attn_fwd(&p, plan, info, s); });
    written(optional_tensor(a[7], "o_out"));
    written(optional_tensor(a[8], "lse_out"));
    return tuple(out(a[7], r.o), out(a[8], r.lse), out(Py_None, ws));
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XSETREF(g_skv_error, Py_NewRef(cls));
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {
    {"set_error", set_error, METH_O, "The exception class raised for C status codes."},
    {"rope_apply", FAST(rope_apply), METH_FASTCALL, nullptr},
    {"paged_kv_append", FAST(paged_kv_append), METH_FASTCALL, nullptr},
    {"paged_attention_scaled", FAST(paged_attention_scaled), METH_FASTCALL, nullptr},
    {"prompt_attention", FAST(prompt_attention), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&module); }
