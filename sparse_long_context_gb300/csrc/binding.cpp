// Python binding of the calls whose host time counts (the norm/rotation, the
// 8-bit cache and the paged cache: a decode step makes them one after the other, each a
// few microseconds on the device).  It does what the ctypes binding does, reading
// tensors through the C++ API: checks device, type, shape and strides, and passes
// pointers and the current stream to the C ABI.  Every function returns the
// sls_status; a tensor that does not fit raises ValueError.
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>

#include "sls.h"

namespace {

struct Calls {
  decltype(&sls_qk_norm_rope) qk_norm_rope = nullptr;
  decltype(&sls_kv8_append) append = nullptr;
  decltype(&sls_kv8_decode_attend) attend = nullptr;
  decltype(&sls_kv8_evict) evict = nullptr;
  decltype(&sls_paged_append) paged_append = nullptr;
  decltype(&sls_paged_select_pages) paged_select = nullptr;
  decltype(&sls_paged_decode_attend) paged_attend = nullptr;
  decltype(&sls_paged_fork) paged_fork = nullptr;
  decltype(&sls_paged_compact) paged_compact = nullptr;
} calls;

[[noreturn]] void bad(const std::string& what) { throw std::invalid_argument(what); }

std::string text(at::IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << ")";
  return o.str();
}

// A ctypes structure's memory.
template <typename S>
class Struct {
 public:
  Struct(PyObject* o, const char* name) {
    if (PyObject_GetBuffer(o, &buf_, PyBUF_SIMPLE) != 0) {
      PyErr_Clear();
      bad(std::string(name) + " must be a descriptor structure");
    }
    if (buf_.len != (Py_ssize_t)sizeof(S)) {
      PyBuffer_Release(&buf_);
      bad(std::string(name) + " is not the structure this call takes");
    }
  }
  Struct(const Struct&) = delete;
  ~Struct() { PyBuffer_Release(&buf_); }
  const S* get() const { return static_cast<const S*>(buf_.buf); }
  const S* operator->() const { return get(); }

 private:
  Py_buffer buf_;
};

class Args {
 public:
  Args(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
    if (n != want) bad("wrong number of arguments");
  }
  PyObject* at(int i) const { return a_[i]; }
  bool none(int i) const { return a_[i] == Py_None; }
  int64_t integer(int i) const {
    const int64_t v = PyLong_AsLongLong(a_[i]);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      bad("an integer argument is out of range");
    }
    return v;
  }
  const at::Tensor& any(int i, const char* name) const {
    if (!THPVariable_Check(a_[i])) bad(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(a_[i]);
  }
  // A tensor of the current device (whose stream the call goes to) of this
  // type and shape; strided: only the last dimension must be contiguous.
  const at::Tensor& tensor(int i, const char* name, at::ScalarType dt, std::initializer_list<int64_t> shape,
                           bool strided = false) {
    const at::Tensor& t = any(i, name);
    if (!t.is_cuda() || t.get_device() != device()) bad(std::string(name) + " must be a CUDA tensor on the current device");
    if (t.scalar_type() != dt)
      bad(std::string(name) + " must be " + at::toString(dt) + ", got " + at::toString(t.scalar_type()));
    const at::IntArrayRef want(shape.begin(), shape.size());
    if (t.sizes() != want) bad(std::string(name) + " must have shape " + text(want) + ", got " + text(t.sizes()));
    if (strided ? t.numel() && t.stride(-1) != 1 : !t.is_contiguous())
      bad(std::string(name) + (strided ? " must have contiguous channels" : " must be contiguous"));
    return t;
  }
  template <typename T = void>
  T* data(int i, const char* name, at::ScalarType dt, std::initializer_list<int64_t> shape) {
    return none(i) ? nullptr : static_cast<T*>(tensor(i, name, dt, shape).data_ptr());
  }
  int device() {
    if (device_ < 0) device_ = c10::cuda::current_device();
    return device_;
  }

 private:
  PyObject* const* a_;
  int device_ = -1;
};

// Stride of a dimension in elements (of a single entry: none is ever taken).
int64_t step(const at::Tensor& t, int dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }

void* stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

template <typename F>
PyObject* guarded(F f) {
  try {
    if (!calls.evict) bad("the library has not been bound (bind)");
    return PyLong_FromLong(f());
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

constexpr auto I32 = at::kInt;
constexpr auto F32 = at::kFloat;
constexpr auto BF16 = at::kBFloat16;

// (rope, q, k, positions, q_weight, k_weight, q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 8);
    Struct<sls_rope_desc> r(a.at(0), "rope");
    const at::Tensor& pos = a.any(3, "positions");
    const int64_t N = pos.dim() == 1 ? pos.size(0) : -1, D = r->head_dim;
    if (N < 0 || N > INT32_MAX) bad("positions must have one dimension of at most 2^31 - 1 tokens");
    const int32_t* pp = a.data<int32_t>(3, "positions", I32, {N});
    const auto dt = r->dtype == SLS_DTYPE_F32 ? F32 : BF16;
    struct Side {
      const void *in = nullptr, *w = nullptr;
      void* out = nullptr;
      int64_t it = 0, ih = 0, ot = 0, oh = 0;
    };
    auto side = [&](int64_t heads, int in, int w, int out, const char* nin, const char* nw, const char* nout) {
      Side s;
      if (heads == 0) return s;
      const at::Tensor& x = a.tensor(in, nin, dt, {N, heads, D}, true);
      const at::Tensor& y = a.tensor(out, nout, dt, {N, heads, D}, true);
      s.in = x.data_ptr();
      s.out = y.data_ptr();
      s.w = a.data(w, nw, dt, {D});
      s.it = step(x, 0); s.ih = step(x, 1); s.ot = step(y, 0); s.oh = step(y, 1);
      return s;
    };
    const Side q = side(r->num_q_heads, 1, 4, 6, "q", "q_weight", "q_out");
    const Side k = side(r->num_kv_heads, 2, 5, 7, "k", "k_weight", "k_out");
    return calls.qk_norm_rope(r.get(), (int32_t)N, q.in, q.it, q.ih, k.in, k.it, k.ih, q.w, k.w, pp, q.out, q.ot, q.oh,
                              k.out, k.ot, k.oh, stream());
  });
}

// (desc, cache, k_new, v_new, ctx_len, new_len, kmin, kmax, mass, ctx_out, pos_out)
PyObject* kv8_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 11);
    Struct<sls_attn_desc> d(a.at(0), "desc");
    Struct<sls_kv8_cache> c(a.at(1), "cache");
    const int64_t B = d->batch, H = d->num_kv_heads, D = d->head_dim, Cap = d->capacity;
    const at::Tensor& first = a.any(2, "k_new");
    if (first.dim() != 4) bad("k_new must be [B, T, Hkv, D], got " + text(first.sizes()));
    const int64_t T = first.size(1);
    if (T > INT32_MAX) bad("k_new holds too many tokens");
    const at::Tensor& k = a.tensor(2, "k_new", BF16, {B, T, H, D}, true);
    const at::Tensor& v = a.tensor(3, "v_new", BF16, {B, T, H, D}, true);
    if (a.none(4)) bad("ctx_len must be a tensor");
    int32_t* ctx = a.data<int32_t>(4, "ctx_len", I32, {B});
    const int32_t* len = a.data<int32_t>(5, "new_len", I32, {B});
    if (a.none(6) != a.none(7)) bad("kmin and kmax: both or neither");
    const int64_t pages = d->page_size > 0 ? Cap / d->page_size : 0, blocks = c->block > 0 ? Cap / c->block : 0;
    void* lo = a.data(6, "kmin", BF16, {B, H, pages, D});
    void* hi = a.data(7, "kmax", BF16, {B, H, pages, D});
    float* mass = a.data<float>(8, "mass", F32, {B, H, blocks});
    int32_t* to = a.none(9) ? ctx : a.data<int32_t>(9, "ctx_out", I32, {B});
    int32_t* pos = a.data<int32_t>(10, "pos_out", I32, {B});
    return calls.append(d.get(), c.get(), k.data_ptr(), step(k, 0), step(k, 1), step(k, 2), v.data_ptr(), step(v, 0),
                        step(v, 1), step(v, 2), (int32_t)T, len, lo, hi, mass, ctx, to, pos, stream());
  });
}

// (desc, cache, q, ctx_len, page_idx, count, k_fixed, sink, mass_in, mass_out, out, lse, workspace)
PyObject* kv8_decode_attend(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 13);
    Struct<sls_attn_desc> d(a.at(0), "desc");
    Struct<sls_kv8_cache> c(a.at(1), "cache");
    const int64_t B = d->batch, Hq = d->num_q_heads, H = d->num_kv_heads, D = d->head_dim;
    const at::Tensor& q = a.tensor(2, "q", BF16, {B, Hq, D});
    if (a.none(3)) bad("ctx_len must be a tensor");
    const int32_t* ctx = a.data<int32_t>(3, "ctx_len", I32, {B});
    const int32_t *pages = nullptr, *count = nullptr;
    int64_t stride = 0, fixed = 0;
    if (!a.none(4)) {
      const at::Tensor& p = a.any(4, "page_idx");
      if (p.dim() != 2 || p.size(1) > INT32_MAX) bad("page_idx must be [B * Hkv, entries], got " + text(p.sizes()));
      // a list without columns has no memory, and no pointer to it means every page
      if (p.size(1) < 1) bad("page_idx must have at least one entry a row (count says how many hold)");
      stride = p.size(1);
      pages = a.data<int32_t>(4, "page_idx", I32, {B * H, stride});
      count = a.data<int32_t>(5, "count", I32, {B * H});
      fixed = a.none(6) ? stride : a.integer(6);
      if (fixed < INT32_MIN || fixed > INT32_MAX) bad("k_fixed is out of range");
    }
    const float* sink = a.data<float>(7, "sink", F32, {Hq});
    const int64_t blocks = c->block > 0 ? d->capacity / c->block : 0;
    const float* mi = a.data<float>(8, "mass_in", F32, {B, H, blocks});
    float* mo = a.data<float>(9, "mass_out", F32, {B, H, blocks});
    void* out = a.tensor(10, "out", BF16, {B, Hq, D}).data_ptr();
    float* lse = a.data<float>(11, "lse", F32, {B, Hq});
    const int64_t bytes = a.any(12, "workspace").numel();
    void* ws = a.data(12, "workspace", at::kByte, {bytes});
    return calls.attend(d.get(), c.get(), q.data_ptr(), pages, (int32_t)stride, count, (int32_t)fixed, ctx, sink, out,
                        lse, mi, mo, ws, (size_t)bytes, stream());
  });
}

// (desc, src, dst_capacity, dst, keep, n_sink_blocks, n_recent_blocks, mass, mass_out, kmin, kmax, kmin_out,
//  kmax_out, kept_idx, ctx_len, ctx_out)
PyObject* kv8_evict(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 16);
    Struct<sls_attn_desc> d(a.at(0), "desc");
    Struct<sls_kv8_cache> src(a.at(1), "cache");
    const int64_t B = d->batch, H = d->num_kv_heads, D = d->head_dim, Cap = d->capacity, dcap = a.integer(2);
    int64_t num[3];
    for (int i = 0; i < 3; ++i) {
      num[i] = a.integer(4 + i);
      if (num[i] < INT32_MIN || num[i] > INT32_MAX) bad("keep, n_sink_blocks or n_recent_blocks is out of range");
    }
    if (dcap < 0 || dcap > INT32_MAX) bad("dst capacity is out of range");
    const int64_t block = src->block > 0 ? src->block : 1, page = d->page_size > 0 ? d->page_size : 1;
    if (a.none(7) || a.none(13) || a.none(14) || a.none(15)) bad("mass, kept_idx, ctx_len and ctx_out must be tensors");
    const float* mass = a.data<float>(7, "mass", F32, {B, H, Cap / block});
    float* mass_out = a.data<float>(8, "mass_out", F32, {B, H, dcap / block});
    void* lo = a.data(9, "kmin", BF16, {B, H, Cap / page, D});
    void* hi = a.data(10, "kmax", BF16, {B, H, Cap / page, D});
    void* lo2 = a.data(11, "kmin_out", BF16, {B, H, dcap / page, D});
    void* hi2 = a.data(12, "kmax_out", BF16, {B, H, dcap / page, D});
    int32_t* kept = a.data<int32_t>(13, "kept_idx", I32, {B * H, num[0]});
    const int32_t* ctx = a.data<int32_t>(14, "ctx_len", I32, {B});
    int32_t* to = a.data<int32_t>(15, "ctx_out", I32, {B});
    auto call = [&](const sls_kv8_cache* dst) {
      return calls.evict(d.get(), src.get(), (int32_t)dcap, dst, (int32_t)num[0], (int32_t)num[1], (int32_t)num[2], mass,
                         mass_out, lo, hi, lo2, hi2, kept, ctx, to, stream());
    };
    if (a.none(3)) return call(nullptr);
    Struct<sls_kv8_cache> dst(a.at(3), "dst");
    return call(dst.get());
  });
}

at::ScalarType type_of(const sls_attn_desc* d) { return d->dtype == SLS_DTYPE_F32 ? F32 : BF16; }

// An int32 argument.
int32_t word(const Args& a, int i, const char* name) {
  const int64_t v = a.integer(i);
  if (v < INT32_MIN || v > INT32_MAX) bad(std::string(name) + " is out of range");
  return (int32_t)v;
}

// (desc, cache, k_new, v_new, new_len, pos_out)
PyObject* paged_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 6);
    Struct<sls_attn_desc> d(a.at(0), "desc");
    Struct<sls_paged_cache> c(a.at(1), "cache");
    const int64_t B = d->batch, H = d->num_kv_heads, D = d->head_dim;
    const at::Tensor& first = a.any(2, "k_new");
    if (first.dim() != 4) bad("k_new must be [B, T, Hkv, D], got " + text(first.sizes()));
    const int64_t T = first.size(1);
    if (T > INT32_MAX) bad("k_new holds too many tokens");
    const at::Tensor& k = a.tensor(2, "k_new", type_of(d.get()), {B, T, H, D}, true);
    const at::Tensor& v = a.tensor(3, "v_new", type_of(d.get()), {B, T, H, D}, true);
    const int32_t* len = a.data<int32_t>(4, "new_len", I32, {B});
    int32_t* pos = a.data<int32_t>(5, "pos_out", I32, {B});
    return calls.paged_append(d.get(), c.get(), k.data_ptr(), step(k, 0), step(k, 1), step(k, 2), v.data_ptr(), step(v, 0),
                              step(v, 1), step(v, 2), (int32_t)T, len, pos, stream());
  });
}

// (desc, cache, q, k, n_sink_pages, n_local_tokens, page_idx, workspace)
PyObject* paged_select_pages(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 8);
    Struct<sls_attn_desc> d(a.at(0), "desc");
    Struct<sls_paged_cache> c(a.at(1), "cache");
    const int64_t B = d->batch, Hq = d->num_q_heads, H = d->num_kv_heads, D = d->head_dim;
    const at::Tensor& q = a.tensor(2, "q", type_of(d.get()), {B, Hq, D});
    const int32_t k = word(a, 3, "k"), sinks = word(a, 4, "n_sink_pages"), local = word(a, 5, "n_local_tokens");
    int32_t* idx = static_cast<int32_t*>(a.tensor(6, "page_idx", I32, {B * H, (int64_t)k}).data_ptr());
    const int64_t bytes = a.any(7, "workspace").numel();
    void* ws = a.data(7, "workspace", at::kByte, {bytes});
    return calls.paged_select(d.get(), c.get(), q.data_ptr(), k, sinks, local, idx, ws, (size_t)bytes, stream());
  });
}

// (desc, cache, q, page_idx, count, k_fixed, sink, out, lse, workspace)
PyObject* paged_decode_attend(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 10);
    Struct<sls_attn_desc> d(a.at(0), "desc");
    Struct<sls_paged_cache> c(a.at(1), "cache");
    const int64_t B = d->batch, Hq = d->num_q_heads, H = d->num_kv_heads, D = d->head_dim;
    const auto dt = type_of(d.get());
    const at::Tensor& q = a.tensor(2, "q", dt, {B, Hq, D});
    const int32_t *pages = nullptr, *count = nullptr;
    int64_t stride = 0;
    int32_t fixed = 0;
    if (!a.none(3)) {
      const at::Tensor& p = a.any(3, "page_idx");
      if (p.dim() != 2 || p.size(1) > INT32_MAX) bad("page_idx must be [B * Hkv, entries], got " + text(p.sizes()));
      // a list without columns has no memory, and no pointer to it means every page
      if (p.size(1) < 1) bad("page_idx must have at least one entry a row (count says how many hold)");
      stride = p.size(1);
      pages = a.data<int32_t>(3, "page_idx", I32, {B * H, stride});
      count = a.data<int32_t>(4, "count", I32, {B * H});
      fixed = a.none(5) ? (int32_t)stride : word(a, 5, "k_fixed");
    } else if (!a.none(4) || !a.none(5)) {
      bad("count and k_fixed say how much of page_idx holds, and there is no page_idx");
    }
    const float* sink = a.data<float>(6, "sink", F32, {Hq});
    void* out = a.tensor(7, "out", dt, {B, Hq, D}).data_ptr();
    float* lse = a.data<float>(8, "lse", F32, {B, Hq});
    const int64_t bytes = a.any(9, "workspace").numel();
    void* ws = a.data(9, "workspace", at::kByte, {bytes});
    return calls.paged_attend(d.get(), c.get(), q.data_ptr(), pages, (int32_t)stride, count, fixed, sink, out, lse, ws,
                              (size_t)bytes, stream());
  });
}

// (desc, cache, parent, keep_len, done, workspace)
PyObject* paged_fork(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 6);
    Struct<sls_attn_desc> d(a.at(0), "desc");
    Struct<sls_paged_cache> c(a.at(1), "cache");
    const int64_t B = d->batch;
    const int32_t* parent = static_cast<const int32_t*>(a.tensor(2, "parent", I32, {B}).data_ptr());
    const int32_t* keep = a.data<int32_t>(3, "keep_len", I32, {B});
    int32_t* done = a.data<int32_t>(4, "done", I32, {1});
    const int64_t bytes = a.any(5, "workspace").numel();
    void* ws = a.data(5, "workspace", at::kByte, {bytes});
    return calls.paged_fork(d.get(), c.get(), parent, keep, done, ws, (size_t)bytes, stream());
  });
}

// (desc, cache, moved, workspace)
PyObject* paged_compact(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&] {
    Args a(args, n, 4);
    Struct<sls_attn_desc> d(a.at(0), "desc");
    Struct<sls_paged_cache> c(a.at(1), "cache");
    int32_t* moved = a.data<int32_t>(2, "moved", I32, {(int64_t)c->num_pages});
    const int64_t bytes = a.any(3, "workspace").numel();
    void* ws = a.data(3, "workspace", at::kByte, {bytes});
    return calls.paged_compact(d.get(), c.get(), moved, ws, (size_t)bytes, stream());
  });
}

// (path): looks the entry points up in the library the ctypes binding has loaded.
PyObject* bind(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* lib = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  if (!lib) {
    PyErr_SetString(PyExc_RuntimeError, dlerror());
    return nullptr;
  }
  Calls c;
  c.qk_norm_rope = reinterpret_cast<decltype(c.qk_norm_rope)>(dlsym(lib, "sls_qk_norm_rope"));
  c.append = reinterpret_cast<decltype(c.append)>(dlsym(lib, "sls_kv8_append"));
  c.attend = reinterpret_cast<decltype(c.attend)>(dlsym(lib, "sls_kv8_decode_attend"));
  c.evict = reinterpret_cast<decltype(c.evict)>(dlsym(lib, "sls_kv8_evict"));
  c.paged_append = reinterpret_cast<decltype(c.paged_append)>(dlsym(lib, "sls_paged_append"));
  c.paged_select = reinterpret_cast<decltype(c.paged_select)>(dlsym(lib, "sls_paged_select_pages"));
  c.paged_attend = reinterpret_cast<decltype(c.paged_attend)>(dlsym(lib, "sls_paged_decode_attend"));
  c.paged_fork = reinterpret_cast<decltype(c.paged_fork)>(dlsym(lib, "sls_paged_fork"));
  c.paged_compact = reinterpret_cast<decltype(c.paged_compact)>(dlsym(lib, "sls_paged_compact"));
  if (!c.qk_norm_rope || !c.append || !c.attend || !c.evict || !c.paged_append || !c.paged_select || !c.paged_attend ||
      !c.paged_fork || !c.paged_compact) {
    PyErr_SetString(PyExc_RuntimeError, "the library lacks an entry point of the 8-bit or the paged cache");
    return nullptr;
  }
  calls = c;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_O, "Looks the C entry points up in libsls.so."},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"kv8_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv8_append)), METH_FASTCALL, nullptr},
    {"kv8_decode_attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv8_decode_attend)), METH_FASTCALL,
     nullptr},
    {"kv8_evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv8_evict)), METH_FASTCALL, nullptr},
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_append)), METH_FASTCALL,
     nullptr},
    {"paged_select_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_select_pages)), METH_FASTCALL,
     nullptr},
    {"paged_decode_attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_decode_attend)), METH_FASTCALL,
     nullptr},
    {"paged_fork", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_fork)), METH_FASTCALL,
     nullptr},
    {"paged_compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_compact)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Tensor binding of the 8-bit and the paged cache's calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
