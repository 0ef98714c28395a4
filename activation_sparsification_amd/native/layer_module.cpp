// Python binding of the cache, attention and norm entry points: argument marshalling only.
//
// A CPython module, not ctypes: the calls between two layers of a decode step run for a few microseconds on the
// GPU, and a ctypes call with its checks takes 14 to 22 on the host, this one 3 to 5.  Tensors are unpacked, checked
// and passed to libspa.so's C entries; outputs and workspaces come from torch's allocator on the current stream.
#include <Python.h>
#include <structmember.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>
#include <initializer_list>
#include <optional>
#include <string>
#include <utility>

#include "spa.h"

namespace {

// Thrown after a Python error is set.
struct Raised {};

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Raised();
}
void need(bool ok, const char* what) {
  if (!ok) refuse(what);
}

PyObject* g_error = nullptr;      // SpaError, set by the package
void check(spa_status s, const char* where) {
  if (s == SPA_OK) return;
  PyObject* args = Py_BuildValue("(is)", (int)s, where);
  PyObject* e = args && g_error ? PyObject_Call(g_error, args, nullptr) : nullptr;
  Py_XDECREF(args);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_SetString(PyExc_RuntimeError, where);
  }
  throw Raised();
}

// ---------------------------------------------------------------------------
// arguments
// ---------------------------------------------------------------------------
// Positional and keyword arguments in the order of `names`; the first `required` must be given.
template <int N>
struct Args {
  PyObject* v[N] = {};
  Args(const char* fn, const char* const (&names)[N], int required, int positional, PyObject* const* args, Py_ssize_t n,
       PyObject* kwnames) {
    if (n > positional) {
      PyErr_Format(PyExc_TypeError, "%s() takes at most %d positional arguments (%zd given)", fn, positional, n);
      throw Raised();
    }
    for (Py_ssize_t i = 0; i < n; ++i) v[i] = args[i];
    const Py_ssize_t kw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t i = 0; i < kw; ++i) {
      const char* name = PyUnicode_AsUTF8(PyTuple_GET_ITEM(kwnames, i));
      if (!name) throw Raised();
      int at = 0;
      while (at < N && std::strcmp(name, names[at])) ++at;
      if (at == N || v[at]) {
        PyErr_Format(PyExc_TypeError, at == N ? "%s() got an unexpected keyword argument '%s'"
                                              : "%s() got multiple values for argument '%s'", fn, name);
        throw Raised();
      }
      v[at] = args[n + i];
    }
    for (int i = 0; i < required; ++i)
      if (!v[i]) {
        PyErr_Format(PyExc_TypeError, "%s() missing required argument: '%s'", fn, names[i]);
        throw Raised();
      }
    for (int i = required; i < N; ++i)
      if (v[i] == Py_None) v[i] = nullptr;
  }
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: expected a tensor, not %s", name, Py_TYPE(o)->tp_name);
    throw Raised();
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  // forward only: a graph must not end here unnoticed
  if (t.requires_grad() && at::GradMode::is_enabled()) {
    PyErr_Format(PyExc_ValueError, "%s: requires a gradient, and this call has no backward; detach it or call under "
                 "torch.no_grad()", name);
    throw Raised();
  }
  return t;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}
int32_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + ": out of range");
  return (int32_t)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v;
}
int32_t size32(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(std::string(name) + ": too large");
  return (int32_t)v;
}

int dtype_code(at::ScalarType t) {
  return t == at::kFloat ? SPA_F32 : t == at::kHalf ? SPA_F16 : t == at::kBFloat16 ? SPA_BF16 : -1;
}

// Refuses a tensor whose storage no longer holds it (resized, or given back): `elements` from its first to its last.
void held(const at::Tensor& x, int64_t elements, const char* name) {
  const c10::TensorImpl* t = x.unsafeGetTensorImpl();
  if (elements > 0 && t->unsafe_storage().nbytes() < (uint64_t)(t->storage_offset() + elements) * t->itemsize())
    refuse(std::string(name) + ": its storage is smaller than the tensor");
}

using Shape = std::initializer_list<int64_t>;
// A contiguous tensor of exactly this shape, type and device.
void given(const at::Tensor& x, Shape shape, at::ScalarType type, at::Device dev, const char* name) {
  if (x.scalar_type() == type && x.device() == dev && x.sizes() == c10::IntArrayRef(shape.begin(), shape.size()) &&
      x.is_contiguous()) {
    held(x, x.numel(), name);
    return;
  }
  std::string s = std::string(name) + ": expected a contiguous " + c10::toString(type) + " tensor of shape [";
  for (auto it = shape.begin(); it != shape.end(); ++it) s += (it == shape.begin() ? "" : ", ") + std::to_string(*it);
  refuse(s + "] on " + dev.str());
}

// [rows, heads, head_dim] with a dense last axis.  The stride of an axis of one element is never used, and torch
// leaves any number in it.
spa_heads heads(const at::Tensor& x, const char* name) {
  if (!x.is_cuda()) refuse(std::string(name) + ": expected a device tensor");
  if (x.dim() != 3) refuse(std::string(name) + ": expected [rows, heads, head_dim]");
  const int64_t* n = x.sizes().data();
  const int64_t* step = x.strides().data();
  if (n[2] > 1 && step[2] != 1) refuse(std::string(name) + ": expected a dense last axis");
  const spa_heads h{x.data_ptr(), n[0] > 1 ? step[0] : 0, n[1] > 1 ? step[1] : 0};
  held(x, x.numel() ? (n[0] - 1) * h.row_stride + (n[1] - 1) * h.head_stride + n[2] : 0, name);
  return h;
}

// Makes a device current while it lives, if it is not.  Kernels go to the current device whatever their stream: every call
// holds one around its allocations and the library's entry.
struct OnDevice {
  std::optional<c10::DeviceGuard> guard;
  explicit OnDevice(at::Device dev) {
    if (c10::impl::getDeviceGuardImpl(dev.type())->getDevice() != dev) guard.emplace(dev);
  }
};
// The current stream of a device.
void* stream_of(at::Device dev) { return c10::hip::getCurrentHIPStream(dev.index()).stream(); }

at::Tensor fresh(c10::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}
// The tensor an argument gives, checked, or a new one.
at::Tensor output(PyObject* o, Shape shape, at::ScalarType type, at::Device dev, const char* name) {
  if (!o) return fresh(c10::IntArrayRef(shape.begin(), shape.size()), type, dev);
  const at::Tensor& t = tensor(o, name);
  given(t, shape, type, dev, name);
  return t;
}
// Several one-dimensional outputs, given or new.  The new ones are parts of one allocation: a plan of four tensors takes the
// host 4.4 us so, 3.2 with all of them given; six allocations alone took 4.
template <int N>
void outputs(PyObject* const* given_ones, const int64_t (&sizes)[N], const char* const (&names)[N], at::ScalarType type,
             at::Device dev, at::Tensor (&out)[N]) {
  constexpr int64_t kApart = 64;      // elements: the parts begin on 64 bytes at the least
  int64_t total = 0;
  for (int i = 0; i < N; ++i) total += given_ones[i] ? 0 : (sizes[i] + kApart - 1) / kApart * kApart;
  const at::Tensor all = total ? fresh({total}, type, dev) : at::Tensor();
  int64_t at = 0;
  for (int i = 0; i < N; ++i) {
    if (given_ones[i] || !sizes[i]) {
      out[i] = output(given_ones[i], {sizes[i]}, type, dev, names[i]);
      continue;
    }
    auto part = c10::make_intrusive<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
    part->set_storage_offset(at);
    part->set_sizes_contiguous({sizes[i]});
    out[i] = at::Tensor(std::move(part));
    at += (sizes[i] + kApart - 1) / kApart * kApart;
  }
}
// Tells autograd that a tensor was written, as torch's own operations in place do: a backward that kept its old values is
// then an error.
void written(const at::Tensor& t) {
  if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
// `o` itself where it was given (callers compare identity), else a new Python tensor.
PyObject* back(PyObject* o, const at::Tensor& t) {
  if (o) {
    written(t);
    Py_INCREF(o);
    return o;
  }
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}

// Runs a binding body; any C++ exception becomes a Python one.
template <typename F>
PyObject* guarded(F body) {
  try {
    return body();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// ---------------------------------------------------------------------------
// KvCache
// ---------------------------------------------------------------------------
struct KvCache {
  PyObject_HEAD
  PyObject* part[4];      // k, v, k_scale, v_scale; None or NULL where there are none
};

// What a cache's tensors are now.  They are looked at for each call: a program may give them other memory.
struct Pages {
  spa_kv_cache c;         // dtype is filled in by cache_for
  at::ScalarType type;
  at::Device dev;
};
Pages pages_of(PyObject* const (&p)[4]) {
  need(p[0] && p[1], "KvCache: not initialised");
  const at::Tensor &k = tensor(p[0], "KvCache.k"), &v = tensor(p[1], "KvCache.v");
  need(k.is_cuda(), "KvCache: expected device tensors");
  need(k.dim() == 4 && k.is_contiguous(), "KvCache: k is [n_pages, n_heads, page_size, head_dim], contiguous");
  const at::ScalarType type = k.scalar_type();
  const int64_t n = k.sizes()[0], h = k.sizes()[1], s = k.sizes()[2], d = k.sizes()[3];
  held(k, k.numel(), "KvCache.k");
  given(v, {n, h, s, d}, type, k.device(), "KvCache.v");
  spa_kv_cache c{};
  c.format = type == at::kFloat8_e4m3fn ? SPA_KV_FP8 : type == at::kChar ? SPA_KV_INT8
             : type == at::kByte ? SPA_KV_MXFP4 : SPA_KV_NATIVE;
  const bool mx = c.format == SPA_KV_MXFP4;      // two elements to a byte
  const bool scales[2] = {p[2] && p[2] != Py_None, p[3] && p[3] != Py_None};
  if (c.format != SPA_KV_NATIVE) {
    need(scales[0] && scales[1], "KvCache: 8-bit and 4-bit pages need k_scale and v_scale");
    const at::Tensor &ks = tensor(p[2], "KvCache.k_scale"), &vs = tensor(p[3], "KvCache.v_scale");
    for (const auto& [x, name] : {std::pair(&ks, "KvCache.k_scale"), std::pair(&vs, "KvCache.v_scale")}) {
      if (mx) given(*x, {n, h, (d + 15) / 16, s}, at::kByte, k.device(), name);      // d bytes: 2 d elements, 32 to a scale
      else given(*x, {n, h, s}, at::kFloat, k.device(), name);
    }
    c.k_scale = ks.data_ptr();
    c.v_scale = vs.data_ptr();
  } else {
    need(dtype_code(type) >= 0, "KvCache: pages are float16, bfloat16, float8_e4m3fn, int8 or uint8 (two 4-bit codes)");
    need(!scales[0] && !scales[1], "KvCache: scales belong to 8-bit and 4-bit pages");
  }
  c.n_pages = size32(n, "n_pages"); c.n_heads = size32(h, "n_heads");
  c.page_size = size32(s, "page_size"); c.head_dim = size32(mx ? 2 * d : d, "head_dim");
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  return Pages{c, type, k.device()};
}

int cache_init(KvCache* self, PyObject* args, PyObject* kw) {
  static const char* names[] = {"k", "v", "k_scale", "v_scale", nullptr};
  PyObject* p[4] = {nullptr, nullptr, nullptr, nullptr};
  if (!PyArg_ParseTupleAndKeywords(args, kw, "OO|OO", const_cast<char**>(names), &p[0], &p[1], &p[2], &p[3])) return -1;
  PyObject* ok = guarded([&]() -> PyObject* {
    pages_of(p);
    for (int i = 0; i < 4; ++i) {
      PyObject* now = p[i] ? p[i] : Py_None;
      Py_INCREF(now);
      Py_XSETREF(self->part[i], now);
    }
    Py_RETURN_NONE;
  });
  Py_XDECREF(ok);
  return ok ? 0 : -1;
}
int cache_traverse(KvCache* self, visitproc visit, void* arg) {
  for (PyObject* p : self->part) Py_VISIT(p);
  return 0;
}
int cache_clear(KvCache* self) {
  for (PyObject*& p : self->part) Py_CLEAR(p);
  return 0;
}
void cache_dealloc(KvCache* self) {
  PyObject_GC_UnTrack(self);
  cache_clear(self);
  Py_TYPE(self)->tp_free(reinterpret_cast<PyObject*>(self));
}

PyMemberDef cache_members[] = {
    {"k", T_OBJECT, offsetof(KvCache, part), READONLY, "keys, or their codes"},
    {"v", T_OBJECT, offsetof(KvCache, part) + sizeof(PyObject*), READONLY, "values, or their codes"},
    {"k_scale", T_OBJECT, offsetof(KvCache, part) + 2 * sizeof(PyObject*), READONLY, "scales of 8-bit or 4-bit keys, or None"},
    {"v_scale", T_OBJECT, offsetof(KvCache, part) + 3 * sizeof(PyObject*), READONLY, "scales of 8-bit or 4-bit values, or None"},
    {nullptr, 0, 0, 0, nullptr}};

template <int32_t spa_kv_cache::*SIZE>
PyObject* cache_size(PyObject* self, void*) {
  return guarded([&]() -> PyObject* { return PyLong_FromLong(pages_of(reinterpret_cast<KvCache*>(self)->part).c.*SIZE); });
}
PyGetSetDef cache_sizes[] = {
    {"n_pages", cache_size<&spa_kv_cache::n_pages>, nullptr, nullptr, nullptr},
    {"page_size", cache_size<&spa_kv_cache::page_size>, nullptr, nullptr, nullptr},
    {"n_heads", cache_size<&spa_kv_cache::n_heads>, nullptr, nullptr, nullptr},
    {"head_dim", cache_size<&spa_kv_cache::head_dim>, nullptr, nullptr, nullptr},
    {nullptr, nullptr, nullptr, nullptr, nullptr}};

PyTypeObject g_cache_type = {PyVarObject_HEAD_INIT(nullptr, 0)};

// The C descriptor for vectors of `type` going in or out.
spa_kv_cache cache_for(const Pages& kv, at::ScalarType type) {
  need(dtype_code(type) >= 0 && (kv.c.format != SPA_KV_NATIVE || kv.type == type),
       "KvCache: the vectors' type is not the pages'");
  spa_kv_cache c = kv.c;
  c.dtype = dtype_code(type);
  return c;
}
Pages cache(PyObject* o) {
  if (!PyObject_TypeCheck(o, &g_cache_type)) {
    PyErr_Format(PyExc_TypeError, "cache: expected a KvCache, not %s", Py_TYPE(o)->tp_name);
    throw Raised();
  }
  return pages_of(reinterpret_cast<const KvCache*>(o)->part);
}

// ---------------------------------------------------------------------------
// calls
// ---------------------------------------------------------------------------
PyDoc_STRVAR(kv_write_doc,
             "kv_write($module, /, k, v, slots, cache)\n--\n\n"
             "Store the rows of k and v [t, n_heads, head_dim] at slots [t] int32 of a KvCache.\n\n"
             "Slot s is position s % page_size of page s // page_size; a slot outside the cache (-1) skips its row.");
PyObject* py_kv_write(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"k", "v", "slots", "cache"};
    Args<4> a("kv_write", names, 4, 4, args, n, kw);
    const at::Tensor &k = tensor(a.v[0], "k"), &v = tensor(a.v[1], "v"), &slots = tensor(a.v[2], "slots");
    const Pages kv = cache(a.v[3]);
    const spa_heads kh = heads(k, "k"), vh = heads(v, "v");
    const OnDevice on(kv.dev);
    need(k.device() == kv.dev && v.device() == kv.dev, "kv_write: tensors on several devices");
    need(k.sizes() == v.sizes() && k.scalar_type() == v.scalar_type(), "kv_write: k and v differ in shape or type");
    need(k.size(1) == kv.c.n_heads && k.size(2) == kv.c.head_dim, "kv_write: the cache has other heads");
    given(slots, {k.size(0)}, at::kInt, kv.dev, "slots");
    const spa_kv_cache c = cache_for(kv, k.scalar_type());
    check(spa_kv_write(&kh, &vh, size32(k.size(0), "k"), static_cast<const int32_t*>(slots.data_ptr()), &c,
                       stream_of(kv.dev)), "spa_kv_write");
    for (PyObject* part : reinterpret_cast<const KvCache*>(a.v[3])->part)
      if (part && part != Py_None) written(THPVariable_Unpack(part));
    Py_RETURN_NONE;
  });
}

PyDoc_STRVAR(kv_plan_doc,
             "kv_plan($module, /, lens, new, page_table, page_size, free_pages, free_count, t, *, done=None, slots=None,"
             " positions=None, cu_q=None, cu_k=None, lens_out=None, count_out=None)\n--\n\n"
             "Page tables, slots and offsets of a step from request lengths, all int32 on the device.\n\n"
             "lens and new [n_seqs]: cached positions and new tokens of each sequence; done [n_seqs]: sequences that are over\n"
             "give their pages back first and begin anew.  page_table [n_seqs, max_pages] receives pages from the stack\n"
             "free_pages [n_pages], of which free_count[0] are free (new_page_pool makes both).  Returns (slots [t],\n"
             "positions [t], cu_q [n_seqs + 1], cu_k [n_seqs + 1], lens [n_seqs], count [2]): the rows' slots (-1 without a\n"
             "page and past the last token) and positions, running sums of the new tokens and of the new lengths, the new\n"
             "lengths, and the pages free now and lacking.  lens_out may be lens and count_out may be free_count.");
PyObject* py_kv_plan(PyObject*, PyObject* const* args, Py_ssize_t n_args, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"lens", "new", "page_table", "page_size", "free_pages", "free_count", "t", "done",
                                        "slots", "positions", "cu_q", "cu_k", "lens_out", "count_out"};
    Args<14> a("kv_plan", names, 7, 7, args, n_args, kw);
    const at::Tensor &lens = tensor(a.v[0], "lens"), &fresh_tokens = tensor(a.v[1], "new"), &table = tensor(a.v[2], "page_table");
    const at::Tensor &stack = tensor(a.v[4], "free_pages"), &count = tensor(a.v[5], "free_count");
    const at::Device dev = lens.device();
    need(lens.is_cuda() && lens.dim() == 1, "lens: expected a device tensor [n_seqs]");
    const OnDevice on(dev);
    const int32_t n = size32(lens.size(0), "lens"), page_size = integer(a.v[3], "page_size"), t = integer(a.v[6], "t");
    need(t >= 0, "t: expected 0 or more");
    given(lens, {n}, at::kInt, dev, "lens");
    given(fresh_tokens, {n}, at::kInt, dev, "new");
    need(table.dim() == 2, "page_table: expected [n_seqs, max_pages]");
    given(table, {n, table.size(1)}, at::kInt, dev, "page_table");
    need(stack.dim() == 1, "free_pages: expected [n_pages]");
    given(stack, {stack.size(0)}, at::kInt, dev, "free_pages");
    given(count, {2}, at::kInt, dev, "free_count");
    const int32_t* done = nullptr;
    if (a.v[7]) {
      const at::Tensor& d = tensor(a.v[7], "done");
      given(d, {n}, at::kInt, dev, "done");
      done = static_cast<const int32_t*>(d.data_ptr());
    }
    static const char* const out_names[6] = {"slots", "positions", "cu_q", "cu_k", "lens_out", "count_out"};
    const int64_t sizes[6] = {t, t, (int64_t)n + 1, (int64_t)n + 1, n, 2};
    at::Tensor out[6];
    int32_t* to[6];
    outputs(&a.v[8], sizes, out_names, at::kInt, dev, out);
    for (int i = 0; i < 6; ++i) to[i] = static_cast<int32_t*>(out[i].data_ptr());
    const spa_page_pool pool{static_cast<int32_t*>(stack.data_ptr()), static_cast<const int32_t*>(count.data_ptr()), to[5],
                             size32(stack.size(0), "free_pages")};
    check(spa_kv_plan(static_cast<const int32_t*>(lens.data_ptr()), static_cast<const int32_t*>(fresh_tokens.data_ptr()), done, n,
                      static_cast<int32_t*>(table.data_ptr()), size32(table.size(1), "page_table"), page_size, &pool, t, to[0],
                      to[1], to[2], to[3], to[4], stream_of(dev)),
          "spa_kv_plan");
    written(table);
    written(stack);
    PyObject* r = PyTuple_New(6);
    if (!r) return nullptr;
    for (int i = 0; i < 6; ++i) {
      PyObject* o = back(a.v[8 + i], out[i]);
      if (!o) {
        Py_DECREF(r);
        return nullptr;
      }
      PyTuple_SET_ITEM(r, i, o);
    }
    return r;
  });
}

// A page table of n sequences; n < 0 takes it from the table.
int32_t table_width(const at::Tensor& t, int64_t n, at::Device dev) {
  need(t.dim() == 2, "page_table: expected [n_seqs, max_pages]");
  given(t, {n < 0 ? t.size(0) : n, t.size(1)}, at::kInt, dev, "page_table");
  return size32(t.size(1), "page_table");
}

PyDoc_STRVAR(kv_read_doc,
             "kv_read($module, /, cache, page_table, cu_seqlens, total, k_out=None, v_out=None, dtype=None)\n--\n\n"
             "The first cu_seqlens[s+1] - cu_seqlens[s] positions of each sequence as packed rows (k, v), each\n"
             "[total, n_heads, head_dim].\n\n"
             "page_table [n_seqs, max_pages] and cu_seqlens [n_seqs + 1] are int32.  dtype is needed for 8-bit and 4-bit\n"
             "pages when no outputs are given.  Positions on absent pages read as zeros.");
PyObject* py_kv_read(PyObject*, PyObject* const* args, Py_ssize_t n_args, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"cache", "page_table", "cu_seqlens", "total", "k_out", "v_out", "dtype"};
    Args<7> a("kv_read", names, 4, 7, args, n_args, kw);
    const Pages kv = cache(a.v[0]);
    const at::Tensor &table = tensor(a.v[1], "page_table"), &cu = tensor(a.v[2], "cu_seqlens");
    const int32_t total = integer(a.v[3], "total");
    need(total >= 0, "total: expected 0 or more");
    const OnDevice on(kv.dev);
    const int32_t max_pages = table_width(table, -1, kv.dev);
    const int32_t n = size32(table.size(0), "page_table");
    given(cu, {(int64_t)n + 1}, at::kInt, kv.dev, "cu_seqlens");
    at::ScalarType type = kv.type;
    if (a.v[6]) {
      if (!THPDtype_Check(a.v[6])) {
        PyErr_SetString(PyExc_TypeError, "dtype: expected a torch.dtype");
        throw Raised();
      }
      type = reinterpret_cast<THPDtype*>(a.v[6])->scalar_type;
    } else if (a.v[4] || a.v[5]) {
      type = tensor(a.v[4] ? a.v[4] : a.v[5], "k_out").scalar_type();
    } else {
      need(kv.c.format == SPA_KV_NATIVE, "kv_read: 8-bit and 4-bit pages need dtype or outputs");
    }
    const spa_kv_cache c = cache_for(kv, type);
    const at::Tensor k = output(a.v[4], {total, c.n_heads, c.head_dim}, type, kv.dev, "k_out");
    const at::Tensor v = output(a.v[5], {total, c.n_heads, c.head_dim}, type, kv.dev, "v_out");
    check(spa_kv_read(&c, static_cast<const int32_t*>(table.data_ptr()), n, max_pages,
                      static_cast<const int32_t*>(cu.data_ptr()), total, k.data_ptr(), v.data_ptr(), stream_of(kv.dev)),
          "spa_kv_read");
    return pair(back(a.v[4], k), back(a.v[5], v));
  });
}

float scale_of(PyObject* o, int64_t d) { return (float)(o ? number(o) : 1.0 / std::sqrt((double)(d > 0 ? d : 1))); }

// A workspace argument, checked for its device, or a new one of the size needed (undefined for 0 bytes).
at::Tensor workspace(PyObject* o, size_t bytes, at::Device dev) {
  if (o) {
    const at::Tensor& t = tensor(o, "ws");
    need(t.device() == dev && t.is_contiguous() && t.scalar_type() == at::kByte, "ws: expected a contiguous uint8 tensor");
    held(t, t.numel(), "ws");
    return t;
  }
  return bytes ? fresh({(int64_t)bytes}, at::kByte, dev) : at::Tensor();
}

PyDoc_STRVAR(attention_decode_doc,
             "attention_decode($module, /, q, cache, page_table, seq_lens, scale=None, want_lse=False, out=None, ws=None)\n"
             "--\n\n"
             "Attention of one new token per sequence, q [n_seqs, n_q_heads, head_dim], over its cached positions.\n\n"
             "page_table [n_seqs, max_pages] and seq_lens [n_seqs] are int32; scale defaults to head_dim ** -0.5.\n"
             "Returns (out [n_seqs, n_q_heads, head_dim], lse [n_seqs, n_q_heads] float32 or None).");
PyObject* py_attention_decode(PyObject*, PyObject* const* args, Py_ssize_t n_args, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"q", "cache", "page_table", "seq_lens", "scale", "want_lse", "out", "ws"};
    Args<8> a("attention_decode", names, 4, 8, args, n_args, kw);
    const at::Tensor& q = tensor(a.v[0], "q");
    const Pages kv = cache(a.v[1]);
    const at::Tensor &table = tensor(a.v[2], "page_table"), &lens = tensor(a.v[3], "seq_lens");
    const spa_heads qh = heads(q, "q");
    const at::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    const OnDevice on(dev);
    need(kv.dev == dev, "attention_decode: tensors on several devices");
    need(q.size(2) == kv.c.head_dim, "attention_decode: the cache has another head_dim");
    const int32_t n = size32(q.size(0), "q"), hq = size32(q.size(1), "q"), d = kv.c.head_dim;
    const int32_t max_pages = table_width(table, n, dev);
    given(lens, {n}, at::kInt, dev, "seq_lens");
    const spa_kv_cache c = cache_for(kv, type);
    const at::Tensor out = output(a.v[6], {n, hq, d}, type, dev, "out");
    at::Tensor lse;
    if (a.v[5] && truth(a.v[5])) lse = fresh({n, hq}, at::kFloat, dev);
    const at::Tensor ws = workspace(a.v[7], a.v[7] ? 0 : spa_attention_decode_workspace_bytes(n, hq, c.n_heads, d), dev);
    check(attention_decode(&qh, n, hq, &c, static_cast<const int32_t*>(table.data_ptr()), max_pages,
                           static_cast<const int32_t*>(lens.data_ptr()), scale_of(a.v[4], d), out.data_ptr(),
                           lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr,
                           ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (size_t)ws.numel() : 0, stream_of(dev)),
          "attention_decode");
    return pair(back(a.v[6], out), back(nullptr, lse));
  });
}

PyDoc_STRVAR(attention_prefill_doc,
             "attention_prefill($module, /, q, k, v, cu_q, cu_k=None, causal=True, scale=None, want_lse=False, out=None,"
             " ws=None)\n--\n\n"
             "Attention over packed prompts: q [tq, n_q_heads, head_dim], k and v [tk, n_kv_heads, head_dim].\n\n"
             "cu_q and cu_k [n_seqs + 1] int32 are the sequences' first rows and the end (cu_k defaults to cu_q); with\n"
             "causal, query i of a sequence sees the keys j <= i + lk - lq.  Returns (out [tq, n_q_heads, head_dim],\n"
             "lse [tq, n_q_heads] float32 or None).");
PyObject* py_attention_prefill(PyObject*, PyObject* const* args, Py_ssize_t n_args, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"q", "k", "v", "cu_q", "cu_k", "causal", "scale", "want_lse", "out", "ws"};
    Args<10> a("attention_prefill", names, 4, 10, args, n_args, kw);
    const at::Tensor &q = tensor(a.v[0], "q"), &k = tensor(a.v[1], "k"), &v = tensor(a.v[2], "v");
    const at::Tensor &cu_q = tensor(a.v[3], "cu_q"), &cu_k = a.v[4] ? tensor(a.v[4], "cu_k") : cu_q;
    const spa_heads qh = heads(q, "q"), kh = heads(k, "k"), vh = heads(v, "v");
    const at::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    const OnDevice on(dev);
    need(k.sizes() == v.sizes() && k.size(2) == q.size(2), "attention_prefill: k and v are [tk, n_kv_heads, head_dim]");
    need(dtype_code(type) >= 0 && k.scalar_type() == type && v.scalar_type() == type,
         "attention_prefill: q, k and v differ in type");
    need(k.device() == dev && v.device() == dev, "attention_prefill: tensors on several devices");
    need(cu_q.dim() == 1 && cu_q.size(0) >= 1, "cu_q: expected [n_seqs + 1]");
    given(cu_q, {cu_q.size(0)}, at::kInt, dev, "cu_q");
    given(cu_k, {cu_q.size(0)}, at::kInt, dev, "cu_k");
    const int32_t tq = size32(q.size(0), "q"), tk = size32(k.size(0), "k"), n = size32(cu_q.size(0) - 1, "cu_q");
    const int32_t hq = size32(q.size(1), "q"), hkv = size32(k.size(1), "k"), d = size32(q.size(2), "q");
    const at::Tensor out = output(a.v[8], {tq, hq, d}, type, dev, "out");
    at::Tensor lse;
    if (a.v[7] && truth(a.v[7])) lse = fresh({tq, hq}, at::kFloat, dev);
    const at::Tensor ws = workspace(a.v[9], a.v[9] ? 0 : spa_attention_prefill_workspace_bytes(tq, tk, n, hq, d), dev);
    check(attention_prefill(&qh, &kh, &vh, dtype_code(type), tq, tk, hq, hkv, d, static_cast<const int32_t*>(cu_q.data_ptr()),
                            static_cast<const int32_t*>(cu_k.data_ptr()), n, a.v[5] ? truth(a.v[5]) : 1,
                            scale_of(a.v[6], d), out.data_ptr(),
                            lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr,
                            ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (size_t)ws.numel() : 0, stream_of(dev)),
          "attention_prefill");
    return pair(back(a.v[8], out), back(nullptr, lse));
  });
}

spa_norm norm_of(PyObject* kind, int32_t dflt, PyObject* w, PyObject* b, int64_t c, at::ScalarType type, at::Device dev,
                 const char* name) {
  spa_norm n{dflt, nullptr, nullptr};
  if (kind) {
    const char* s = PyUnicode_AsUTF8(kind);
    if (!s) throw Raised();
    n.kind = !std::strcmp(s, "none") ? SPA_NORM_NONE : !std::strcmp(s, "rms") ? SPA_NORM_RMS
             : !std::strcmp(s, "layer") ? SPA_NORM_LAYER : -1;
    if (n.kind < 0) refuse(std::string(name) + ": unknown norm '" + s + "'");
  }
  if (w) {
    const at::Tensor& t = tensor(w, name);
    given(t, {c}, type, dev, name);
    n.weight = t.data_ptr();
  }
  if (b) {
    const at::Tensor& t = tensor(b, name);
    given(t, {c}, type, dev, name);
    n.bias = t.data_ptr();
  }
  return n;
}

PyDoc_STRVAR(gated_residual_norm_doc,
             "gated_residual_norm($module, /, x, residual=None, *, post='none', post_weight=None, post_bias=None, gate=None,"
             " scale=1.0, pre='rms', pre_weight=None, pre_bias=None, eps=1e-05, h_out=None, y_out=None)\n--\n\n"
             "h = residual + scale * gate * post(x) and y = pre(h) for rows x [t, c]: returns (h, y).\n\n"
             "residual [t, c] is of x's type or float32 and gives h its type (None: zeros of x's type); gate is [c] or\n"
             "[t, c]; post and pre are 'none', 'rms' or 'layer'.  h_out may be residual and y_out may be x.");
PyObject* py_gated_residual_norm(PyObject*, PyObject* const* args, Py_ssize_t n_args, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"x", "residual", "post", "post_weight", "post_bias", "gate", "scale", "pre",
                                        "pre_weight", "pre_bias", "eps", "h_out", "y_out"};
    Args<13> a("gated_residual_norm", names, 1, 2, args, n_args, kw);
    const at::Tensor& x = tensor(a.v[0], "x");
    need(x.is_cuda() && x.dim() == 2 && x.is_contiguous(), "x: expected a contiguous device tensor [t, c]");
    const int64_t t = x.size(0), c = x.size(1);
    const at::Device dev = x.device();
    const OnDevice on(dev);
    const at::ScalarType type = x.scalar_type();
    need(dtype_code(type) >= 0, "x: expected float32, float16 or bfloat16");
    held(x, x.numel(), "x");
    at::ScalarType stream_type = type;
    const void* residual = nullptr;
    if (a.v[1]) {
      const at::Tensor& r = tensor(a.v[1], "residual");
      stream_type = r.scalar_type();
      need(dtype_code(stream_type) >= 0, "residual: expected float32, float16 or bfloat16");
      given(r, {t, c}, stream_type, dev, "residual");
      residual = r.data_ptr();
    }
    const void* gate = nullptr;
    int32_t rows = 0;
    if (a.v[5]) {
      const at::Tensor& g = tensor(a.v[5], "gate");
      if (g.dim() == 1) given(g, {c}, type, dev, "gate");
      else given(g, {t, c}, type, dev, "gate");
      rows = g.dim() == 1 ? 1 : size32(t, "gate");
      gate = g.data_ptr();
    }
    const spa_norm post = norm_of(a.v[2], SPA_NORM_NONE, a.v[3], a.v[4], c, type, dev, "post");
    const spa_norm pre = norm_of(a.v[7], SPA_NORM_RMS, a.v[8], a.v[9], c, type, dev, "pre");
    const at::Tensor h = output(a.v[11], {t, c}, stream_type, dev, "h_out");
    const at::Tensor y = output(a.v[12], {t, c}, type, dev, "y_out");
    check(gated_residual_norm(x.data_ptr(), dtype_code(type), size32(t, "x"), size32(c, "x"), residual,
                              dtype_code(stream_type), &post, gate, rows, a.v[6] ? (float)number(a.v[6]) : 1.f, &pre,
                              a.v[10] ? (float)number(a.v[10]) : 1e-5f, h.data_ptr(), y.data_ptr(), stream_of(dev)),
          "gated_residual_norm");
    return pair(back(a.v[11], h), back(a.v[12], y));
  });
}

// Vectors of several heads that a call writes, of this shape, type and device.
spa_heads heads_out(const at::Tensor& x, c10::IntArrayRef shape, at::ScalarType type, at::Device dev, const char* name) {
  const spa_heads h = heads(x, name);
  if (x.sizes() != shape || x.scalar_type() != type || x.device() != dev)
    refuse(std::string(name) + ": differs from its input in shape, type or device");
  return h;
}

PyDoc_STRVAR(qk_norm_rope_doc,
             "qk_norm_rope($module, /, q, k, positions=None, inv_freq=None, *, norm='rms', q_weight=None, k_weight=None,"
             " q_bias=None, k_bias=None, eps=1e-05, interleaved=False, q_out=None, k_out=None, v=None, slots=None,"
             " cache=None)\n--\n\n"
             "The norm of each head of q [t, n_q_heads, head_dim] and k [t, n_kv_heads, head_dim] ('none', 'rms' or 'layer',\n"
             "weights and biases [head_dim]), and the rotation of its first 2 * len(inv_freq) elements by the angles\n"
             "positions[row] * inv_freq (int32 [t], float32): pairs (i, i + len(inv_freq)), or neighbours with interleaved.\n\n"
             "q_out may be q and k_out may be k.  With a cache, the new keys and v [t, n_kv_heads, head_dim] are stored at\n"
             "slots [t] int32 as kv_write would, and the keys are returned only where k_out is given.  Returns (q, k or None).");
PyObject* py_qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n_args, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    static const char* const names[] = {"q", "k", "positions", "inv_freq", "norm", "q_weight", "k_weight", "q_bias", "k_bias",
                                        "eps", "interleaved", "q_out", "k_out", "v", "slots", "cache"};
    Args<16> a("qk_norm_rope", names, 2, 4, args, n_args, kw);
    const at::Tensor &q = tensor(a.v[0], "q"), &k = tensor(a.v[1], "k");
    const spa_heads qh = heads(q, "q"), kh = heads(k, "k");
    const at::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    const OnDevice on(dev);
    need(dtype_code(type) >= 0 && k.scalar_type() == type, "qk_norm_rope: q and k are float16 or bfloat16, both the same");
    need(k.device() == dev, "qk_norm_rope: tensors on several devices");
    need(k.size(0) == q.size(0) && k.size(2) == q.size(2), "qk_norm_rope: q and k differ in rows or head_dim");
    const int64_t t = q.size(0), d = q.size(2);
    need(!a.v[2] == !a.v[3], "qk_norm_rope: positions and inv_freq belong together");
    spa_rope rope{nullptr, 0, a.v[10] ? truth(a.v[10]) : 0};
    const int32_t* pos = nullptr;
    if (a.v[2]) {
      const at::Tensor &p = tensor(a.v[2], "positions"), &f = tensor(a.v[3], "inv_freq");
      given(p, {t}, at::kInt, dev, "positions");
      need(f.dim() == 1, "inv_freq: expected [rotary_dim / 2]");
      given(f, {f.size(0)}, at::kFloat, dev, "inv_freq");
      need(2 * f.size(0) <= d, "inv_freq: more pairs than the head has");
      pos = static_cast<const int32_t*>(p.data_ptr());
      rope.inv_freq = static_cast<const float*>(f.data_ptr());
      rope.rotary_dim = (int32_t)(2 * f.size(0));
    }
    const spa_norm qn = norm_of(a.v[4], SPA_NORM_RMS, a.v[5], a.v[7], d, type, dev, "q_norm");
    const spa_norm kn = norm_of(a.v[4], SPA_NORM_RMS, a.v[6], a.v[8], d, type, dev, "k_norm");
    need(!a.v[13] == !a.v[15] && !a.v[14] == !a.v[15], "qk_norm_rope: v, slots and cache belong together");
    spa_kv_cache c{};
    spa_heads vh{};
    const int32_t* slots = nullptr;
    if (a.v[15]) {
      const Pages kv = cache(a.v[15]);
      const at::Tensor &v = tensor(a.v[13], "v"), &s = tensor(a.v[14], "slots");
      need(kv.dev == dev, "qk_norm_rope: tensors on several devices");
      need(k.size(1) == kv.c.n_heads && d == kv.c.head_dim, "qk_norm_rope: the cache has other heads");
      vh = heads_out(v, k.sizes(), type, dev, "v");
      given(s, {t}, at::kInt, dev, "slots");
      slots = static_cast<const int32_t*>(s.data_ptr());
      c = cache_for(kv, type);
    }
    const at::Tensor qo = a.v[11] ? tensor(a.v[11], "q_out") : fresh(q.sizes(), type, dev);
    const spa_heads qoh = heads_out(qo, q.sizes(), type, dev, "q_out");
    at::Tensor ko;
    spa_heads koh{};
    if (a.v[12] || !a.v[15]) {
      ko = a.v[12] ? tensor(a.v[12], "k_out") : fresh(k.sizes(), type, dev);
      koh = heads_out(ko, k.sizes(), type, dev, "k_out");
    }
    check(qk_norm_rope(&qh, &kh, a.v[15] ? &vh : nullptr, dtype_code(type), size32(t, "q"), size32(q.size(1), "q"),
                       size32(k.size(1), "k"), size32(d, "q"), pos, &rope, &qn, &kn, a.v[9] ? (float)number(a.v[9]) : 1e-5f, &qoh,
                       ko.defined() ? &koh : nullptr, slots, a.v[15] ? &c : nullptr, stream_of(dev)),
          "qk_norm_rope");
    if (a.v[15])
      for (PyObject* part : reinterpret_cast<const KvCache*>(a.v[15])->part)
        if (part && part != Py_None) written(THPVariable_Unpack(part));
    return pair(back(a.v[11], qo), back(a.v[12], ko));
  });
}

PyObject* py_set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

#define FAST(name, fn) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(fn)), METH_FASTCALL | METH_KEYWORDS, name##_doc}
PyMethodDef g_methods[] = {FAST(kv_write, py_kv_write),
                           FAST(kv_read, py_kv_read),
                           FAST(kv_plan, py_kv_plan),
                           FAST(attention_decode, py_attention_decode),
                           FAST(attention_prefill, py_attention_prefill),
                           FAST(gated_residual_norm, py_gated_residual_norm),
                           FAST(qk_norm_rope, py_qk_norm_rope),
                           {"_set_error", py_set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_layer_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_native() {
  g_cache_type.tp_name = "activation_sparsification_amd.KvCache";
  g_cache_type.tp_basicsize = sizeof(KvCache);
  g_cache_type.tp_flags = Py_TPFLAGS_DEFAULT | Py_TPFLAGS_HAVE_GC;
  g_cache_type.tp_doc =
      "KvCache(k, v, k_scale=None, v_scale=None)\n--\n\n"
      "A paged cache of one layer: k and v are [n_pages, n_heads, page_size, head_dim].\n\n"
      "float16 or bfloat16 pages hold the vectors as they are; float8_e4m3fn and int8 pages hold codes, with float32\n"
      "k_scale and v_scale [n_pages, n_heads, page_size]; uint8 pages [n_pages, n_heads, page_size, head_dim / 2] hold two\n"
      "e2m1 codes to a byte, with uint8 scales [n_pages, n_heads, ceil(head_dim / 32), page_size], exponent + 127 of a power\n"
      "of two for every 32 elements.  The cache keeps its tensors; each call works on the memory and sizes that they have\n"
      "then.";
  g_cache_type.tp_new = PyType_GenericNew;
  g_cache_type.tp_init = reinterpret_cast<initproc>(cache_init);
  g_cache_type.tp_dealloc = reinterpret_cast<destructor>(cache_dealloc);
  g_cache_type.tp_traverse = reinterpret_cast<traverseproc>(cache_traverse);
  g_cache_type.tp_clear = reinterpret_cast<inquiry>(cache_clear);
  g_cache_type.tp_members = cache_members;
  g_cache_type.tp_getset = cache_sizes;
  if (PyType_Ready(&g_cache_type) < 0) return nullptr;
  PyObject* m = PyModule_Create(&g_module);
  if (!m) return nullptr;
  Py_INCREF(&g_cache_type);
  if (PyModule_AddObject(m, "KvCache", reinterpret_cast<PyObject*>(&g_cache_type)) < 0) {
    Py_DECREF(&g_cache_type);
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
