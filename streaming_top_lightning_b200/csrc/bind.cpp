// Python calls of the key/value cache operators: argument checks and tensor
// addresses for the C ABI (include/streamindex.h), compiled.
//
// A decode step makes several of these calls per layer, each on kernels of a
// few microseconds, so what a call costs on the host is what it costs: checking
// the tensors and marshalling twenty-odd arguments takes about 8 us through
// Python and ctypes and well under 1 us here.  Nothing is computed here.
//
// Every function takes all its arguments by position and returns its result;
// None when the tensors are not on the current device (the caller switches to
// it); or a whole number, the library's error status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "streamindex.h"

namespace {

// The library's functions, found in the copy that ctypes has loaded.
struct Abi {
  decltype(&si_window_attention) window_attention;
  decltype(&si_window_attention_workspace_size) window_attention_workspace_size;
  decltype(&si_cache4_page_bytes) cache4_page_bytes;
  decltype(&si_cache4_append) cache4_append;
  decltype(&si_cache4_read) cache4_read;
  decltype(&si_cache4_attention) cache4_attention;
  decltype(&si_cache4_attention_workspace_size) cache4_attention_workspace_size;
  decltype(&si_cache_workspace_size) cache_workspace_size;
  decltype(&si_cache_extend) cache_extend;
  decltype(&si_cache_fork) cache_fork;
  decltype(&si_cache_free) cache_free;
  decltype(&si_cache_compact) cache_compact;
} abi;

struct PyError {};  // a Python exception is set

[[noreturn]] void fail(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw PyError{};
}

const at::Tensor& tensor(PyObject* o, const char* name, int64_t dims) {
  if (!THPVariable_Check(o)) fail(std::string(name) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) fail(std::string(name) + " must be a CUDA tensor");
  if (t.dim() != dims)
    fail(std::string(name) + " must be a " + std::to_string(dims) + "-d tensor");
  return t;
}

std::string list(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}

// The address of a contiguous tensor of this type and shape on device `dev`.
void* address(PyObject* o, const char* name, int dev, at::ScalarType type,
              std::initializer_list<int64_t> shape) {
  const at::Tensor& t = tensor(o, name, (int64_t)shape.size());
  if (t.get_device() != dev)
    fail(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
         ", the call's tensors are on cuda:" + std::to_string(dev));
  const at::IntArrayRef want(shape.begin(), shape.size());
  if (t.scalar_type() != type || t.sizes() != want || !t.is_contiguous())
    fail(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor " +
         list(want) + ", got " + c10::toString(t.scalar_type()) + " " + list(t.sizes()) +
         " with strides " + list(t.strides()));
  return t.data_ptr();
}
void* optional(PyObject* o, const char* name, int dev, at::ScalarType type,
               std::initializer_list<int64_t> shape) {
  return o == Py_None ? nullptr : address(o, name, dev, type, shape);
}

int whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  if (v < INT_MIN || v > INT_MAX) fail(std::string(name) + " is out of range");
  return (int)v;
}
// A size of a tensor as the C ABI's int (-1, which the library refuses, for more).
int size(int64_t n) { return n > INT_MAX ? -1 : (int)n; }

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError{};
  return (float)v;
}

const si_options* options(PyObject* o) {
  return o == Py_None ? nullptr : static_cast<const si_options*>(PyLong_AsVoidPtr(o));
}

void* stream(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

at::Tensor empty(const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

// The call's workspace: the caller's, or one of its own that lives until the
// kernels are in the stream.
struct Scratch {
  at::Tensor own;
  void* at = nullptr;
  size_t bytes = 0;
  Scratch(PyObject* given, size_t need, const at::Tensor& like) {
    if (given != Py_None) {
      const at::Tensor& t = tensor(given, "workspace", 1);
      if (t.scalar_type() != at::kByte || t.get_device() != like.get_device() ||
          !t.is_contiguous())
        fail("workspace must be a contiguous uint8 tensor on the call's device");
      at = t.data_ptr();
      bytes = (size_t)t.numel();
    } else if (need) {
      own = empty(like, {(int64_t)need}, at::kByte);
      at = own.data_ptr();
      bytes = need;
    }
  }
};

PyObject* status(int rc) { return PyLong_FromLong(rc); }

// out and lse of an attention call: the caller's or new ones.
struct Out {
  at::Tensor out, lse;
  PyObject *given_out, *given_lse;
  void *o, *l;
  Out(PyObject* go, PyObject* gl, const at::Tensor& q) : given_out(go), given_lse(gl) {
    const int dev = q.get_device();
    const int64_t B = q.size(0), S = q.size(1), H = q.size(2), D = q.size(3);
    if (go == Py_None) {
      out = empty(q, {B, S, H, D}, at::kBFloat16);
      o = out.data_ptr();
    } else {
      o = address(go, "out", dev, at::kBFloat16, {B, S, H, D});
    }
    if (gl == Py_None) {
      lse = empty(q, {B, S, H}, at::kFloat);
      l = lse.data_ptr();
    } else {
      l = address(gl, "lse", dev, at::kFloat, {B, S, H});
    }
  }
  PyObject* result() {
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, given_out == Py_None ? THPVariable_Wrap(out) : Py_NewRef(given_out));
    PyTuple_SET_ITEM(r, 1, given_lse == Py_None ? THPVariable_Wrap(lse) : Py_NewRef(given_lse));
    return r;
  }
};

bool elsewhere(const at::Tensor& t) {
  return t.get_device() != (int)c10::cuda::current_device();
}

// qa, ka, va, window, sinks, lens, q_lens, scale, out, lse, opts, workspace
PyObject* window_attention(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "qa", 4);
  const at::Tensor& k = tensor(a[1], "ka", 4);
  if (elsewhere(q)) Py_RETURN_NONE;
  const int dev = q.get_device();
  const int64_t B = q.size(0), S = q.size(1), H = q.size(2), D = q.size(3);
  const int64_t T = k.size(1), Hk = k.size(2);
  void* qp = address(a[0], "qa", dev, at::kBFloat16, {B, S, H, D});
  void* kp = address(a[1], "ka", dev, at::kBFloat16, {B, T, Hk, D});
  void* vp = address(a[2], "va", dev, at::kBFloat16, {B, T, Hk, D});
  const int window = whole(a[3], "window"), sinks = whole(a[4], "sinks");
  void* lens = optional(a[5], "lens", dev, at::kInt, {B});
  void* q_lens = optional(a[6], "q_lens", dev, at::kInt, {B});
  const float scale = a[7] == Py_None ? 1.0f / std::sqrt((float)D) : number(a[7]);
  const si_options* o = options(a[10]);
  size_t need = 0;
  int rc = abi.window_attention_workspace_size(size(B), size(S), size(T), size(H), size(Hk),
                                               size(D), window, sinks, o, &need);
  if (rc) return status(rc);
  Out out(a[8], a[9], q);
  const Scratch ws(a[11], need, q);
  rc = abi.window_attention(qp, kp, vp, (int32_t*)lens, (int32_t*)q_lens, size(B), size(S), size(T),
                            size(H), size(Hk), size(D), window, sinks, scale, out.o, (float*)out.l,
                            o, ws.at, ws.bytes, stream(dev));
  return rc ? status(rc) : out.result();
}

// A cache's pages, table and lengths.
struct Cache {
  int n, width;
  void *pages, *table, *lens, *q_lens;
  Cache(PyObject* const* a, int dev, int64_t B, int heads, int dim, int page) {
    size_t bytes = 0;
    const int rc = abi.cache4_page_bytes(heads, dim, page, &bytes);
    if (rc) fail("a 4-bit cache has 64 or 128 elements a head and pages of 16 to 256 tokens, a "
                 "power of two");
    n = size(tensor(a[0], "pages", 2).size(0));
    width = size(tensor(a[1], "table", 2).size(1));
    pages = address(a[0], "pages", dev, at::kByte, {n, (int64_t)bytes});
    table = address(a[1], "table", dev, at::kInt, {B, width});
    lens = address(a[2], "lens", dev, at::kInt, {B});
    q_lens = optional(a[3], "q_lens", dev, at::kInt, {B});
  }
};

// k, v, pages, table, lens, q_lens, page, k_scale, v_scale
PyObject* cache4_append(PyObject* const* a) {
  const at::Tensor& k = tensor(a[0], "k", 4);
  if (elsewhere(k)) Py_RETURN_NONE;
  const int dev = k.get_device();
  const int64_t B = k.size(0), S = k.size(1), Hk = k.size(2), D = k.size(3);
  const int page = whole(a[6], "page");
  void* kp = address(a[0], "k", dev, at::kBFloat16, {B, S, Hk, D});
  void* vp = address(a[1], "v", dev, at::kBFloat16, {B, S, Hk, D});
  const Cache c(a + 2, dev, B, size(Hk), size(D), page);
  const int rc = abi.cache4_append(kp, vp, size(B), size(S), size(Hk), size(D), c.pages, c.n,
                                   (int32_t*)c.table, c.width, page, (int32_t*)c.lens,
                                   (int32_t*)c.q_lens, number(a[7]), number(a[8]), stream(dev));
  return rc ? status(rc) : Py_NewRef(a[2]);
}

// pages, table, lens, q_lens, S, heads, dim, page, k_scale, v_scale, out k, out v
PyObject* cache4_read(PyObject* const* a) {
  const at::Tensor& pages = tensor(a[0], "pages", 2);
  if (elsewhere(pages)) Py_RETURN_NONE;
  const int dev = pages.get_device();
  const int64_t B = tensor(a[1], "table", 2).size(0);
  const int S = whole(a[4], "S"), heads = whole(a[5], "heads"), dim = whole(a[6], "dim");
  const int page = whole(a[7], "page");
  const Cache c(a, dev, B, heads, dim, page);
  if (S < 1) return status(SI_ERR_DIM);
  at::Tensor own[2];
  void* p[2];
  static const char* const names[2] = {"out[0]", "out[1]"};
  for (int i = 0; i < 2; ++i) {
    if (a[10 + i] == Py_None) {
      own[i] = empty(pages, {B, S, heads, dim}, at::kBFloat16);
      p[i] = own[i].data_ptr();
    } else {
      p[i] = address(a[10 + i], names[i], dev, at::kBFloat16, {B, S, heads, dim});
    }
  }
  const int rc = abi.cache4_read(p[0], p[1], size(B), S, heads, dim, c.pages, c.n,
                                 (int32_t*)c.table, c.width, page, (int32_t*)c.lens,
                                 (int32_t*)c.q_lens, number(a[8]), number(a[9]), stream(dev));
  if (rc) return status(rc);
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  for (int i = 0; i < 2; ++i)
    PyTuple_SET_ITEM(r, i, a[10 + i] == Py_None ? THPVariable_Wrap(own[i]) : Py_NewRef(a[10 + i]));
  return r;
}

// qa, pages, table, lens, q_lens, idx, heads, page, window, sinks, scale, k_scale, v_scale, out,
// lse, opts, workspace
PyObject* cache4_attention(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "qa", 4);
  if (elsewhere(q)) Py_RETURN_NONE;
  const int dev = q.get_device();
  const int64_t B = q.size(0), S = q.size(1), H = q.size(2), D = q.size(3);
  const int heads = whole(a[6], "heads"), page = whole(a[7], "page");
  const int window = whole(a[8], "window"), sinks = whole(a[9], "sinks");
  void* qp = address(a[0], "qa", dev, at::kBFloat16, {B, S, H, D});
  const Cache c(a + 1, dev, B, heads, size(D), page);
  int topk = 0;
  void* idx = nullptr;
  if (a[5] != Py_None) {
    topk = size(tensor(a[5], "idx", 3).size(2));
    idx = address(a[5], "idx", dev, at::kInt, {B, S, topk});
    if (topk < 1) return status(SI_ERR_TOPK);
  }
  const float scale = a[10] == Py_None ? 1.0f / std::sqrt((float)D) : number(a[10]);
  const float ks = number(a[11]), vs = number(a[12]);
  const si_options* o = options(a[15]);
  size_t need = 0;
  int rc = abi.cache4_attention_workspace_size(c.width, page, topk, size(B), size(S), size(H),
                                               heads, size(D), window, sinks, o, &need);
  if (rc) return status(rc);
  Out out(a[13], a[14], q);
  const Scratch ws(a[16], need, q);
  rc = abi.cache4_attention(qp, c.pages, c.n, (int32_t*)c.table, c.width, page, (int32_t*)c.lens,
                            (int32_t*)c.q_lens, (int32_t*)idx, topk, size(B), size(S), size(H),
                            heads, size(D), window, sinks, scale, ks, vs, out.o, (float*)out.l, o,
                            ws.at, ws.bytes, stream(dev));
  return rc ? status(rc) : out.result();
}

// A pool's counts, table and lengths (lens None: not part of the call).
struct Pool {
  int n, B, width;
  int32_t *refs, *table, *lens;
  Pool(PyObject* r, PyObject* t, PyObject* l, int dev) {
    n = size(tensor(r, "refs", 1).size(0));
    const at::Tensor& tt = tensor(t, "table", 2);
    B = size(tt.size(0));
    width = size(tt.size(1));
    refs = (int32_t*)address(r, "refs", dev, at::kInt, {n});
    table = (int32_t*)address(t, "table", dev, at::kInt, {B, width});
    lens = l == Py_None ? nullptr : (int32_t*)address(l, "lens", dev, at::kInt, {B});
  }
};

// refs, table, lens, page, workspace
PyObject* cache_extend(PyObject* const* a) {
  const at::Tensor& refs = tensor(a[0], "refs", 1);
  if (elsewhere(refs)) Py_RETURN_NONE;
  const int dev = refs.get_device(), page = whole(a[3], "page");
  tensor(a[2], "lens", 1);
  const Pool p(a[0], a[1], a[2], dev);
  size_t need = 0;
  int rc = abi.cache_workspace_size(p.n, p.B, 0, &need);
  if (rc) return status(rc);
  at::Tensor missing = empty(refs, {1}, at::kInt);
  const Scratch ws(a[4], need, refs);
  rc = abi.cache_extend(p.refs, p.n, p.table, p.B, p.width, p.lens, page,
                        missing.data_ptr<int32_t>(), ws.at, ws.bytes, stream(dev));
  return rc ? status(rc) : THPVariable_Wrap(missing);
}

// pages, refs, table, lens, src, dst, page, workspace
PyObject* cache_fork(PyObject* const* a) {
  const at::Tensor& refs = tensor(a[1], "refs", 1);
  if (elsewhere(refs)) Py_RETURN_NONE;
  const int dev = refs.get_device(), page = whole(a[6], "page");
  tensor(a[3], "lens", 1);
  const Pool p(a[1], a[2], a[3], dev);
  const int64_t bytes = tensor(a[0], "pages", 2).size(1);
  void* pages = address(a[0], "pages", dev, at::kByte, {p.n, bytes});
  const int64_t count = tensor(a[4], "src", 1).size(0);
  void* src = address(a[4], "src", dev, at::kInt, {count});
  void* dst = address(a[5], "dst", dev, at::kInt, {count});
  size_t need = 0;
  int rc = abi.cache_workspace_size(p.n, p.B, size(count), &need);
  if (rc) return status(rc);
  at::Tensor missing = empty(refs, {1}, at::kInt);
  const Scratch ws(a[7], need, refs);
  rc = abi.cache_fork(pages, bytes, p.refs, p.n, p.table, p.B, p.width, p.lens, (int32_t*)src,
                      (int32_t*)dst, size(count), page, missing.data_ptr<int32_t>(), ws.at,
                      ws.bytes, stream(dev));
  return rc ? status(rc) : THPVariable_Wrap(missing);
}

// refs, table, lens, rows
PyObject* cache_free(PyObject* const* a) {
  const at::Tensor& refs = tensor(a[0], "refs", 1);
  if (elsewhere(refs)) Py_RETURN_NONE;
  const int dev = refs.get_device();
  tensor(a[2], "lens", 1);
  const Pool p(a[0], a[1], a[2], dev);
  const int64_t count = tensor(a[3], "rows", 1).size(0);
  void* rows = address(a[3], "rows", dev, at::kInt, {count});
  const int rc = abi.cache_free(p.refs, p.n, p.table, p.B, p.width, p.lens, (int32_t*)rows,
                                size(count), stream(dev));
  return status(rc);
}

// pages, refs, table, new table, new refs, workspace
PyObject* cache_compact(PyObject* const* a) {
  const at::Tensor& refs = tensor(a[1], "refs", 1);
  if (elsewhere(refs)) Py_RETURN_NONE;
  const int dev = refs.get_device();
  const Pool p(a[1], a[2], Py_None, dev);
  const int64_t bytes = tensor(a[0], "pages", 2).size(1);
  void* pages = address(a[0], "pages", dev, at::kByte, {p.n, bytes});
  at::Tensor own_table, own_refs;
  int32_t *table, *counts;
  if (a[3] == Py_None) {
    own_table = empty(refs, {p.B, p.width}, at::kInt);
    own_refs = empty(refs, {p.n}, at::kInt);
    table = own_table.data_ptr<int32_t>();
    counts = own_refs.data_ptr<int32_t>();
  } else {
    table = (int32_t*)address(a[3], "out[0]", dev, at::kInt, {p.B, p.width});
    counts = (int32_t*)address(a[4], "out[1]", dev, at::kInt, {p.n});
  }
  size_t need = 0;
  int rc = abi.cache_workspace_size(p.n, p.B, 0, &need);
  if (rc) return status(rc);
  at::Tensor live = empty(refs, {1}, at::kInt);
  const Scratch ws(a[5], need, refs);
  rc = abi.cache_compact(pages, bytes, p.refs, p.n, p.table, p.B, p.width, counts, table,
                         live.data_ptr<int32_t>(), ws.at, ws.bytes, stream(dev));
  if (rc) return status(rc);
  PyObject* r = PyTuple_New(3);
  if (!r) return nullptr;
  const bool own = a[3] == Py_None;
  PyTuple_SET_ITEM(r, 0, own ? THPVariable_Wrap(own_table) : Py_NewRef(a[3]));
  PyTuple_SET_ITEM(r, 1, own ? THPVariable_Wrap(own_refs) : Py_NewRef(a[4]));
  PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(live));
  return r;
}

// Argument count and C++ exceptions of a call.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(a);
  } catch (const PyError&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// attach(path): find the library's functions.
PyObject* attach(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* h = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  if (!h) {
    PyErr_SetString(PyExc_ImportError, dlerror());
    return nullptr;
  }
  bool ok = true;
#define SI_FIND(NAME) \
  ok = ok && (abi.NAME = reinterpret_cast<decltype(abi.NAME)>(dlsym(h, "si_" #NAME))) != nullptr
  SI_FIND(window_attention);
  SI_FIND(window_attention_workspace_size);
  SI_FIND(cache4_page_bytes);
  SI_FIND(cache4_append);
  SI_FIND(cache4_read);
  SI_FIND(cache4_attention);
  SI_FIND(cache4_attention_workspace_size);
  SI_FIND(cache_workspace_size);
  SI_FIND(cache_extend);
  SI_FIND(cache_fork);
  SI_FIND(cache_free);
  SI_FIND(cache_compact);
#undef SI_FIND
  if (!ok) {
    PyErr_SetString(PyExc_ImportError, "the library lacks a function of this binding; build it again");
    return nullptr;
  }
  Py_RETURN_NONE;
}

#define SI_CALL(NAME, N) \
  {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<NAME, N>)), \
   METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"attach", attach, METH_O, nullptr},
    SI_CALL(window_attention, 12), SI_CALL(cache4_append, 9),  SI_CALL(cache4_read, 12),
    SI_CALL(cache4_attention, 17), SI_CALL(cache_extend, 5),   SI_CALL(cache_fork, 8),
    SI_CALL(cache_free, 4),        SI_CALL(cache_compact, 6),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods,
                      nullptr,               nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
