// Python entry points of the paged-cache calls (include/paged_attn.h): the checks of their tensors
// and the call, in one step.  A step of a serving loop makes three calls whose kernels take 2 to
// 10 us, and reading dtype, shape, device and strides of ten tensors through Python takes 4 us
// more than reading them here (measured for paged_plan: 8.0 us a call through Python, of which
// 2.2 us the ctypes call; 3.3 from here).
//
// The library is not linked: setup() is handed the addresses of its functions, so that
// whichever librglru.so the package has loaded is the one that is called.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>
#include <string>
#include <vector>

#include "../../include/paged_attn.h"
#include "../../include/paged_pages.h"
#include "../../include/paged_q4.h"

namespace {

decltype(&paged_plan) f_plan;
decltype(&paged_kv_write) f_write;
decltype(&paged_attention) f_attention;
decltype(&paged_attention_workspace_bytes) f_ws_bytes;
decltype(&paged_fork) f_fork;
decltype(&paged_release) f_release;
decltype(&paged_compact) f_compact;
decltype(&paged_copy) f_copy;
decltype(&paged_pages_workspace_bytes) f_pages_ws_bytes;
decltype(&paged_q4_write) f_q4_write;
decltype(&paged_q4_read) f_q4_read;
decltype(&paged_q4_attention) f_q4_attention;
decltype(&paged_q4_attention_workspace_bytes) f_q4_ws_bytes;
PyObject* g_shape_type;  // the package's PagedShape

// A call's arguments as they are taken one by one; after the first wrong one `ok` is false and a
// Python exception is set.
struct Args {
  PyObject* const* at;
  bool ok = true;
  int device = -1;  // of the tensors so far

  bool shape(paged_shape* s) {
    PyObject* o = *at++;
    if (!Py_IS_TYPE(o, reinterpret_cast<PyTypeObject*>(g_shape_type))) {
      PyErr_Format(PyExc_TypeError, "shape: want a PagedShape, not %R", o);
      return ok = false;
    }
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE)) return ok = false;
    memcpy(s, b.buf, sizeof *s);
    PyBuffer_Release(&b);
    return true;
  }

  // The next argument: a CUDA tensor of this type and shape; contiguous, or with `strided` only
  // in its last dimension.  `steps` (strided) receives its strides but the last; a dimension of one
  // element has the stride that a contiguous tensor would have.
  void* tensor(const char* name, at::ScalarType type, std::initializer_list<int64_t> sizes, bool strided = false,
               int64_t* const* steps = nullptr) {
    PyObject* o = *at++;
    if (!ok) return nullptr;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s: want a tensor, not %R", name, o);
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    const c10::IntArrayRef want(sizes);
    if (t.scalar_type() != type || !t.is_cuda() || t.layout() != at::kStrided || t.sizes() != want ||
        (strided ? t.strides().back() != 1 : !t.is_contiguous()) || (device >= 0 && t.get_device() != device)) {
      refuse(name, o, type, want, strided);
      return nullptr;
    }
    device = t.get_device();
    if (steps) {
      int64_t dense = want.back();
      for (size_t i = want.size() - 1; i-- > 0; dense *= want[i]) *steps[i] = want[i] > 1 ? t.strides()[i] : dense;
    }
    return t.data_ptr();
  }

  void refuse(const char* name, PyObject* o, at::ScalarType type, c10::IntArrayRef want, bool strided) {
    ok = false;
    std::string w = "(";
    for (size_t i = 0; i < want.size(); ++i) w += (i ? ", " : "") + std::to_string(want[i]);
    w += want.size() == 1 ? ",)" : ")";
    const char* tn = type == at::kInt ? "int32" : type == at::kLong ? "int64" : type == at::kFloat ? "float32" :
                     type == at::kByte ? "uint8" : type == at::ScalarType::Float8_e4m3fn ? "float8_e4m3fn" : "bfloat16";
    PyObject* n = PyObject_GetAttrString(o, "shape");
    PyObject* sizes = n ? PySequence_Tuple(n) : nullptr;
    PyObject* dtype = sizes ? PyObject_GetAttrString(o, "dtype") : nullptr;
    PyObject* dev = dtype ? PyObject_GetAttrString(o, "device") : nullptr;
    PyObject* st = dev ? PyObject_CallMethod(o, "stride", nullptr) : nullptr;
    if (st)  // (else one of them has raised)
      PyErr_Format(PyExc_ValueError, "%s: want a %s, %s torch.%s, not %S %S on %S with strides %S", name,
                   strided ? "CUDA tensor with a contiguous last dimension" : "contiguous CUDA tensor", w.c_str(), tn,
                   sizes, dtype, dev, st);
    for (PyObject* x : {n, sizes, dtype, dev, st}) Py_XDECREF(x);
  }

  int32_t* i32(const char* name, std::initializer_list<int64_t> sizes) {
    return static_cast<int32_t*>(tensor(name, at::kInt, sizes));
  }

  // The number of rows of the next argument, 0 where it has none; it is not taken yet.
  int64_t rows() const {
    if (!ok || !THPVariable_Check(*at)) return 0;
    const at::Tensor& t = THPVariable_Unpack(*at);
    return t.dim() > 0 && t.layout() == at::kStrided ? t.size(0) : 0;
  }

  // A cache of this many pages: of any type, its pages apart from one another.
  bool pages(PyObject* o, int64_t num_pages, void** base, int64_t* stride, int64_t* bytes) {
    if (!ok) return false;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "caches: want tensors, not %R", o);
      return ok = false;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    const bool strided = t.layout() == at::kStrided;
    int64_t span = 1;  // elements from a page's first to its last
    if (strided)
      for (int64_t d = 1; d < t.dim(); ++d) span += (t.size(d) - 1) * t.stride(d);
    if (!strided || !t.is_cuda() || t.dim() < 1 || t.size(0) != num_pages || t.numel() == 0 ||
        (num_pages > 1 && t.stride(0) < span) || (device >= 0 && t.get_device() != device)) {
      PyObject* n = PyObject_GetAttrString(o, "shape");
      PyObject* dev = n ? PyObject_GetAttrString(o, "device") : nullptr;
      if (dev)  // (else one of them has raised)
        PyErr_Format(PyExc_ValueError, "caches: want CUDA tensors of %lld pages that lie apart, on one device, not %S on %S",
                     (long long)num_pages, n, dev);
      Py_XDECREF(n);
      Py_XDECREF(dev);
      return ok = false;
    }
    device = t.get_device();
    *base = t.data_ptr();
    *bytes = span * t.element_size();
    *stride = num_pages > 1 ? t.stride(0) * t.element_size() : *bytes;
    return true;
  }

  // The next argument: a contiguous CUDA tensor of any type, of that many bytes or more.
  void* scratch(const char* name, size_t bytes) {
    PyObject* o = *at;
    if (!ok || !THPVariable_Check(o)) return tensor(name, at::kByte, {(int64_t)bytes});
    const at::Tensor& t = THPVariable_Unpack(o);
    ++at;
    if (t.layout() != at::kStrided || !t.is_cuda() || !t.is_contiguous() || t.nbytes() < bytes ||
        (device >= 0 && t.get_device() != device)) {
      const int64_t want = bytes;
      refuse(name, o, at::kByte, want, false);
      return nullptr;
    }
    return t.data_ptr();
  }

  // The last argument: a stream's handle, or None for the current one.
  cudaStream_t stream() {
    PyObject* o = *at++;
    if (!ok) return nullptr;
    if (device >= 0 && device != c10::cuda::current_device()) {
      PyErr_Format(PyExc_ValueError, "the tensors are on cuda:%d, the current device is another", device);
      ok = false;
      return nullptr;
    }
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) ok = false;
    return static_cast<cudaStream_t>(p);
  }
};

// One Python function: its number of arguments, and C++ exceptions (a tensor without storage, a
// CUDA error) as Python ones.
template <class F>
PyObject* call(const char* name, Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%s: %zd arguments, not %zd", name, want, n);
    return nullptr;
  }
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// f() without the interpreter's lock (a launch waits while the stream's queue is full)
template <class F>
PyObject* launch(F f) {
  rglru_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

at::ScalarType io_type(const paged_shape& s) { return s.io == RGLRU_F32 ? at::kFloat : at::kBFloat16; }

PyObject* py_plan(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call("paged_plan", n, 12, [&]() -> PyObject* {
    Args a{args};
    paged_shape s;
    if (!a.shape(&s)) return nullptr;
    const int64_t N = s.num_seqs, T = s.tokens;
    auto i32 = [&](const char* name, std::initializer_list<int64_t> sizes) { return a.i32(name, sizes); };
    int32_t* cached = i32("cached_lens", {N});
    int32_t* fresh = i32("new_lens", {N});
    int32_t* ring = i32("free_pages", {s.num_pages});
    int32_t* state = i32("free_state", {3});
    int32_t* table = i32("block_table", {N, s.table_width});
    int32_t* cu = i32("cu_seqlens", {N + 1});
    int32_t* kv = i32("kv_lens", {N});
    int32_t* positions = i32("positions", {T});
    int64_t* slots = static_cast<int64_t*>(a.tensor("slots", at::kLong, {T}));
    int32_t* out = i32("free_state_out", {3});
    const cudaStream_t stream = a.stream();
    if (!a.ok) return nullptr;
    return launch([&] { return f_plan(&s, cached, fresh, ring, state, table, cu, kv, positions, slots, out, stream); });
  });
}

PyObject* py_write(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call("paged_kv_write", n, 7, [&]() -> PyObject* {
    Args a{args};
    paged_shape s;
    if (!a.shape(&s)) return nullptr;
    const at::ScalarType io = io_type(s);
    paged_strides t = {};
    int64_t* const ks[] = {&t.k_token, &t.k_head};
    int64_t* const vs[] = {&t.v_token, &t.v_head};
    int64_t* const kcs[] = {&t.kc_page, &t.kc_token, &t.kc_head};
    int64_t* const vcs[] = {&t.vc_page, &t.vc_token, &t.vc_head};
    void* k = a.tensor("k", io, {s.tokens, s.Hkv, s.D}, true, ks);
    void* v = a.tensor("v", io, {s.tokens, s.Hkv, s.D}, true, vs);
    int64_t* slots = static_cast<int64_t*>(a.tensor("slots", at::kLong, {s.tokens}));
    void* kc = a.tensor("k_cache", io, {s.num_pages, s.page_size, s.Hkv, s.D}, true, kcs);
    void* vc = a.tensor("v_cache", io, {s.num_pages, s.page_size, s.Hkv, s.D}, true, vcs);
    const cudaStream_t stream = a.stream();
    if (!a.ok) return nullptr;
    return launch([&] { return f_write(&s, &t, k, v, slots, kc, vc, stream); });
  });
}

PyObject* py_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call("paged_attention", n, 12, [&]() -> PyObject* {
    Args a{args};
    paged_shape s;
    if (!a.shape(&s)) return nullptr;
    const at::ScalarType io = io_type(s);
    paged_strides t = {};
    int64_t* const qs[] = {&t.q_token, &t.q_head};
    int64_t* const os[] = {&t.o_token, &t.o_head};
    int64_t* const kcs[] = {&t.kc_page, &t.kc_token, &t.kc_head};
    int64_t* const vcs[] = {&t.vc_page, &t.vc_token, &t.vc_head};
    void* q = a.tensor("q", io, {s.tokens, s.Hq, s.D}, true, qs);
    void* kc = a.tensor("k_cache", io, {s.num_pages, s.page_size, s.Hkv, s.D}, true, kcs);
    void* vc = a.tensor("v_cache", io, {s.num_pages, s.page_size, s.Hkv, s.D}, true, vcs);
    int32_t* table = static_cast<int32_t*>(a.tensor("block_table", at::kInt, {s.num_seqs, s.table_width}));
    int32_t* cu = static_cast<int32_t*>(a.tensor("cu_seqlens", at::kInt, {(int64_t)s.num_seqs + 1}));
    int32_t* kv = static_cast<int32_t*>(a.tensor("kv_lens", at::kInt, {s.num_seqs}));
    const double scale = PyFloat_AsDouble(*a.at++);
    if (a.ok && scale == -1.0 && PyErr_Occurred()) return nullptr;
    void* o = a.tensor("o", io, {s.tokens, s.Hq, s.D}, true, os);
    float* lse = nullptr;
    if (*a.at == Py_None)
      ++a.at;
    else
      lse = static_cast<float*>(a.tensor("lse", at::kFloat, {s.tokens, s.Hq}));
    void* ws = a.scratch("workspace", f_ws_bytes(&s));
    const cudaStream_t stream = a.stream();
    if (!a.ok) return nullptr;
    return launch([&] {
      return f_attention(&s, &t, q, kc, vc, table, cu, kv, static_cast<float>(scale), o, lse, ws, stream);
    });
  });
}

PyObject* py_fork(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call("paged_fork", n, 14, [&]() -> PyObject* {
    Args a{args};
    paged_shape s;
    if (!a.shape(&s)) return nullptr;
    const int64_t N = s.num_seqs, W = s.table_width, P = s.num_pages, M = a.rows();
    int32_t* parents = a.i32("parents", {M});
    int32_t* children = a.i32("children", {M});
    int32_t* table = a.i32("block_table", {N, W});
    int32_t* lens = a.i32("kv_lens", {N});
    int32_t* holders = a.i32("holders", {P});
    int32_t* ring = a.i32("free_pages", {P});
    int32_t* state = a.i32("free_state", {3});
    int32_t* table_out = a.i32("block_table_out", {N, W});
    int32_t* lens_out = a.i32("kv_lens_out", {N});
    int32_t* holders_out = a.i32("holders_out", {P});
    int32_t* moves = a.i32("moves", {M, 2});
    int32_t* out = a.i32("free_state_out", {3});
    const cudaStream_t stream = a.stream();
    if (!a.ok) return nullptr;
    const int32_t m = M > 0x7fffffff ? -1 : (int32_t)M;
    return launch([&] {
      return f_fork(&s, m, parents, children, table, lens, holders, ring, state, table_out, lens_out, holders_out, moves, out, stream);
    });
  });
}

PyObject* py_release(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call("paged_release", n, 12, [&]() -> PyObject* {
    Args a{args};
    paged_shape s;
    if (!a.shape(&s)) return nullptr;
    const int64_t N = s.num_seqs, W = s.table_width, P = s.num_pages;
    int32_t* first = a.i32("first_pages", {N});
    int32_t* end = a.i32("end_pages", {N});
    int32_t* table = a.i32("block_table", {N, W});
    int32_t* holders = a.i32("holders", {P});
    int32_t* ring = a.i32("free_pages", {P});
    int32_t* state = a.i32("free_state", {3});
    int32_t* table_out = a.i32("block_table_out", {N, W});
    int32_t* holders_out = a.i32("holders_out", {P});
    int32_t* out = a.i32("free_state_out", {3});
    void* ws = a.scratch("workspace", f_pages_ws_bytes(&s));
    const cudaStream_t stream = a.stream();
    if (!a.ok) return nullptr;
    return launch([&] { return f_release(&s, first, end, table, holders, ring, state, table_out, holders_out, out, ws, stream); });
  });
}

PyObject* py_compact(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call("paged_compact", n, 11, [&]() -> PyObject* {
    Args a{args};
    paged_shape s;
    if (!a.shape(&s)) return nullptr;
    const int64_t N = s.num_seqs, W = s.table_width, P = s.num_pages;
    int32_t* lens = a.i32("kv_lens", {N});
    int32_t* table = a.i32("block_table", {N, W});
    int32_t* holders = a.i32("holders", {P});
    int32_t* table_out = a.i32("block_table_out", {N, W});
    int32_t* holders_out = a.i32("holders_out", {P});
    int32_t* ring = a.i32("free_pages", {P});
    int32_t* out = a.i32("free_state_out", {3});
    int32_t* moves = a.i32("moves", {P / 2, 2});
    void* ws = a.scratch("workspace", f_pages_ws_bytes(&s));
    const cudaStream_t stream = a.stream();
    if (!a.ok) return nullptr;
    return launch([&] { return f_compact(&s, lens, table, holders, table_out, holders_out, ring, out, moves, ws, stream); });
  });
}

// (the caches: a tuple)
PyObject* py_copy(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call("paged_copy", n, 4, [&]() -> PyObject* {
    Args a{args};
    paged_shape s;
    if (!a.shape(&s)) return nullptr;
    const int64_t M = a.rows();
    int32_t* moves = a.i32("moves", {M, 2});
    PyObject* caches = *a.at++;
    const Py_ssize_t k = a.ok ? PyTuple_Size(caches) : 0;
    if (k < 0) return nullptr;
    std::vector<void*> base(k);
    std::vector<int64_t> stride(k), bytes(k);
    for (Py_ssize_t c = 0; c < k; ++c)
      if (!a.pages(PyTuple_GET_ITEM(caches, c), s.num_pages, &base[c], &stride[c], &bytes[c])) return nullptr;
    const cudaStream_t stream = a.stream();
    if (!a.ok) return nullptr;
    const int32_t m = M > 0x7fffffff ? -1 : (int32_t)M;
    return launch([&] { return f_copy(&s, m, moves, (int32_t)k, base.data(), stride.data(), bytes.data(), stream); });
  });
}

// A cache in 4 bits, as it is passed: codes and scales of keys, then of values.
struct Q4Arrays {
  void* at[4];
  bool take(Args& a, const paged_shape& s, paged_q4_strides& t) {
    static const char* const names[4] = {"k_codes", "k_scales", "v_codes", "v_scales"};
    int64_t* const steps[4][3] = {{&t.kc_page, &t.kc_token, &t.kc_head}, {&t.ks_page, &t.ks_token, &t.ks_head},
                                  {&t.vc_page, &t.vc_token, &t.vc_head}, {&t.vs_page, &t.vs_token, &t.vs_head}};
    const int64_t n[3] = {s.num_pages, s.page_size, s.Hkv};
    for (int i = 0; i < 4; ++i) {
      const bool scales = i & 1;
      at[i] = a.tensor(names[i], scales ? at::ScalarType::Float8_e4m3fn : at::kByte,
                       {s.num_pages, s.page_size, s.Hkv, s.D / (scales ? 16 : 2)}, true, steps[i]);
      for (int d = 0; d < 3; ++d)
        if (n[d] == 1) *steps[i][d] = 16;  // (of one element: no step is taken)
    }
    return a.ok;
  }
};

template <bool WRITE>
PyObject* py_q4_rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(WRITE ? "paged_q4_write" : "paged_q4_read", n, 9, [&]() -> PyObject* {
    Args a{args};
    paged_shape s;
    if (!a.shape(&s)) return nullptr;
    paged_q4_strides t = {};
    void *k = nullptr, *v = nullptr;
    int64_t* slots = nullptr;
    Q4Arrays c;
    auto rows = [&] {
      int64_t* const ks[] = {&t.k_token, &t.k_head};
      int64_t* const vs[] = {&t.v_token, &t.v_head};
      k = a.tensor("k", io_type(s), {s.tokens, s.Hkv, s.D}, true, ks);
      v = a.tensor("v", io_type(s), {s.tokens, s.Hkv, s.D}, true, vs);
    };
    if (WRITE) rows();
    slots = static_cast<int64_t*>(a.tensor("slots", at::kLong, {s.tokens}));
    c.take(a, s, t);
    if (!WRITE) rows();
    const cudaStream_t stream = a.stream();
    if (!a.ok) return nullptr;
    return launch([&] {
      return WRITE ? f_q4_write(&s, &t, k, v, slots, c.at[0], c.at[1], c.at[2], c.at[3], stream)
                   : f_q4_read(&s, &t, slots, c.at[0], c.at[1], c.at[2], c.at[3], k, v, stream);
    });
  });
}

PyObject* py_q4_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call("paged_q4_attention", n, 14, [&]() -> PyObject* {
    Args a{args};
    paged_shape s;
    if (!a.shape(&s)) return nullptr;
    paged_q4_strides t = {};
    int64_t* const qs[] = {&t.q_token, &t.q_head};
    int64_t* const os[] = {&t.o_token, &t.o_head};
    void* q = a.tensor("q", io_type(s), {s.tokens, s.Hq, s.D}, true, qs);
    Q4Arrays c;
    c.take(a, s, t);
    int32_t* table = a.i32("block_table", {s.num_seqs, s.table_width});
    int32_t* cu = a.i32("cu_seqlens", {(int64_t)s.num_seqs + 1});
    int32_t* kv = a.i32("kv_lens", {s.num_seqs});
    const double scale = PyFloat_AsDouble(*a.at++);
    if (a.ok && scale == -1.0 && PyErr_Occurred()) return nullptr;
    void* o = a.tensor("o", io_type(s), {s.tokens, s.Hq, s.D}, true, os);
    float* lse = nullptr;
    if (*a.at == Py_None)
      ++a.at;
    else
      lse = static_cast<float*>(a.tensor("lse", at::kFloat, {s.tokens, s.Hq}));
    void* ws = a.scratch("workspace", f_q4_ws_bytes(&s));
    const cudaStream_t stream = a.stream();
    if (!a.ok) return nullptr;
    return launch([&] {
      return f_q4_attention(&s, &t, q, c.at[0], c.at[1], c.at[2], c.at[3], table, cu, kv, static_cast<float>(scale), o, lse, ws, stream);
    });
  });
}

// setup(PagedShape, the addresses of the library's functions in the order of `f`)
PyObject* py_setup(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr int F = 13;
  return call("setup", n, 1 + F, [&]() -> PyObject* {
    void* f[F];
    for (int i = 0; i < F; ++i) {
      f[i] = PyLong_AsVoidPtr(args[1 + i]);
      if (!f[i]) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "setup: a null address");
        return nullptr;
      }
    }
    f_plan = reinterpret_cast<decltype(f_plan)>(f[0]);
    f_write = reinterpret_cast<decltype(f_write)>(f[1]);
    f_attention = reinterpret_cast<decltype(f_attention)>(f[2]);
    f_ws_bytes = reinterpret_cast<decltype(f_ws_bytes)>(f[3]);
    f_fork = reinterpret_cast<decltype(f_fork)>(f[4]);
    f_release = reinterpret_cast<decltype(f_release)>(f[5]);
    f_compact = reinterpret_cast<decltype(f_compact)>(f[6]);
    f_copy = reinterpret_cast<decltype(f_copy)>(f[7]);
    f_pages_ws_bytes = reinterpret_cast<decltype(f_pages_ws_bytes)>(f[8]);
    f_q4_write = reinterpret_cast<decltype(f_q4_write)>(f[9]);
    f_q4_read = reinterpret_cast<decltype(f_q4_read)>(f[10]);
    f_q4_attention = reinterpret_cast<decltype(f_q4_attention)>(f[11]);
    f_q4_ws_bytes = reinterpret_cast<decltype(f_q4_ws_bytes)>(f[12]);
    Py_INCREF(args[0]);
    Py_XDECREF(g_shape_type);
    g_shape_type = args[0];
    Py_RETURN_NONE;
  });
}

template <class F>
PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"setup", fast(py_setup), METH_FASTCALL, nullptr},
                         {"paged_plan", fast(py_plan), METH_FASTCALL, nullptr},
                         {"paged_kv_write", fast(py_write), METH_FASTCALL, nullptr},
                         {"paged_attention", fast(py_attention), METH_FASTCALL, nullptr},
                         {"paged_fork", fast(py_fork), METH_FASTCALL, nullptr},
                         {"paged_release", fast(py_release), METH_FASTCALL, nullptr},
                         {"paged_compact", fast(py_compact), METH_FASTCALL, nullptr},
                         {"paged_copy", fast(py_copy), METH_FASTCALL, nullptr},
                         {"paged_q4_write", fast(py_q4_rows<true>), METH_FASTCALL, nullptr},
                         {"paged_q4_read", fast(py_q4_rows<false>), METH_FASTCALL, nullptr},
                         {"paged_q4_attention", fast(py_q4_attention), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "rglru_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_rglru_binding() { return PyModule_Create(&module); }
