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

#include "../../include/paged_attn.h"

namespace {

decltype(&paged_plan) f_plan;
decltype(&paged_kv_write) f_write;
decltype(&paged_attention) f_attention;
decltype(&paged_attention_workspace_bytes) f_ws_bytes;
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
    const char* tn = type == at::kInt ? "int32" : type == at::kLong ? "int64" : type == at::kFloat ? "float32" : "bfloat16";
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
    auto i32 = [&](const char* name, std::initializer_list<int64_t> sizes) {
      return static_cast<int32_t*>(a.tensor(name, at::kInt, sizes));
    };
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

// setup(PagedShape, addresses of paged_plan, paged_kv_write, paged_attention and
// paged_attention_workspace_bytes)
PyObject* py_setup(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call("setup", n, 5, [&]() -> PyObject* {
    void* f[4];
    for (int i = 0; i < 4; ++i) {
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
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "rglru_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_rglru_binding() { return PyModule_Create(&module); }
