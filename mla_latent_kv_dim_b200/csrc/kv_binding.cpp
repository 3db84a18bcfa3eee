// Python binding of the tpla_kv_* entry points: argument marshalling only.
//
// A decode step makes these calls once a layer, and describing ten tensors
// from Python takes longer than a small call's kernels (30 us against 8).  The
// functions here describe torch tensors, allocate results and workspaces with
// torch and call the C entry points, whose addresses _native.py hands over
// once the library is loaded.  Return values: the library's status (<= 0), or
//   1  a tensor is not on the current CUDA device,
//   2  a tensor's type or rank has no descriptor,
// which _native.py turns into the same exceptions as everywhere else.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tpla.h"

namespace {

decltype(&tpla_kv_append) g_append = nullptr;
decltype(&tpla_kv_decode_workspace_size) g_decode_ws = nullptr;
decltype(&tpla_kv_decode) g_decode = nullptr;
decltype(&tpla_kv_prefill_workspace_size) g_prefill_ws = nullptr;
decltype(&tpla_kv_prefill) g_prefill = nullptr;

constexpr int kWrongDevice = 1, kNoDescriptor = 2;

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return TPLA_BF16;
    case at::kHalf: return TPLA_F16;
    case at::kFloat: return TPLA_F32;
    case at::kInt: return TPLA_I32;
    default: return 0;
  }
}

at::ScalarType scalar_type(int code) {
  return code == TPLA_BF16 ? at::kBFloat16 : code == TPLA_F16 ? at::kHalf : at::kFloat;
}

// One tensor argument: its descriptor, or null for None.
struct Arg {
  at::Tensor t;
  tpla_tensor d;
  bool none = true;
  tpla_tensor* ptr() { return none ? nullptr : &d; }
  void describe() {
    none = false;
    d = tpla_tensor{};
    d.data = t.numel() ? t.data_ptr() : nullptr;
    d.dtype = dtype_code(t.scalar_type());
    d.ndim = (int)t.dim();
    for (int i = 0; i < d.ndim && i < 4; ++i) {
      d.shape[i] = t.size(i);
      d.stride[i] = t.stride(i);
    }
  }
};

// False with a Python error set: not a tensor.  `bad`: a code above.
// `device`: the current one, asked for with the first CUDA tensor (-1 before).
bool get(PyObject* o, int* device, Arg* a, int* bad) {
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "expected a tensor or None, got %s", Py_TYPE(o)->tp_name);
    return false;
  }
  a->t = THPVariable_Unpack(o);
  if (a->t.is_cuda() && *device < 0) *device = c10::cuda::current_device();
  if (!a->t.is_cuda() || a->t.get_device() != *device) {
    *bad = kWrongDevice;
    return true;
  }
  if (dtype_code(a->t.scalar_type()) == 0 || a->t.dim() > 4) {
    if (*bad == 0) *bad = kNoDescriptor;
    return true;
  }
  a->describe();
  return true;
}

void make(Arg* a, at::IntArrayRef size, const at::Tensor& like, at::ScalarType type) {
  a->t = at::empty(size, like.options().dtype(type).requires_grad(false));
  a->describe();
}

PyObject* object_of(const Arg& a) {
  if (a.none) Py_RETURN_NONE;
  return THPVariable_Wrap(a.t);
}

tpla_stream_t stream_of(int device) {
  if (device < 0) return nullptr;  // no tensor at all: the library refuses the call
  return reinterpret_cast<tpla_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
}

bool expect(Py_ssize_t have, Py_ssize_t want) {
  if (have == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, have);
  return false;
}

// The caller's workspace where it is one run of memory and large enough, else
// a new one.
void* workspace(Arg* ws, size_t need, const at::Tensor& like, size_t* bytes) {
  *bytes = 0;
  if (need == 0) return nullptr;
  if (ws->t.defined() && ws->t.is_contiguous()) *bytes = (size_t)ws->t.numel() * ws->t.element_size();
  if (*bytes < need) {
    ws->t = at::empty({(int64_t)need}, like.options().dtype(at::kByte).requires_grad(false));
    *bytes = need;
  }
  return ws->t.data_ptr();
}

// A workspace may be of any type; only its place matters.
bool get_workspace(PyObject* o, int* device, Arg* a, int* bad) {
  int other = 0;
  if (!get(o, device, a, &other)) return false;
  if (other == kWrongDevice) *bad = kWrongDevice;
  return true;
}

// What torch raises (an allocation that does not fit, say) stays its own error.
#define KV_TRY try {
#define KV_CATCH                                                  \
  }                                                               \
  catch (...) {                                                   \
    torch::translate_exception_to_python(std::current_exception()); \
    return nullptr;                                               \
  }

PyObject* py_init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!expect(n, 5)) return nullptr;
  void* f[5];
  for (int i = 0; i < 5; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
      return nullptr;
    }
  }
  g_append = reinterpret_cast<decltype(g_append)>(f[0]);
  g_decode_ws = reinterpret_cast<decltype(g_decode_ws)>(f[1]);
  g_decode = reinterpret_cast<decltype(g_decode)>(f[2]);
  g_prefill_ws = reinterpret_cast<decltype(g_prefill_ws)>(f[3]);
  g_prefill = reinterpret_cast<decltype(g_prefill)>(f[4]);
  Py_RETURN_NONE;
}

// (k, v, positions, requests, page_table, k_cache, v_cache, cos_sin, q, q_out,
//  rope_offset, interleaved, q_rope_offset) -> (status, q_out)
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  KV_TRY
  if (!expect(n, 13)) return nullptr;
  int dev = -1;
  Arg t[10];
  int bad = 0;
  for (int i = 0; i < 10; ++i)
    if (!get(a[i], &dev, &t[i], &bad)) return nullptr;
  const long off = PyLong_AsLong(a[10]), inter = PyLong_AsLong(a[11]), q_off = PyLong_AsLong(a[12]);
  if (PyErr_Occurred()) return nullptr;
  if (bad == 0 && !t[8].none && t[9].none && !t[5].none)
    make(&t[9], t[8].t.sizes(), t[8].t, t[5].t.scalar_type());
  int rc = bad;
  if (bad == 0 && (off != (int)off || q_off != (int)q_off))
    rc = TPLA_ERR_INVALID_ARG;  // no column, and not one modulo 2^32
  else if (bad == 0)
    rc = g_append(t[0].ptr(), t[1].ptr(), t[2].ptr(), t[3].ptr(), t[4].ptr(), t[5].ptr(),
                  t[6].ptr(), t[7].ptr(), (int)off, (int)inter, t[8].ptr(), t[9].ptr(), (int)q_off,
                  stream_of(dev));
  return Py_BuildValue("(iN)", rc, object_of(t[9]));
  KV_CATCH
}

// (q, k_cache, v_cache, seq_lens, page_table, out, lse, workspace, scale,
//  out_dtype, want_lse) -> (status, out, lse)
PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  KV_TRY
  if (!expect(n, 11)) return nullptr;
  int dev = -1;
  Arg t[7], ws;
  int bad = 0;
  for (int i = 0; i < 7; ++i)
    if (!get(a[i], &dev, &t[i], &bad)) return nullptr;
  if (!get_workspace(a[7], &dev, &ws, &bad)) return nullptr;
  const double scale = PyFloat_AsDouble(a[8]);
  const long type = PyLong_AsLong(a[9]), want = PyLong_AsLong(a[10]);
  if (PyErr_Occurred()) return nullptr;
  int rc = bad;
  if (bad == 0) {
    if (!t[0].none && !t[2].none && t[0].t.dim() == 3 && t[2].t.dim() > 0) {
      const at::Tensor& q = t[0].t;
      if (t[5].none)
        make(&t[5], {q.size(0), q.size(1), t[2].t.size(-1)}, q, scalar_type((int)type));
      if (t[6].none && want) make(&t[6], {q.size(0), q.size(1), 1}, q, at::kFloat);
    }
    size_t need = 0, bytes = 0;
    rc = g_decode_ws(t[0].ptr(), t[1].ptr(), t[2].ptr(), t[4].ptr(), &need);
    if (rc == TPLA_OK) {
      void* w = workspace(&ws, need, t[0].t, &bytes);
      rc = g_decode(t[0].ptr(), t[1].ptr(), t[2].ptr(), t[3].ptr(), t[4].ptr(), (float)scale,
                    t[5].ptr(), t[6].ptr(), w, bytes, stream_of(dev));
    }
  }
  return Py_BuildValue("(iNN)", rc, object_of(t[5]), object_of(t[6]));
  KV_CATCH
}

// (q, k, v, cu_q, cu_k, seq_lens, page_table, out, lse, workspace, causal,
//  scale, out_dtype, want_lse) -> (status, out, lse)
PyObject* py_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  KV_TRY
  if (!expect(n, 14)) return nullptr;
  int dev = -1;
  Arg t[9], ws;
  int bad = 0;
  for (int i = 0; i < 9; ++i)
    if (!get(a[i], &dev, &t[i], &bad)) return nullptr;
  if (!get_workspace(a[9], &dev, &ws, &bad)) return nullptr;
  const long causal = PyLong_AsLong(a[10]);
  const double scale = PyFloat_AsDouble(a[11]);
  const long type = PyLong_AsLong(a[12]), want = PyLong_AsLong(a[13]);
  if (PyErr_Occurred()) return nullptr;
  int rc = bad;
  if (bad == 0) {
    if (!t[0].none && !t[2].none && t[0].t.dim() == 3 && t[2].t.dim() > 0) {
      const at::Tensor& q = t[0].t;
      if (t[7].none)
        make(&t[7], {q.size(0), q.size(1), t[2].t.size(-1)}, q, scalar_type((int)type));
      if (t[8].none && want) make(&t[8], {q.size(0), q.size(1), 1}, q, at::kFloat);
    }
    size_t need = 0, bytes = 0;
    rc = g_prefill_ws(t[0].ptr(), t[1].ptr(), t[2].ptr(), t[3].ptr(), t[6].ptr(), &need);
    if (rc == TPLA_OK) {
      void* w = workspace(&ws, need, t[0].t, &bytes);
      rc = g_prefill(t[0].ptr(), t[1].ptr(), t[2].ptr(), t[3].ptr(), t[4].ptr(), t[5].ptr(),
                     t[6].ptr(), (int)causal, (float)scale, t[7].ptr(), t[8].ptr(), w, bytes,
                     stream_of(dev));
    }
  }
  return Py_BuildValue("(iNN)", rc, object_of(t[7]), object_of(t[8]));
  KV_CATCH
}

PyMethodDef kMethods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_init)), METH_FASTCALL,
     "entry points of the loaded library"},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_append)),
     METH_FASTCALL, "tpla_kv_append"},
    {"kv_decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_decode)),
     METH_FASTCALL, "tpla_kv_decode"},
    {"kv_prefill", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_prefill)),
     METH_FASTCALL, "tpla_kv_prefill"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_kvbind", "marshalling of the tpla_kv_* calls", -1,
                       kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__kvbind(void) { return PyModule_Create(&kModule); }
