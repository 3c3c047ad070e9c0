// calls.cpp -- the binding's calls of include/qmm.h's qmm_head*, qmm_cache* and qmm_attend*, natively.
//
// A decode step's calls take a few microseconds on the device, and as long in Python, most of it for looking at tensors one
// attribute at a time.  Each function here takes what its namesake in attention.py takes, makes the checks of the good case
// and the call.  Anything else -- an argument of another kind, a tensor elsewhere, a call that the library refuses -- gives
// None, nothing is launched, and attention.py, which defines the checks, does the same in Python and says what is wrong.
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>

#include <cmath>
#include <initializer_list>

#include "qmm.h"

namespace {

typedef const at::Tensor* Tensor;

// null unless a plain tensor (or parameter)
Tensor tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

int code(at::ScalarType t) {
  return t == at::kFloat ? QMM_F32 : t == at::kHalf ? QMM_F16 : t == at::kBFloat16 ? QMM_BF16 : -1;
}
at::ScalarType scalar(int code) { return code == QMM_F32 ? at::kFloat : code == QMM_F16 ? at::kHalf : at::kBFloat16; }

bool integer(PyObject* o, int64_t* v) {
  *v = PyLong_AsLongLong(o);
  return *v != -1 || !PyErr_Occurred();
}
bool number(PyObject* o, float* v) {
  const double d = PyFloat_AsDouble(o);
  *v = static_cast<float>(d);
  return d != -1.0 || !PyErr_Occurred();
}
// a dtype of the calls' results; *v stays where there is none
bool result_type(PyObject* o, int* v) {
  if (o == Py_None) return true;
  if (!THPDtype_Check(o)) return false;
  *v = code(reinterpret_cast<THPDtype*>(o)->scalar_type);
  return *v >= 0;
}

// [T, heads, D] on a device, the last axis contiguous
struct Rows {
  const void* p;
  int type;
  int64_t T, H, D, token, head;
  bool get(PyObject* o, int64_t device) {
    const Tensor t = tensor(o);
    if (!t || t->dim() != 3 || !t->is_cuda() || t->get_device() != device || t->stride(2) != 1) return false;
    type = code(t->scalar_type());
    T = t->size(0), H = t->size(1), D = t->size(2), token = t->stride(0), head = t->stride(1);
    p = t->data_ptr();
    return type >= 0;
  }
  bool like(const Rows& o) const { return type == o.type && T == o.T && D == o.D; }
};

// a contiguous vector of n elements; its pointer
template <typename P>
bool vector(PyObject* o, int64_t device, at::ScalarType type, int64_t n, P** p) {
  const Tensor t = tensor(o);
  if (!t || t->dim() != 1 || t->size(0) != n || t->scalar_type() != type || !t->is_cuda() || t->get_device() != device ||
      !t->is_contiguous())
    return false;
  *p = static_cast<P*>(t->data_ptr());
  return true;
}
// length of a vector, -1 unless it is one
int64_t length(PyObject* o) {
  const Tensor t = tensor(o);
  return t && t->dim() == 1 ? t->size(0) : -1;
}

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, int64_t device) {
  return at::empty(size, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, static_cast<at::DeviceIndex>(device))));
}

// positions, inv_freq, q_weight, k_weight, eps, interleaved
bool norm_args(PyObject* const* o, int64_t device, qmm_head_args* a) {
  if (o[1] != Py_None) {
    const int64_t n = length(o[1]);
    if (n < 0 || !vector(o[1], device, at::kFloat, n, &a->inv_freq) || !vector(o[0], device, at::kInt, a->T, &a->positions))
      return false;
    a->R = 2 * n;
  }
  const void** const weight[2] = {&a->q_weight, &a->k_weight};
  a->wt = -1;
  for (int i = 0; i < 2; ++i) {
    if (o[2 + i] == Py_None) continue;
    const Tensor t = tensor(o[2 + i]);
    const int type = t ? code(t->scalar_type()) : -1;
    if (type < 0 || (a->wt >= 0 && a->wt != type) || !vector(o[2 + i], device, t->scalar_type(), a->D, weight[i])) return false;
    a->wt = type;
  }
  if (a->wt < 0) a->wt = 0;
  const int on = PyObject_IsTrue(o[5]);
  a->interleaved = on;
  return on >= 0 && number(o[4], &a->eps);
}

void place(qmm_head_args* a, const Rows& q, const Rows& k) {
  a->q = q.p, a->q_token = q.token, a->q_head = q.head;
  a->k = k.p, a->k_token = k.token, a->k_head = k.head;
  a->T = q.T, a->Hq = q.H, a->H = k.H, a->D = q.D;
  a->xt = q.type;
}

qmm_stream_t stream_of(int64_t s) { return reinterpret_cast<qmm_stream_t>(s); }
const qmm_cache* cache_of(int64_t h) { return reinterpret_cast<const qmm_cache*>(h); }

// None where f declines or throws (out of memory, say: attention.py meets it again and lets torch report it)
template <typename F>
PyObject* attempt(F f) {
  try {
    PyObject* r = f();
    if (r) return r;
  } catch (...) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// device, stream, q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, dtype -> (q', k')
PyObject* head_norm_rope(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return attempt([&]() -> PyObject* {
    int64_t device, stream;
    Rows q, k;
    qmm_head_args a{};
    if (n != 11 || !integer(o[0], &device) || !integer(o[1], &stream) || !q.get(o[2], device) || !k.get(o[3], device) || !k.like(q))
      return nullptr;
    place(&a, q, k);
    a.ot = q.type;
    if (!norm_args(o + 4, device, &a) || !result_type(o[10], &a.ot)) return nullptr;
    at::Tensor qo = empty({q.T, q.H, q.D}, scalar(a.ot), device), ko = empty({k.T, k.H, k.D}, scalar(a.ot), device);
    a.q_out = qo.data_ptr(), a.k_out = ko.data_ptr();
    if (qmm_head_norm_rope(&a, stream_of(stream)) != QMM_OK) return nullptr;
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(qo)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(ko)));
    return r;
  });
}

// device, stream, cache, heads, D, type, q, k, v, slots, positions, inv_freq, q_weight, k_weight, eps, interleaved, dtype -> q'
PyObject* norm_rope_write(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return attempt([&]() -> PyObject* {
    int64_t device, stream, h, H, D, type;
    Rows q, k, v;
    qmm_head_args a{};
    if (n != 17 || !integer(o[0], &device) || !integer(o[1], &stream) || !integer(o[2], &h) || !integer(o[3], &H) ||
        !integer(o[4], &D) || !integer(o[5], &type) || !q.get(o[6], device) || !k.get(o[7], device) || !v.get(o[8], device) ||
        !k.like(q) || !v.like(q) || k.H != H || v.H != H || q.D != D)
      return nullptr;
    place(&a, q, k);
    a.v = v.p, a.v_token = v.token, a.v_head = v.head;
    a.ot = type == QMM_E4M3 ? q.type : static_cast<int>(type);
    if (!vector(o[9], device, at::kInt, q.T, &a.slots) || !norm_args(o + 10, device, &a) || !result_type(o[16], &a.ot) ||
        (type != QMM_E4M3 && a.ot != type))
      return nullptr;
    at::Tensor qo = empty({q.T, q.H, q.D}, scalar(a.ot), device);
    a.q_out = qo.data_ptr();
    return qmm_cache_norm_rope_write(cache_of(h), &a, stream_of(stream)) == QMM_OK ? THPVariable_Wrap(std::move(qo)) : nullptr;
  });
}

// device, stream, cache, heads, D, k, v, slots -> True
PyObject* write(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return attempt([&]() -> PyObject* {
    int64_t device, stream, h, H, D;
    Rows k, v;
    qmm_cache_write_args a{};
    if (n != 8 || !integer(o[0], &device) || !integer(o[1], &stream) || !integer(o[2], &h) || !integer(o[3], &H) ||
        !integer(o[4], &D) || !k.get(o[5], device) || !v.get(o[6], device) || !v.like(k) || k.H != H || v.H != H || k.D != D ||
        !vector(o[7], device, at::kInt, k.T, &a.slots))
      return nullptr;
    a.k = k.p, a.k_token = k.token, a.k_head = k.head;
    a.v = v.p, a.v_token = v.token, a.v_head = v.head;
    a.T = k.T, a.xt = k.type;
    if (qmm_cache_write(cache_of(h), &a, stream_of(stream)) != QMM_OK) return nullptr;
    Py_RETURN_TRUE;
  });
}

// a contiguous int32 [B, W] table
bool table_of(PyObject* o, int64_t device, int64_t B, const int32_t** p, int64_t* W) {
  const Tensor t = tensor(o);
  if (!t || t->dim() != 2 || t->size(0) != B || t->scalar_type() != at::kInt || !t->is_cuda() || t->get_device() != device ||
      !t->is_contiguous())
    return false;
  *p = static_cast<const int32_t*>(t->data_ptr());
  *W = t->size(1);
  return true;
}

// device, stream, cache, heads, D, type, table, starts, total, dtype -> (k, v)
PyObject* read(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return attempt([&]() -> PyObject* {
    int64_t device, stream, h, H, D, type;
    qmm_cache_read_args a{};
    if (n != 10 || !integer(o[0], &device) || !integer(o[1], &stream) || !integer(o[2], &h) || !integer(o[3], &H) ||
        !integer(o[4], &D) || !integer(o[5], &type) || !integer(o[8], &a.total))
      return nullptr;
    a.B = length(o[7]) - 1;
    a.ot = type == QMM_E4M3 ? QMM_BF16 : static_cast<int>(type);
    if (a.B < 0 || a.total < 0 || !table_of(o[6], device, a.B, &a.table, &a.W) ||
        !vector(o[7], device, at::kInt, a.B + 1, &a.starts) || !result_type(o[9], &a.ot))
      return nullptr;
    at::Tensor k = empty({a.total, H, D}, scalar(a.ot), device), v = empty({a.total, H, D}, scalar(a.ot), device);
    a.k = k.data_ptr(), a.v = v.data_ptr();
    if (qmm_cache_read(cache_of(h), &a, stream_of(stream)) != QMM_OK) return nullptr;
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(k)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(v)));
    return r;
  });
}

// device, stream, cache, heads, D, type, page, q, table, lengths, scale, max_length -> out
PyObject* attend(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return attempt([&]() -> PyObject* {
    int64_t device, stream, h, H, D, type, page;
    Rows q;
    qmm_attend_args a{};
    if (n != 12 || !integer(o[0], &device) || !integer(o[1], &stream) || !integer(o[2], &h) || !integer(o[3], &H) ||
        !integer(o[4], &D) || !integer(o[5], &type) || !integer(o[6], &page) || !q.get(o[7], device) || q.type == QMM_F32 ||
        (type != QMM_E4M3 && q.type != type) || q.D != D || H < 1 || q.H == 0 || q.H % H || !table_of(o[8], device, q.T, &a.table, &a.W) ||
        !vector(o[9], device, at::kInt, q.T, &a.lengths))
      return nullptr;
    a.max_length = a.W * page;
    if (o[11] != Py_None) {
      int64_t known;
      if (!PyLong_CheckExact(o[11]) || !integer(o[11], &known)) return nullptr;
      a.max_length = known < 0 ? 0 : known < a.max_length ? known : a.max_length;
    }
    a.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
    if (o[10] != Py_None && !number(o[10], &a.scale)) return nullptr;
    a.q = q.p, a.q_token = q.token, a.q_head = q.head;
    a.B = q.T, a.Hq = q.H, a.qt = q.type;
    a.ws_bytes = qmm_cache_attend_workspace_bytes(cache_of(h), a.B, a.Hq, a.max_length);
    at::Tensor out = empty({q.T, q.H, q.D}, scalar(q.type), device), ws;
    if (a.ws_bytes) {
      ws = empty({static_cast<int64_t>(a.ws_bytes)}, at::kByte, device);
      a.ws = ws.data_ptr();
    }
    a.out = out.data_ptr();
    return qmm_cache_attend(cache_of(h), &a, stream_of(stream)) == QMM_OK ? THPVariable_Wrap(std::move(out)) : nullptr;
  });
}

// device, stream, q, k, v, starts, k_starts, causal, scale -> out
PyObject* attend_prompt(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return attempt([&]() -> PyObject* {
    int64_t device, stream;
    Rows q, k, v;
    qmm_prompt_args a{};
    if (n != 9 || !integer(o[0], &device) || !integer(o[1], &stream) || !q.get(o[2], device) || !k.get(o[3], device) ||
        !v.get(o[4], device) || q.type == QMM_F32 || k.type != q.type || k.D != q.D || !v.like(k) || v.H != k.H || k.H == 0 ||
        q.H == 0 || q.H % k.H)
      return nullptr;
    const int64_t starts = length(o[5]);
    if (starts < 1 || !vector(o[5], device, at::kInt, starts, &a.q_starts)) return nullptr;
    a.k_starts = a.q_starts;
    if (o[6] == Py_None || o[6] == o[5]) {
      if (k.T != q.T) return nullptr;
    } else if (!vector(o[6], device, at::kInt, starts, &a.k_starts)) {
      return nullptr;
    }
    a.causal = PyObject_IsTrue(o[7]);
    a.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(q.D)));
    if (a.causal < 0 || (o[8] != Py_None && !number(o[8], &a.scale))) return nullptr;
    a.q = q.p, a.q_token = q.token, a.q_head = q.head;
    a.k = k.p, a.k_token = k.token, a.k_head = k.head;
    a.v = v.p, a.v_token = v.token, a.v_head = v.head;
    a.B = starts - 1, a.Tq = q.T, a.Tk = k.T, a.Hq = q.H, a.H = k.H, a.D = q.D, a.dt = q.type;
    at::Tensor out = empty({q.T, q.H, q.D}, scalar(q.type), device);
    a.out = out.data_ptr();
    return qmm_attend_prompt(&a, stream_of(stream)) == QMM_OK ? THPVariable_Wrap(std::move(out)) : nullptr;
  });
}

PyMethodDef kMethods[] = {
    {"head_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(head_norm_rope)), METH_FASTCALL, nullptr},
    {"norm_rope_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm_rope_write)), METH_FASTCALL, nullptr},
    {"write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(write)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(read)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"attend_prompt", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend_prompt)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// QMM_BUILT_FOR: torch.__version__ and Python's of the build.  Tensors' insides and Python's are inlined above, so a module of
// another build is refused, whether its symbols resolve or not; attention.py then goes without.
PyMODINIT_FUNC PyInit__calls() {
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
  PyObject* python = PySys_GetObject("version_info");  // borrowed
  PyObject* major = version && python ? PySequence_GetItem(python, 0) : nullptr;
  PyObject* minor = major ? PySequence_GetItem(python, 1) : nullptr;
  PyObject* here = minor ? PyUnicode_FromFormat("%S %S.%S", version, major, minor) : nullptr;
  const bool same = here && PyUnicode_CompareWithASCIIString(here, QMM_BUILT_FOR) == 0;
  if (here && !same) PyErr_Format(PyExc_ImportError, "built for torch and Python %s, not %U", QMM_BUILT_FOR, here);
  for (PyObject* o : {torch, version, major, minor, here}) Py_XDECREF(o);
  return same ? PyModule_Create(&kModule) : nullptr;
}
