// Calls of the operators (include/cdb_ops.h) on PyTorch tensors, for ops.py: each
// takes the addresses of a C entry point and of its argument structure, checks
// the tensors, fills in their pointers and strides and makes the call.  The
// checks cost a few nanoseconds a tensor here, where the same ones in Python
// cost 0.4 to 0.8 us, in total more than the kernel of a small call takes (cache
// write of one row, calls one behind another: 7.6 us a call so, 3.8 with these;
// attention of one row 9.4 and 8.7, where its two kernels take 7.3).
//
// A call returns the entry point's result, or None if a tensor is not what the
// operator takes: ops.py then says which and why.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>

#include "../../include/cdb.h"
#include "../../include/cdb_ops.h"

namespace {

const at::Tensor* tensor(PyObject* o, int dev) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.layout() == at::kStrided && t.get_device() == dev && !t.is_neg() ? &t : nullptr;
}

// A contiguous vector of at least n elements; None where it may be absent.
bool vec(PyObject* o, int dev, at::ScalarType type, int64_t n, const void** p, bool needed) {
  *p = nullptr;
  if (o == Py_None) return !needed;
  const at::Tensor* t = tensor(o, dev);
  if (!t || t->scalar_type() != type || t->numel() < n || !t->is_contiguous()) return false;
  *p = t->data_ptr();
  return true;
}

// [>= rows, >= cols] with contiguous rows, one behind another.
bool mat(const at::Tensor& t, int64_t rows, int64_t cols, const void** p, int64_t* ld) {
  if (t.dim() != 2 || t.size(0) < rows || t.size(1) < cols || (t.stride(1) != 1 && t.size(1) > 1) ||
      (t.stride(0) < t.size(1) && t.size(0) > 1))
    return false;
  *p = t.data_ptr();
  *ld = std::max(t.stride(0), t.size(1));  // one row: its stride says nothing
  return true;
}
// An fp32 or bf16 input: its rows and its CDB_* type.
bool input(PyObject* o, int dev, int* dtype, int* rows, int most, int64_t cols, const void** p, int64_t* ld) {
  const at::Tensor* t = tensor(o, dev);
  if (!t || t->dim() != 2 || t->size(0) > most) return false;
  if (t->scalar_type() == at::kFloat) *dtype = CDB_FP32;
  else if (t->scalar_type() == at::kBFloat16) *dtype = CDB_BF16;
  else return false;
  *rows = (int)t->size(0);
  return mat(*t, *rows, cols, p, ld);
}
bool bf16_mat(PyObject* o, int dev, int64_t rows, int64_t cols, const void** p, int64_t* ld) {
  const at::Tensor* t = tensor(o, dev);
  return t && t->scalar_type() == at::kBFloat16 && mat(*t, rows, cols, p, ld);
}

// The first four arguments of every call: entry point, argument structure, stream, device.
template <typename A>
struct Head {
  int (*fn)(const A*, void*) = nullptr;
  A* a = nullptr;
  void* stream = nullptr;
  int dev = -1;
  bool get(PyObject* const* v) {
    fn = reinterpret_cast<int (*)(const A*, void*)>(PyLong_AsVoidPtr(v[0]));
    a = static_cast<A*>(PyLong_AsVoidPtr(v[1]));
    stream = PyLong_AsVoidPtr(v[2]);
    dev = (int)PyLong_AsLong(v[3]);
    return !PyErr_Occurred() && fn && a;
  }
  PyObject* call() const {
    int rc;
    const A args = *a;  // another thread may fill in the structure as soon as this one lets go
    Py_BEGIN_ALLOW_THREADS rc = fn(&args, stream);
    Py_END_ALLOW_THREADS return PyLong_FromLong(rc);
  }
};

// An int argument into a C int.
bool get_int(PyObject* o, int* out) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) return false;
  if (v < INT_MIN || v > INT_MAX) {
    PyErr_SetString(PyExc_OverflowError, "argument does not fit an int");
    return false;
  }
  *out = (int)v;
  return true;
}

PyObject* wrong_call() {
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "wrong arguments");
  return nullptr;
}

// (fn, args, stream, dev, max_rows, logits, u, temperature, top_k, top_p, min_p); logits as wide as the vocabulary
PyObject* sample(PyObject*, PyObject* const* v, Py_ssize_t n) {
  Head<cdb_sample_args> h;
  int most;
  if (n != 11 || !h.get(v) || !get_int(v[4], &most)) return wrong_call();
  try {
    cdb_sample_args& a = *h.a;
    if (!input(v[5], h.dev, &a.dtype, &a.rows, most, a.vocab, &a.logits, &a.ld) ||
        THPVariable_Unpack(v[5]).size(1) != a.vocab ||
        !vec(v[6], h.dev, at::kFloat, a.rows, (const void**)&a.u, true) ||
        !vec(v[7], h.dev, at::kFloat, a.rows, (const void**)&a.temperature, true) ||
        !vec(v[8], h.dev, at::kInt, a.rows, (const void**)&a.top_k, false) ||
        !vec(v[9], h.dev, at::kFloat, a.rows, (const void**)&a.top_p, false) ||
        !vec(v[10], h.dev, at::kFloat, a.rows, (const void**)&a.min_p, false))
      Py_RETURN_NONE;
  } catch (...) {  // a tensor without memory
    Py_RETURN_NONE;
  }
  return h.call();
}

// (fn, args, stream, dev, qkv, seq, pos, depth, slot_base, q)
PyObject* cache_write(PyObject*, PyObject* const* v, Py_ssize_t n) {
  Head<cdb_cache_write_args> h;
  if (n != 10 || !h.get(v) || !get_int(v[8], &h.a->slot_base)) return wrong_call();
  try {
    cdb_cache_write_args& a = *h.a;
    const int64_t hd = a.cache.head_dim, width = a.n_heads * hd;
    if (!input(v[4], h.dev, &a.dtype, &a.rows, INT_MAX, width + 2 * a.cache.n_kv_heads * hd, &a.qkv, &a.ldqkv) ||
        !vec(v[5], h.dev, at::kInt, a.rows, (const void**)&a.seq, true) ||
        !vec(v[6], h.dev, at::kInt, a.rows, (const void**)&a.pos, true) ||
        !vec(v[7], h.dev, at::kInt, a.rows, (const void**)&a.depth, false) ||
        !bf16_mat(v[9], h.dev, a.rows, width, (const void**)&a.q, &a.ldq))
      Py_RETURN_NONE;
  } catch (...) {
    Py_RETURN_NONE;
  }
  return h.call();
}

// (fn, args, stream, dev, max_rows, q, seq, pos, depth, slot_base, shared_len, out)
PyObject* attention(PyObject*, PyObject* const* v, Py_ssize_t n) {
  Head<cdb_attention_args> h;
  int most;
  if (n != 12 || !h.get(v) || !get_int(v[4], &most) || !get_int(v[9], &h.a->slot_base) || !get_int(v[10], &h.a->shared_len))
    return wrong_call();
  try {
    cdb_attention_args& a = *h.a;
    const int64_t width = (int64_t)a.n_heads * a.cache.head_dim;
    int dtype;
    if (!input(v[5], h.dev, &dtype, &a.rows, most, width, &a.q, &a.ldq) || dtype != CDB_BF16 ||
        !vec(v[6], h.dev, at::kInt, a.rows, (const void**)&a.seq, true) ||
        !vec(v[7], h.dev, at::kInt, a.rows, (const void**)&a.pos, true) ||
        !vec(v[8], h.dev, at::kInt, a.rows, (const void**)&a.depth, false) ||
        !bf16_mat(v[11], h.dev, a.rows, width, (const void**)&a.out, &a.ldo))
      Py_RETURN_NONE;
  } catch (...) {
    Py_RETURN_NONE;
  }
  return h.call();
}

PyMethodDef kMethods[] = {
    {"sample", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(sample)), METH_FASTCALL, nullptr},
    {"cache_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_write)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "cdb_tensor_calls", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit_cdb_tensor_calls(void) { return PyModule_Create(&kModule); }
