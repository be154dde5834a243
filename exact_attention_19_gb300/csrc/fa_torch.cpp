// fa_torch.cpp -- the usual case of the torch entry points in serving.py (CUDA
// tensors that pass every check, the current stream) without the interpreter:
// checks, outputs from torch's allocator, the current stream and the C-ABI call.
//
// Anything else returns None with nothing done, and the Python code, which holds
// the checks' messages and every other case, takes the call.  A decoding step's
// kernels run for a few microseconds, and attribute lookups, marshalling and
// three allocations from Python took longer than that (fwd_paged: 25 us).
//
// The C functions' addresses come from the loaded libfa_gb300.so (bind), so this
// module links only torch.
#include <Python.h>

#include <cmath>
#include <cstdint>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa.h"

namespace {

decltype(&fa_rope) g_rope = nullptr;
decltype(&fa_kv_append) g_append = nullptr;
decltype(&fa_fwd_paged) g_paged = nullptr;
decltype(&fa_fwd_prefix) g_prefix = nullptr;
decltype(&fa_paged_workspace_bytes) g_bytes = nullptr;

// A CUDA tensor of the given type and number of dimensions, or nullptr.
const at::Tensor* tensor(PyObject* o, at::ScalarType type, int64_t dim) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.scalar_type() == type && t.dim() == dim && t.is_cuda() ? &t : nullptr;
}
const at::Tensor* bf16_4d(PyObject* o) {
  const at::Tensor* t = tensor(o, at::kBFloat16, 4);
  return t && (t->stride(3) == 1 || t->numel() == 0) ? t : nullptr;
}

// Batch, head and row strides; a dimension of size 1 gets one that is valid anywhere.
void strides3(const at::Tensor& t, long long* s) {
  for (int i = 0; i < 3; ++i) s[i] = t.size(i) > 1 ? t.stride(i) : t.size(3);
}

bool same(const at::Tensor& t, int64_t a, int64_t b, int64_t c, int64_t d) {
  return t.size(0) == a && t.size(1) == b && t.size(2) == c && t.size(3) == d;
}

// `o`, or for None a new contiguous tensor, shaped like `like`; an undefined tensor when it does not fit.
at::Tensor output(PyObject* o, const at::Tensor& like) {
  if (o == Py_None) return at::empty(like.sizes(), like.options().memory_format(at::MemoryFormat::Contiguous));
  const at::Tensor* t = bf16_4d(o);
  return t && t->sizes() == like.sizes() ? *t : at::Tensor();
}

bool integer(PyObject* o, long long* v) {
  if (!PyLong_Check(o)) return false;
  int over = 0;
  *v = PyLong_AsLongLongAndOverflow(o, &over);
  return over == 0;
}
bool fits_int(int64_t v) { return v >= INT32_MIN && v <= INT32_MAX; }
// Sizes as the C ABI's ints.
bool ints(const at::Tensor& t) {
  for (int64_t i = 0; i < t.dim(); ++i)
    if (!fits_int(t.size(i))) return false;
  return true;
}
bool number(PyObject* o, double* v) {
  if (!PyFloat_Check(o) && !PyLong_Check(o)) return false;
  *v = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

cudaStream_t stream_of(const at::Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

PyObject* none() { Py_RETURN_NONE; }

PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[5];
  if (n != 5) return none();
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_rope = reinterpret_cast<decltype(g_rope)>(p[0]);
  g_append = reinterpret_cast<decltype(g_append)>(p[1]);
  g_paged = reinterpret_cast<decltype(g_paged)>(p[2]);
  g_prefix = reinterpret_cast<decltype(g_prefix)>(p[3]);
  g_bytes = reinterpret_cast<decltype(g_bytes)>(p[4]);
  return none();
}

// rope(backward, q, k, inv_freq, positions, offset, interleaved, mag, q_out, k_out)
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* q = n == 10 ? bf16_4d(a[1]) : nullptr;
  const at::Tensor* w = q ? tensor(a[3], at::kDouble, 1) : nullptr;
  long long offset = 0;
  double mag = 0;
  if (!w || !w->is_contiguous() || !ints(*q) || !integer(a[5], &offset) || !number(a[7], &mag)) return none();
  const int interleaved = PyObject_IsTrue(a[6]);
  if (interleaved < 0) return nullptr;
  const int64_t B = q->size(0), H = q->size(1), N = q->size(2), d = q->size(3);
  const at::Tensor* k = nullptr;
  if (a[2] != Py_None) {
    k = bf16_4d(a[2]);
    if (!k || !ints(*k) || k->size(1) == 0 || !same(*k, B, k->size(1), N, d)) return none();
  } else if (a[9] != Py_None) {
    return none();
  }
  const int* pos = nullptr;
  long long pos_stride = 0;
  if (a[4] != Py_None) {
    if (!THPVariable_Check(a[4])) return none();
    const at::Tensor& t = THPVariable_Unpack(a[4]);
    const int64_t dim = t.dim();
    if (t.scalar_type() != at::kInt || !t.is_cuda() || dim < 1 || dim > 2 || t.size(dim - 1) != N ||
        (dim == 2 && t.size(0) != B) || (N > 1 && t.stride(dim - 1) != 1))
      return none();
    if (dim == 2 && B > 1) pos_stride = t.stride(0);
    pos = t.const_data_ptr<int>();
  }
  const at::Tensor qo = output(a[8], *q);
  const at::Tensor ko = k ? output(a[9], *k) : at::Tensor();
  if (!qo.defined() || (k && !ko.defined())) return none();
  long long s[12];
  for (long long& x : s) x = d;
  strides3(*q, s);
  strides3(qo, s + 6);
  if (k) {
    strides3(*k, s + 3);
    strides3(ko, s + 9);
  }
  const int st = g_rope(q->const_data_ptr(), k ? k->const_data_ptr() : nullptr, qo.data_ptr(),
                        k ? ko.data_ptr() : nullptr, w->const_data_ptr<double>(), pos, pos_stride, offset, s,
                        static_cast<int>(B), static_cast<int>(H), k ? static_cast<int>(k->size(1)) : 0,
                        static_cast<int>(N), static_cast<int>(d), static_cast<int>(2 * w->size(0)),
                        static_cast<float>(mag), interleaved, a[0] == Py_True ? 1 : 0, stream_of(*q));
  if (st != FA_OK) return none();
  PyObject* const first = a[8] != Py_None ? Py_NewRef(a[8]) : THPVariable_Wrap(qo);
  PyObject* const second = !k ? Py_NewRef(Py_None) : a[9] != Py_None ? Py_NewRef(a[9]) : THPVariable_Wrap(ko);
  PyObject* const r = first && second ? PyTuple_Pack(2, first, second) : nullptr;
  Py_XDECREF(first);
  Py_XDECREF(second);
  return r;
  END_HANDLE_TH_ERRORS
}

// The cache's tensors, checked, with their strides.
struct Cache {
  const at::Tensor *k, *v, *table, *lens;
  const int* fresh = nullptr;
  bool take(PyObject* kc, PyObject* vc, PyObject* tb, PyObject* ln, PyObject* nl, int64_t B, int64_t d, long long* s) {
    k = bf16_4d(kc);
    v = bf16_4d(vc);
    table = tensor(tb, at::kInt, 2);
    lens = tensor(ln, at::kInt, 1);
    if (!k || !v || !table || !lens || !ints(*k) || !ints(*table) || v->sizes() != k->sizes() || k->size(3) != d ||
        table->size(0) != B || !table->is_contiguous() || lens->size(0) != B || !lens->is_contiguous())
      return false;
    if (nl != Py_None) {
      const at::Tensor* t = tensor(nl, at::kInt, 1);
      if (!t || t->size(0) != B || !t->is_contiguous()) return false;
      fresh = t->const_data_ptr<int>();
    }
    strides3(*k, s);
    strides3(*v, s + 3);
    return true;
  }
};

// kv_append(q, k, v, k_cache, v_cache, block_table, seq_lens, inv_freq, new_lens, offset, interleaved, mag, q_out)
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* q = n == 13 ? bf16_4d(a[0]) : nullptr;
  const at::Tensor* k = q ? bf16_4d(a[1]) : nullptr;
  const at::Tensor* v = k ? bf16_4d(a[2]) : nullptr;
  long long offset = 0;
  double mag = 0;
  if (!v || !ints(*q) || !ints(*k) || !integer(a[9], &offset) || !number(a[11], &mag)) return none();
  const int interleaved = PyObject_IsTrue(a[10]);
  if (interleaved < 0) return nullptr;
  const int64_t B = k->size(0), Hk = k->size(1), T = k->size(2), d = k->size(3);
  Cache c;
  long long s[18];
  if (v->sizes() != k->sizes() || q->size(1) == 0 || !same(*q, B, q->size(1), T, d) ||
      !c.take(a[3], a[4], a[5], a[6], a[8], B, d, s + 12) || c.k->size(1) != Hk)
    return none();
  const double* w = nullptr;
  int rot = 0;
  if (a[7] != Py_None) {
    const at::Tensor* t = tensor(a[7], at::kDouble, 1);
    if (!t || !t->is_contiguous()) return none();
    w = t->const_data_ptr<double>();
    rot = static_cast<int>(2 * t->size(0));
  }
  const at::Tensor qo = output(a[12], *q);
  if (!qo.defined()) return none();
  strides3(*q, s);
  strides3(*k, s + 3);
  strides3(*v, s + 6);
  strides3(qo, s + 9);
  const int st = g_append(q->const_data_ptr(), k->const_data_ptr(), v->const_data_ptr(), qo.data_ptr(),
                          c.k->data_ptr(), c.v->data_ptr(), w, c.table->const_data_ptr<int>(),
                          c.lens->const_data_ptr<int>(), c.fresh, s, static_cast<int>(B),
                          static_cast<int>(q->size(1)), static_cast<int>(Hk), static_cast<int>(T), static_cast<int>(d),
                          rot, static_cast<int>(c.k->size(0)), static_cast<int>(c.k->size(2)),
                          static_cast<int>(c.table->size(1)), offset, static_cast<float>(mag), interleaved,
                          stream_of(*k));
  if (st != FA_OK) return none();
  return a[12] != Py_None ? Py_NewRef(a[12]) : THPVariable_Wrap(qo);
  END_HANDLE_TH_ERRORS
}

// paged(q, k_cache, v_cache, prefix_pages, prefix_len, block_table, seq_lens, scale, new_lens, left, right, out, lse,
//       workspace)
PyObject* py_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* q = n == 14 ? bf16_4d(a[0]) : nullptr;
  long long prefix = 0, left = 0, right = 0;
  if (!q || !q->is_contiguous() || !ints(*q) || !integer(a[4], &prefix) || !integer(a[9], &left) ||
      !integer(a[10], &right) || !fits_int(prefix) || !fits_int(left) || !fits_int(right))
    return none();
  const int B = static_cast<int>(q->size(0)), H = static_cast<int>(q->size(1)), T = static_cast<int>(q->size(2)),
            d = static_cast<int>(q->size(3));
  Cache c;
  long long s[6];
  if (!c.take(a[1], a[2], a[5], a[6], a[8], B, d, s)) return none();
  const int Hk = static_cast<int>(c.k->size(1)), page = static_cast<int>(c.k->size(2));
  if (Hk == 0 || H % Hk != 0) return none();
  const int* pages = nullptr;
  if (a[3] != Py_None) {
    const at::Tensor* t = tensor(a[3], at::kInt, 1);
    if (!t || !t->is_contiguous() || prefix <= 0 || t->size(0) * page < prefix) return none();
    pages = t->const_data_ptr<int>();
  }
  double scale = 1.0 / std::sqrt(static_cast<double>(d));
  if (a[7] != Py_None && !number(a[7], &scale)) return none();
  at::Tensor out, lse, ws;
  if (a[11] == Py_None) {
    out = at::empty(q->sizes(), q->options());
  } else {
    const at::Tensor* t = bf16_4d(a[11]);
    if (!t || t->sizes() != q->sizes() || !t->is_contiguous()) return none();
    out = *t;
  }
  if (a[12] == Py_None) {
    lse = at::empty({B, H, T}, q->options().dtype(at::kFloat));
  } else {
    const at::Tensor* t = tensor(a[12], at::kFloat, 3);
    if (!t || t->size(0) != B || t->size(1) != H || t->size(2) != T || !t->is_contiguous()) return none();
    lse = *t;
  }
  size_t bytes = 0;
  if (a[13] == Py_None) {
    bytes = g_bytes(B, H, Hk, T, d, pages ? static_cast<int>(prefix) : 0);
    ws = at::empty({static_cast<int64_t>(bytes)}, q->options().dtype(at::kByte));
  } else {
    if (!THPVariable_Check(a[13])) return none();
    ws = THPVariable_Unpack(a[13]);
    if (!ws.is_cuda() || !ws.is_contiguous()) return none();
    bytes = ws.nbytes();
  }
  const int n_pages = static_cast<int>(c.k->size(0)), max_pages = static_cast<int>(c.table->size(1));
  const int st =
      pages ? g_prefix(q->const_data_ptr(), c.k->const_data_ptr(), c.v->const_data_ptr(), out.data_ptr(),
                       lse.data_ptr<float>(), pages, static_cast<int>(prefix), c.table->const_data_ptr<int>(),
                       c.lens->const_data_ptr<int>(), c.fresh, s, B, H, Hk, T, d, n_pages, page, max_pages,
                       static_cast<float>(scale), ws.data_ptr(), bytes, stream_of(*q))
            : g_paged(q->const_data_ptr(), c.k->const_data_ptr(), c.v->const_data_ptr(), out.data_ptr(),
                      lse.data_ptr<float>(), c.table->const_data_ptr<int>(), c.lens->const_data_ptr<int>(), c.fresh, s,
                      B, H, Hk, T, d, n_pages, page, max_pages, static_cast<float>(scale), static_cast<int>(left),
                      static_cast<int>(right), ws.data_ptr(), bytes, stream_of(*q));
  if (st != FA_OK) return none();
  PyObject* const first = a[11] != Py_None ? Py_NewRef(a[11]) : THPVariable_Wrap(out);
  PyObject* const second = a[12] != Py_None ? Py_NewRef(a[12]) : THPVariable_Wrap(lse);
  PyObject* const r = first && second ? PyTuple_Pack(2, first, second) : nullptr;
  Py_XDECREF(first);
  Py_XDECREF(second);
  return r;
  END_HANDLE_TH_ERRORS
}

#define FA_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef g_methods[] = {{"bind", FA_FAST(py_bind)},
                           {"rope", FA_FAST(py_rope)},
                           {"kv_append", FA_FAST(py_append)},
                           {"paged", FA_FAST(py_paged)},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "fa_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fa_torch(void) { return PyModule_Create(&g_module); }
