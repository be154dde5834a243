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
decltype(&fa_norm_rope) g_norm = nullptr;
decltype(&fa_norm_rope_bwd) g_norm_bwd = nullptr;
decltype(&fa_norm_bwd_workspace_bytes) g_norm_bytes = nullptr;
decltype(&fa_kv_append_norm) g_append_norm = nullptr;
decltype(&fa_kv_weights) g_weights = nullptr;
decltype(&fa_kv_evict) g_evict = nullptr;
decltype(&fa_evict_workspace_bytes) g_evict_bytes = nullptr;

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
  constexpr int kFunctions = 12;
  void* p[kFunctions];
  if (n != kFunctions) return none();
  for (int i = 0; i < kFunctions; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_rope = reinterpret_cast<decltype(g_rope)>(p[0]);
  g_append = reinterpret_cast<decltype(g_append)>(p[1]);
  g_paged = reinterpret_cast<decltype(g_paged)>(p[2]);
  g_prefix = reinterpret_cast<decltype(g_prefix)>(p[3]);
  g_bytes = reinterpret_cast<decltype(g_bytes)>(p[4]);
  g_norm = reinterpret_cast<decltype(g_norm)>(p[5]);
  g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(p[6]);
  g_norm_bytes = reinterpret_cast<decltype(g_norm_bytes)>(p[7]);
  g_append_norm = reinterpret_cast<decltype(g_append_norm)>(p[8]);
  g_weights = reinterpret_cast<decltype(g_weights)>(p[9]);
  g_evict = reinterpret_cast<decltype(g_evict)>(p[10]);
  g_evict_bytes = reinterpret_cast<decltype(g_evict_bytes)>(p[11]);
  return none();
}

// Positions [B, N] or [N], or None: their pointer and the stride from one sequence to the next.
bool positions_of(PyObject* o, int64_t B, int64_t N, const int** pos, long long* stride) {
  *pos = nullptr;
  *stride = 0;
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  const int64_t dim = t.dim();
  if (t.scalar_type() != at::kInt || !t.is_cuda() || dim < 1 || dim > 2 || t.size(dim - 1) != N ||
      (dim == 2 && t.size(0) != B) || (N > 1 && t.stride(dim - 1) != 1))
    return false;
  if (dim == 2 && B > 1) *stride = t.stride(0);
  *pos = t.const_data_ptr<int>();
  return true;
}

// Frequencies [rot / 2], or None where that is allowed.
bool frequencies(PyObject* o, bool optional, const double** w, int* rot) {
  *w = nullptr;
  *rot = 0;
  if (optional && o == Py_None) return true;
  const at::Tensor* t = tensor(o, at::kDouble, 1);
  if (!t || !t->is_contiguous() || !fits_int(2 * t->size(0))) return false;
  *w = t->const_data_ptr<double>();
  *rot = static_cast<int>(2 * t->size(0));
  return true;
}

// The weights of a norm, [d] in bf16 or fp32 alike, or None each.
struct Norm {
  const void* w[2] = {nullptr, nullptr};
  int f32 = 0;
  double eps = 0;
  bool take(PyObject* q, PyObject* k, PyObject* e, int64_t d) {
    int known = -1;
    PyObject* const o[2] = {q, k};
    for (int i = 0; i < 2; ++i) {
      if (o[i] == Py_None) continue;
      if (!THPVariable_Check(o[i])) return false;
      const at::Tensor& t = THPVariable_Unpack(o[i]);
      const int type = t.scalar_type() == at::kFloat ? 1 : (t.scalar_type() == at::kBFloat16 ? 0 : -1);
      if (type < 0 || (known >= 0 && known != type) || !t.is_cuda() || t.dim() != 1 || t.size(0) != d ||
          !t.is_contiguous())
        return false;
      f32 = known = type;
      w[i] = t.const_data_ptr();
    }
    return number(e, &eps);
  }
};

// What a call returns: the tensor that the caller gave, or the new one; None for none.
PyObject* given_or(PyObject* o, const at::Tensor& t) {
  return o != Py_None ? Py_NewRef(o) : t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
}
template <int N>
PyObject* tuple(PyObject* const (&o)[N]) {
  PyObject* r = PyTuple_New(N);
  for (int i = 0; i < N; ++i)
    if (!o[i]) Py_CLEAR(r);
  for (int i = 0; i < N; ++i) {
    if (r) PyTuple_SET_ITEM(r, i, o[i]);
    else Py_XDECREF(o[i]);
  }
  return r;
}

// rope(backward, q, k, inv_freq, positions, offset, interleaved, mag, q_out, k_out)
// norm_rope(q, k, inv_freq, q_weight, k_weight, eps, positions, offset, interleaved, mag, q_out, k_out)
PyObject* rope_call(PyObject* oq, PyObject* ok, PyObject* ow, PyObject* const* a, bool backward, PyObject* const* nw) {
  const at::Tensor* q = bf16_4d(oq);
  const double* w = nullptr;
  int rot = 0;
  long long offset = 0;
  double mag = 0;
  if (!q || !frequencies(ow, nw != nullptr, &w, &rot) || !ints(*q) || !integer(a[1], &offset) || !number(a[3], &mag))
    return none();
  const int interleaved = PyObject_IsTrue(a[2]);
  if (interleaved < 0) return nullptr;
  const int64_t B = q->size(0), H = q->size(1), N = q->size(2), d = q->size(3);
  const at::Tensor* k = nullptr;
  if (ok != Py_None) {
    k = bf16_4d(ok);
    if (!k || !ints(*k) || k->size(1) == 0 || !same(*k, B, k->size(1), N, d)) return none();
  } else if (a[5] != Py_None) {
    return none();
  }
  Norm norm;
  if (nw && !norm.take(nw[0], nw[1], nw[2], d)) return none();
  const int* pos = nullptr;
  long long pos_stride = 0;
  if (!positions_of(a[0], B, N, &pos, &pos_stride)) return none();
  const at::Tensor qo = output(a[4], *q);
  const at::Tensor ko = k ? output(a[5], *k) : at::Tensor();
  if (!qo.defined() || (k && !ko.defined())) return none();
  long long s[12];
  for (long long& x : s) x = d;
  strides3(*q, s);
  strides3(qo, s + 6);
  if (k) {
    strides3(*k, s + 3);
    strides3(ko, s + 9);
  }
  const void *qp = q->const_data_ptr(), *kp = k ? k->const_data_ptr() : nullptr;
  void *qop = qo.data_ptr(), *kop = k ? ko.data_ptr() : nullptr;
  const int b = static_cast<int>(B), h = static_cast<int>(H), hk = k ? static_cast<int>(k->size(1)) : 0,
            rows = static_cast<int>(N), dd = static_cast<int>(d);
  const float m = static_cast<float>(mag);
  const cudaStream_t stream = stream_of(*q);
  const int st = nw ? g_norm(qp, kp, qop, kop, w, norm.w[0], norm.w[1], pos, pos_stride, offset, s, b, h, hk, rows, dd,
                             rot, m, interleaved, static_cast<float>(norm.eps), norm.f32, stream)
                    : g_rope(qp, kp, qop, kop, w, pos, pos_stride, offset, s, b, h, hk, rows, dd, rot, m, interleaved,
                             backward ? 1 : 0, stream);
  if (st != FA_OK) return none();
  return tuple<2>({given_or(a[4], qo), given_or(a[5], ko)});
}
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return n == 10 ? rope_call(a[1], a[2], a[3], a + 4, a[0] == Py_True, nullptr) : none();
  END_HANDLE_TH_ERRORS
}
PyObject* py_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return n == 12 ? rope_call(a[0], a[1], a[2], a + 6, false, a + 3) : none();
  END_HANDLE_TH_ERRORS
}

// norm_rope_bwd(dq, dk, q, k, inv_freq, q_weight, k_weight, eps, positions, offset, interleaved, mag, q_out, k_out,
//               workspace)
PyObject* py_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* dq = n == 15 ? bf16_4d(a[0]) : nullptr;
  const at::Tensor* q = dq ? bf16_4d(a[2]) : nullptr;
  const double* w = nullptr;
  int rot = 0;
  long long offset = 0;
  double mag = 0;
  if (!q || !ints(*q) || dq->sizes() != q->sizes() || !frequencies(a[4], true, &w, &rot) || !integer(a[9], &offset) ||
      !number(a[11], &mag))
    return none();
  const int interleaved = PyObject_IsTrue(a[10]);
  if (interleaved < 0) return nullptr;
  const int64_t B = q->size(0), H = q->size(1), N = q->size(2), d = q->size(3);
  const at::Tensor *k = nullptr, *dk = nullptr;
  if (a[3] != Py_None) {
    k = bf16_4d(a[3]);
    dk = bf16_4d(a[1]);
    if (!k || !dk || !ints(*k) || k->size(1) == 0 || !same(*k, B, k->size(1), N, d) || dk->sizes() != k->sizes())
      return none();
  } else if (a[1] != Py_None || a[13] != Py_None || a[6] != Py_None) {
    return none();
  }
  Norm norm;
  const int* pos = nullptr;
  long long pos_stride = 0;
  if (!norm.take(a[5], a[6], a[7], d) || !positions_of(a[8], B, N, &pos, &pos_stride)) return none();
  const at::Tensor qo = output(a[12], *q);
  const at::Tensor ko = k ? output(a[13], *k) : at::Tensor();
  if (!qo.defined() || (k && !ko.defined())) return none();
  at::Tensor dw[2], ws;
  for (int i = 0; i < 2; ++i)
    if (norm.w[i]) dw[i] = at::empty({d}, q->options().dtype(at::kFloat));
  size_t bytes = 0;
  if (norm.w[0] || norm.w[1]) {
    if (a[14] == Py_None) {
      bytes = g_norm_bytes(static_cast<int>(d));
      ws = at::empty({static_cast<int64_t>(bytes)}, q->options().dtype(at::kByte));
    } else {
      if (!THPVariable_Check(a[14])) return none();
      ws = THPVariable_Unpack(a[14]);
      if (!ws.is_cuda() || !ws.is_contiguous()) return none();
      bytes = ws.nbytes();
    }
  }
  long long s[18];
  for (long long& x : s) x = d;
  strides3(*dq, s);
  strides3(*q, s + 6);
  strides3(qo, s + 12);
  if (k) {
    strides3(*dk, s + 3);
    strides3(*k, s + 9);
    strides3(ko, s + 15);
  }
  const int st = g_norm_bwd(
      dq->const_data_ptr(), k ? dk->const_data_ptr() : nullptr, q->const_data_ptr(), k ? k->const_data_ptr() : nullptr,
      qo.data_ptr(), k ? ko.data_ptr() : nullptr, norm.w[0] ? dw[0].data_ptr<float>() : nullptr,
      norm.w[1] ? dw[1].data_ptr<float>() : nullptr, w, norm.w[0], norm.w[1], pos, pos_stride, offset, s,
      static_cast<int>(B), static_cast<int>(H), k ? static_cast<int>(k->size(1)) : 0, static_cast<int>(N),
      static_cast<int>(d), rot, static_cast<float>(mag), interleaved, static_cast<float>(norm.eps), norm.f32,
      ws.defined() ? ws.data_ptr() : nullptr, bytes, stream_of(*q));
  if (st != FA_OK) return none();
  return tuple<4>({given_or(a[12], qo), given_or(a[13], ko), given_or(Py_None, dw[0]), given_or(Py_None, dw[1])});
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
// kv_append_norm(the same, eps, q_weight, k_weight, shift)
PyObject* append_call(PyObject* const* a, PyObject* const* nw) {
  const at::Tensor* q = bf16_4d(a[0]);
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
  if (!frequencies(a[7], true, &w, &rot)) return none();
  Norm norm;
  const int* shift = nullptr;
  if (nw && nw[0] != Py_None && !norm.take(nw[1], nw[2], nw[0], d)) return none();
  if (nw && nw[0] == Py_None && (nw[1] != Py_None || nw[2] != Py_None)) return none();
  if (nw && nw[3] != Py_None) {
    const at::Tensor* t = tensor(nw[3], at::kInt, 1);
    if (!t || t->size(0) != B || !t->is_contiguous()) return none();
    shift = t->const_data_ptr<int>();
  }
  const at::Tensor qo = output(a[12], *q);
  if (!qo.defined()) return none();
  strides3(*q, s);
  strides3(*k, s + 3);
  strides3(*v, s + 6);
  strides3(qo, s + 9);
  const void *qp = q->const_data_ptr(), *kp = k->const_data_ptr(), *vp = v->const_data_ptr();
  void *qop = qo.data_ptr(), *kc = c.k->data_ptr(), *vc = c.v->data_ptr();
  const int *table = c.table->const_data_ptr<int>(), *lens = c.lens->const_data_ptr<int>();
  const int b = static_cast<int>(B), h = static_cast<int>(q->size(1)), hk = static_cast<int>(Hk),
            rows = static_cast<int>(T), dd = static_cast<int>(d), pages = static_cast<int>(c.k->size(0)),
            page = static_cast<int>(c.k->size(2)), max_pages = static_cast<int>(c.table->size(1));
  const float m = static_cast<float>(mag);
  const cudaStream_t stream = stream_of(*k);
  const int st = nw ? g_append_norm(qp, kp, vp, qop, kc, vc, w, norm.w[0], norm.w[1], table, lens, c.fresh, shift, s, b,
                                    h, hk, rows, dd, rot, pages, page, max_pages, offset, m, interleaved,
                                    nw[0] != Py_None ? 1 : 0, static_cast<float>(norm.eps), norm.f32, stream)
                    : g_append(qp, kp, vp, qop, kc, vc, w, table, lens, c.fresh, s, b, h, hk, rows, dd, rot, pages, page,
                               max_pages, offset, m, interleaved, stream);
  return st == FA_OK ? given_or(a[12], qo) : none();
}
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return n == 13 ? append_call(a, nullptr) : none();
  END_HANDLE_TH_ERRORS
}
PyObject* py_append_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return n == 17 ? append_call(a, a + 13) : none();
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
  return tuple<2>({given_or(a[11], out), given_or(a[12], lse)});
  END_HANDLE_TH_ERRORS
}

// The weights beside a cache: fp32 [n_pages, Hk, page], with their page and head strides.
const at::Tensor* key_weights(PyObject* o, const at::Tensor& cache, long long* s) {
  const at::Tensor* t = tensor(o, at::kFloat, 3);
  if (!t || t->size(0) != cache.size(0) || t->size(1) != cache.size(1) || t->size(2) != cache.size(2) ||
      (t->stride(2) != 1 && t->numel() != 0))
    return nullptr;
  for (int i = 0; i < 2; ++i) s[i] = t->size(i) > 1 ? t->stride(i) : t->size(2);
  return t;
}
const at::Tensor* ints_of(PyObject* o, int64_t B) {
  const at::Tensor* t = tensor(o, at::kInt, 1);
  return t && t->size(0) == B && t->is_contiguous() ? t : nullptr;
}

// kv_weights(q, lse, k_cache, weights, block_table, seq_lens, scale, new_lens, left, right, decay)
PyObject* py_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* q = n == 11 ? bf16_4d(a[0]) : nullptr;
  const at::Tensor* lse = q ? tensor(a[1], at::kFloat, 3) : nullptr;
  long long left = 0, right = 0;
  double decay = 0;
  if (!lse || !q->is_contiguous() || !ints(*q) || !lse->is_contiguous() || !integer(a[8], &left) ||
      !integer(a[9], &right) || !fits_int(left) || !fits_int(right) || !number(a[10], &decay))
    return none();
  const int B = static_cast<int>(q->size(0)), H = static_cast<int>(q->size(1)), T = static_cast<int>(q->size(2)),
            d = static_cast<int>(q->size(3));
  if (lse->size(0) != B || lse->size(1) != H || lse->size(2) != T) return none();
  Cache c;
  long long s[6], ws[2];
  if (!c.take(a[2], a[2], a[4], a[5], a[7], B, d, s)) return none();
  const at::Tensor* w = key_weights(a[3], *c.k, ws);
  const int Hk = static_cast<int>(c.k->size(1));
  if (!w || Hk == 0 || H % Hk != 0) return none();
  double scale = 1.0 / std::sqrt(static_cast<double>(d));
  if (a[6] != Py_None && !number(a[6], &scale)) return none();
  s[3] = ws[0];
  s[4] = ws[1];
  const int st = g_weights(q->const_data_ptr(), lse->const_data_ptr<float>(), c.k->const_data_ptr(),
                           w->data_ptr<float>(), c.table->const_data_ptr<int>(), c.lens->const_data_ptr<int>(), c.fresh,
                           s, B, H, Hk, T, d, static_cast<int>(c.k->size(0)), static_cast<int>(c.k->size(2)),
                           static_cast<int>(c.table->size(1)), static_cast<float>(scale), static_cast<int>(left),
                           static_cast<int>(right), static_cast<float>(decay), stream_of(*q));
  return st == FA_OK ? Py_NewRef(a[3]) : none();
  END_HANDLE_TH_ERRORS
}

// kv_evict(k_cache, v_cache, weights, block_table, seq_lens, budget, recent, sinks, slack, table_out, lens_out, shift,
//          kept, workspace)
PyObject* py_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor* k = n == 14 ? bf16_4d(a[0]) : nullptr;
  const at::Tensor* lens = k ? tensor(a[4], at::kInt, 1) : nullptr;
  if (!lens || !ints(*lens)) return none();
  long long v[4];
  for (int i = 0; i < 4; ++i)
    if (!integer(a[5 + i], v + i) || v[i] < 0 || !fits_int(v[i])) return none();
  const int64_t most = v[0] + v[3], B = lens->size(0);
  if (v[0] < 1 || v[1] + v[2] > v[0] || !fits_int(most)) return none();
  Cache c;
  long long s[8];
  if (!c.take(a[0], a[1], a[3], a[4], Py_None, B, k->size(3), s)) return none();
  const at::Tensor* w = key_weights(a[2], *k, s + 6);
  if (!w) return none();
  const int64_t Hk = k->size(1);
  const int* to = nullptr;
  int out_pages = 0;
  if (a[9] != Py_None) {
    const at::Tensor* t = tensor(a[9], at::kInt, 2);
    if (!t || !ints(*t) || t->size(0) != B || !t->is_contiguous() || t->size(1) * k->size(2) < most) return none();
    to = t->const_data_ptr<int>();
    out_pages = static_cast<int>(t->size(1));
  }
  at::Tensor lens_out, kept, ws;
  if (a[10] == Py_None) {
    lens_out = at::empty({B}, lens->options());
  } else {
    const at::Tensor* t = ints_of(a[10], B);
    if (!t) return none();
    lens_out = *t;
  }
  int* shift = nullptr;
  if (a[11] != Py_None) {
    const at::Tensor* t = ints_of(a[11], B);
    if (!t) return none();
    shift = t->data_ptr<int>();
  }
  if (a[12] == Py_None) {
    kept = at::empty({B, Hk, most}, lens->options());
  } else {
    const at::Tensor* t = tensor(a[12], at::kInt, 3);
    if (!t || t->size(0) != B || t->size(1) != Hk || t->size(2) != most || !t->is_contiguous()) return none();
    kept = *t;
  }
  size_t bytes = 0;
  if (a[13] == Py_None) {
    bytes = g_evict_bytes(static_cast<int>(B), static_cast<int>(Hk));
    ws = at::empty({static_cast<int64_t>(bytes)}, lens->options().dtype(at::kByte));
  } else {
    if (!THPVariable_Check(a[13])) return none();
    ws = THPVariable_Unpack(a[13]);
    if (!ws.is_cuda() || !ws.is_contiguous()) return none();
    bytes = ws.nbytes();
  }
  const int st = g_evict(k->data_ptr(), c.v->data_ptr(), w->data_ptr<float>(), c.table->const_data_ptr<int>(), to,
                         out_pages, lens->const_data_ptr<int>(), lens_out.data_ptr<int>(), shift, kept.data_ptr<int>(), s,
                         static_cast<int>(B), static_cast<int>(Hk), static_cast<int>(k->size(3)),
                         static_cast<int>(k->size(0)), static_cast<int>(k->size(2)), static_cast<int>(c.table->size(1)),
                         static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]), static_cast<int>(v[3]),
                         ws.data_ptr(), bytes, stream_of(*k));
  if (st != FA_OK) return none();
  return tuple<2>({given_or(a[10], lens_out), given_or(a[12], kept)});
  END_HANDLE_TH_ERRORS
}

#define FA_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef g_methods[] = {{"bind", FA_FAST(py_bind)},
                           {"rope", FA_FAST(py_rope)},
                           {"norm_rope", FA_FAST(py_norm_rope)},
                           {"norm_rope_bwd", FA_FAST(py_norm_bwd)},
                           {"kv_append", FA_FAST(py_append)},
                           {"kv_append_norm", FA_FAST(py_append_norm)},
                           {"paged", FA_FAST(py_paged)},
                           {"kv_weights", FA_FAST(py_weights)},
                           {"kv_evict", FA_FAST(py_evict)},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "fa_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fa_torch(void) { return PyModule_Create(&g_module); }
