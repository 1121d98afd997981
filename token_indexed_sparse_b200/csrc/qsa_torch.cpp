// Short way from PyTorch tensors to the paged-cache calls of include/qsa.h.
//
// A decode step's kernels take a few microseconds and the same calls marshalled
// in Python take fifteen, so this module does what qsa.py does for arguments
// that need nothing done to them: exact tensors of the right types, shapes and
// layouts on one CUDA device.  For anything else it returns NotImplemented without
// having done anything, and qsa.py goes its own way, which converts or raises.
// A call returns the outputs, or the library's status as an int when it is not
// QSA_OK.  The library's entry points come from qsa.py (bind), so both always
// use the one library that is loaded.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "qsa.h"

namespace {

decltype(&qsa_rope) p_rope = nullptr;
decltype(&qsa_cache_append) p_append = nullptr;
decltype(&qsa_paged_forward) p_forward = nullptr;
decltype(&qsa_paged_forward_workspace_size) p_forward_size = nullptr;
decltype(&qsa_paged_causal) p_causal = nullptr;
decltype(&qsa_paged_causal_workspace_size) p_causal_size = nullptr;

PyObject* not_mine() { Py_RETURN_NOTIMPLEMENTED; }

// The tensor of an argument, or null (an undefined one for None where that is allowed).
const at::Tensor* tensor(PyObject* x, bool none_too = false) {
  static const at::Tensor none;
  if (none_too && x == Py_None) return &none;
  return THPVariable_CheckExact(x) ? &THPVariable_Unpack(x) : nullptr;
}

// All on CUDA device `index` (undefined ones aside).
template <typename... Ts>
bool on(int index, const Ts*... ts) {
  return ((!ts->defined() || (ts->is_cuda() && ts->get_device() == index)) && ...);
}

struct Rows {  // a [T, heads, 256] BF16 operand
  void* p = nullptr;
  int64_t ts = 0, hs = 0;
};
bool rows(const at::Tensor& x, int64_t T, Rows* r) {
  if (x.scalar_type() != at::kBFloat16 || x.dim() != 3 || x.size(2) != 256 || x.stride(2) != 1 || x.size(0) != T)
    return false;
  *r = {x.data_ptr(), T > 1 ? x.stride(0) : 0, x.size(1) > 1 ? x.stride(1) : 0};
  return true;
}
bool vec(const at::Tensor& x, int64_t n, at::ScalarType type) {
  return x.scalar_type() == type && x.dim() == 1 && x.size(0) == n && x.is_contiguous();
}

struct Cache {
  int64_t B, n_pages, page, max_pages, G;
};
bool cache(const at::Tensor& kp, const at::Tensor& vp, const at::Tensor& table, const at::Tensor& kv_len,
           const at::Tensor& cu_q, Cache* c) {
  if (kp.scalar_type() != at::kBFloat16 || vp.scalar_type() != at::kBFloat16 || kp.dim() != 4 || kp.size(3) != 256 ||
      kp.sizes() != vp.sizes() || !kp.is_contiguous() || !vp.is_contiguous() || table.scalar_type() != at::kInt ||
      table.dim() != 2 || !table.is_contiguous())
    return false;
  *c = {table.size(0), kp.size(0), kp.size(1), table.size(1), kp.size(2)};
  return c->B < INT32_MAX && c->page <= INT32_MAX && c->G <= INT32_MAX / 12 && vec(kv_len, c->B, at::kInt) &&
         vec(cu_q, c->B + 1, at::kInt);
}

template <typename T>
T* ptr(const at::Tensor& x) {
  return x.defined() ? static_cast<T*>(x.data_ptr()) : nullptr;
}

// Runs f(stream) with the device current.
template <class F>
int enqueue(int index, F f) {
  const auto stream = reinterpret_cast<qsa_stream_t>(c10::cuda::getCurrentCUDAStream(index).stream());
  if (c10::cuda::current_device() == index) return f(stream);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  return f(stream);
}

at::Tensor bytes_like(const at::Tensor& q, size_t n) {
  return at::empty({static_cast<int64_t>(n < 256 ? 256 : n)}, q.options().dtype(at::kByte));
}

// rope(q, k | None, positions, inv_freq, interleaved, mscale, out_q | None, out_k | None, backward)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9 || !p_rope) return not_mine();
  const at::Tensor *q = tensor(a[0]), *k = tensor(a[1], true), *pos = tensor(a[2]), *f = tensor(a[3]),
                   *oq = tensor(a[6], true), *ok = tensor(a[7], true);
  if (!q || !k || !pos || !f || !oq || !ok || !q->is_cuda() || q->dim() != 3) return not_mine();
  const int64_t T = q->size(0), H = q->size(1), G = k->defined() && k->dim() == 3 ? k->size(1) : 0;
  const int inter = PyObject_IsTrue(a[4]), backward = PyObject_IsTrue(a[8]);
  const double m = PyFloat_AsDouble(a[5]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return not_mine();
  }
  const int dev = q->get_device();
  Rows rq, rk, roq, rok;
  if (!rows(*q, T, &rq) || (k->defined() ? !rows(*k, T, &rk) : ok->defined()) || !vec(*pos, T, at::kInt) ||
      !vec(*f, f->dim() == 1 ? f->size(0) : -1, at::kDouble) || H > INT32_MAX || G > INT32_MAX || f->size(0) > 128 ||
      !on(dev, k, pos, f, oq, ok) || (oq->defined() && oq->sizes() != q->sizes()) ||
      (ok->defined() && ok->sizes() != k->sizes()))
    return not_mine();
  const at::Tensor yq = oq->defined() ? *oq : at::empty_like(*q);
  const at::Tensor yk = !k->defined() || ok->defined() ? *ok : at::empty_like(*k);
  if (!rows(yq, T, &roq) || (k->defined() && !rows(yk, T, &rok))) return not_mine();
  const int st = enqueue(dev, [&](qsa_stream_t s) {
    return p_rope(rq.p, rq.ts, rq.hs, rk.p, rk.ts, rk.hs, roq.p, roq.ts, roq.hs, rok.p, rok.ts, rok.hs,
                  ptr<int32_t>(*pos), ptr<double>(*f), T, static_cast<int>(H), static_cast<int>(G),
                  static_cast<int>(2 * f->size(0)), inter, static_cast<float>(m), backward, s);
  });
  if (st != QSA_OK) return PyLong_FromLong(st);
  PyObject* pair = PyTuple_New(2);
  if (!pair) return nullptr;
  PyTuple_SET_ITEM(pair, 0, oq->defined() ? Py_NewRef(a[6]) : THPVariable_Wrap(yq));
  PyTuple_SET_ITEM(pair, 1, yk.defined() ? (ok->defined() ? Py_NewRef(a[7]) : THPVariable_Wrap(yk)) : Py_NewRef(Py_None));
  return pair;
  END_HANDLE_TH_ERRORS
}

// cache_append(k_new, v_new, k_pages, v_pages, block_table, kv_len, cu_q, q | None, inv_freq | None, interleaved,
//              mscale, out_q | None): out_q, or None without q
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12 || !p_append) return not_mine();
  const at::Tensor *kn = tensor(a[0]), *vn = tensor(a[1]), *kp = tensor(a[2]), *vp = tensor(a[3]), *tb = tensor(a[4]),
                   *len = tensor(a[5]), *cu = tensor(a[6]), *q = tensor(a[7], true), *f = tensor(a[8], true),
                   *oq = tensor(a[11], true);
  if (!kn || !vn || !kp || !vp || !tb || !len || !cu || !q || !f || !oq || !kn->is_cuda() || kn->dim() != 3)
    return not_mine();
  const int inter = PyObject_IsTrue(a[9]);
  const double m = PyFloat_AsDouble(a[10]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return not_mine();
  }
  const int64_t T = kn->size(0);
  const int dev = kn->get_device();
  Cache c;
  Rows rk, rv, rq, ro;
  if (!cache(*kp, *vp, *tb, *len, *cu, &c) || !rows(*kn, T, &rk) || !rows(*vn, T, &rv) || kn->size(1) != c.G ||
      vn->size(1) != c.G || !on(dev, vn, kp, vp, tb, len, cu, q, f, oq) || (oq->defined() && !q->defined()) ||
      (q->defined() && (!f->defined() || !rows(*q, T, &rq))) || (oq->defined() && oq->sizes() != q->sizes()) ||
      (f->defined() && (!vec(*f, f->dim() == 1 ? f->size(0) : -1, at::kDouble) || f->size(0) > 128)))
    return not_mine();
  const int64_t H = q->defined() ? q->size(1) : 12 * c.G;
  if (H > INT32_MAX) return not_mine();
  const at::Tensor y = !q->defined() || oq->defined() ? *oq : at::empty_like(*q);
  if (q->defined() && !rows(y, T, &ro)) return not_mine();
  const int st = enqueue(dev, [&](qsa_stream_t s) {
    return p_append(rk.p, rk.ts, rk.hs, rv.p, rv.ts, rv.hs, rq.p, rq.ts, rq.hs, ro.p, ro.ts, ro.hs, ptr<double>(*f),
                    f->defined() ? static_cast<int>(2 * f->size(0)) : 0, inter, static_cast<float>(m), kp->data_ptr(),
                    vp->data_ptr(), ptr<int32_t>(*tb), ptr<int32_t>(*len), ptr<int32_t>(*cu), T,
                    static_cast<int>(c.B), c.n_pages, static_cast<int>(c.page), c.max_pages, static_cast<int>(H),
                    static_cast<int>(c.G), s);
  });
  if (st != QSA_OK) return PyLong_FromLong(st);
  if (!q->defined()) Py_RETURN_NONE;
  return oq->defined() ? Py_NewRef(a[11]) : THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// What both attentions take and give.
struct Attention {
  const at::Tensor *q, *kp, *vp, *tb, *len, *cu, *out, *lse, *ws;
  at::Tensor y, l, w;
  int64_t T, H;
  int dev;
  Cache c;
  bool take(PyObject* q_, PyObject* kp_, PyObject* vp_, PyObject* tb_, PyObject* len_, PyObject* cu_, PyObject* out_,
            PyObject* lse_, PyObject* ws_) {
    q = tensor(q_), kp = tensor(kp_), vp = tensor(vp_), tb = tensor(tb_), len = tensor(len_), cu = tensor(cu_);
    out = tensor(out_, true), lse = tensor(lse_, true), ws = tensor(ws_, true);
    if (!q || !kp || !vp || !tb || !len || !cu || !out || !lse || !ws || !q->is_cuda() || q->dim() != 3 ||
        q->scalar_type() != at::kBFloat16 || q->size(2) != 256 || !q->is_contiguous())
      return false;
    T = q->size(0), H = q->size(1), dev = q->get_device();
    return H <= INT32_MAX && on(dev, kp, vp, tb, len, cu, out, lse, ws) && cache(*kp, *vp, *tb, *len, *cu, &c) &&
           (!out->defined() ||
            (out->scalar_type() == at::kBFloat16 && out->sizes() == q->sizes() && out->is_contiguous())) &&
           (!lse->defined() || (lse->scalar_type() == at::kFloat && lse->dim() == 2 && lse->size(0) == T &&
                                lse->size(1) == H && lse->is_contiguous())) &&
           (!ws->defined() || (ws->scalar_type() == at::kByte && ws->is_contiguous()));
  }
  void make(size_t ws_bytes) {
    y = out->defined() ? *out : at::empty_like(*q);
    l = lse->defined() ? *lse : at::empty({T, H}, q->options().dtype(at::kFloat));
    w = ws->defined() ? *ws : bytes_like(*q, ws_bytes);
  }
  PyObject* give(int st, PyObject* out_, PyObject* lse_) const {
    if (st != QSA_OK) return PyLong_FromLong(st);
    PyObject* pair = PyTuple_New(2);
    if (!pair) return nullptr;
    PyTuple_SET_ITEM(pair, 0, out->defined() ? Py_NewRef(out_) : THPVariable_Wrap(y));
    PyTuple_SET_ITEM(pair, 1, lse->defined() ? Py_NewRef(lse_) : THPVariable_Wrap(l));
    return pair;
  }
};

// paged_forward(q, k_pages, v_pages, routes, block_table, kv_len, cu_q, scale, out | None, lse | None, workspace | None)
PyObject* paged_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 11 || !p_forward) return not_mine();
  Attention t;
  const at::Tensor* r = tensor(a[3]);
  const double scale = PyFloat_AsDouble(a[7]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return not_mine();
  }
  if (!r || !t.take(a[0], a[1], a[2], a[4], a[5], a[6], a[8], a[9], a[10]) || r->scalar_type() != at::kInt ||
      r->dim() != 2 || r->size(0) != t.T || r->size(1) > INT32_MAX || !r->is_contiguous() || !on(t.dev, r))
    return not_mine();
  const int H = static_cast<int>(t.H), G = static_cast<int>(t.c.G), n_sel = static_cast<int>(r->size(1)),
            page = static_cast<int>(t.c.page);
  t.make(p_forward_size(t.T, H, G, n_sel, page, t.c.max_pages));
  return t.give(enqueue(t.dev,
                        [&](qsa_stream_t s) {
                          return p_forward(t.q->data_ptr(), t.kp->data_ptr(), t.vp->data_ptr(), ptr<int32_t>(*r),
                                           ptr<int32_t>(*t.tb), ptr<int32_t>(*t.len), ptr<int32_t>(*t.cu), t.T,
                                           static_cast<int>(t.c.B), t.c.n_pages, page, t.c.max_pages, H, G, n_sel,
                                           static_cast<float>(scale), t.y.data_ptr(), ptr<float>(t.l), t.w.data_ptr(),
                                           static_cast<size_t>(t.w.numel()), s);
                        }),
                a[8], a[9]);
  END_HANDLE_TH_ERRORS
}

// paged_causal(q, k_pages, v_pages, block_table, kv_len, cu_q, scale, window, sinks, out | None, lse | None,
//              workspace | None)
PyObject* paged_causal(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12 || !p_causal) return not_mine();
  Attention t;
  const double scale = PyFloat_AsDouble(a[6]);
  const long window = PyLong_AsLong(a[7]), sinks = PyLong_AsLong(a[8]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return not_mine();
  }
  if (window > INT32_MAX || window < INT32_MIN || sinks > INT32_MAX || sinks < INT32_MIN ||
      !t.take(a[0], a[1], a[2], a[3], a[4], a[5], a[9], a[10], a[11]))
    return not_mine();
  const int H = static_cast<int>(t.H), G = static_cast<int>(t.c.G), page = static_cast<int>(t.c.page);
  t.make(p_causal_size(t.T, H, G, page, t.c.max_pages, static_cast<int>(window), static_cast<int>(sinks)));
  return t.give(enqueue(t.dev,
                        [&](qsa_stream_t s) {
                          return p_causal(t.q->data_ptr(), t.kp->data_ptr(), t.vp->data_ptr(), ptr<int32_t>(*t.tb),
                                          ptr<int32_t>(*t.len), ptr<int32_t>(*t.cu), t.T, static_cast<int>(t.c.B),
                                          t.c.n_pages, page, t.c.max_pages, H, G, static_cast<int>(window),
                                          static_cast<int>(sinks), static_cast<float>(scale), t.y.data_ptr(),
                                          ptr<float>(t.l), t.w.data_ptr(), static_cast<size_t>(t.w.numel()), s);
                        }),
                a[9], a[10]);
  END_HANDLE_TH_ERRORS
}

// bind(addresses of qsa_rope, qsa_cache_append, qsa_paged_forward, its workspace size, qsa_paged_causal, its workspace size)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  p_rope = reinterpret_cast<decltype(p_rope)>(p[0]);
  p_append = reinterpret_cast<decltype(p_append)>(p[1]);
  p_forward = reinterpret_cast<decltype(p_forward)>(p[2]);
  p_forward_size = reinterpret_cast<decltype(p_forward_size)>(p[3]);
  p_causal = reinterpret_cast<decltype(p_causal)>(p[4]);
  p_causal_size = reinterpret_cast<decltype(p_causal_size)>(p[5]);
  Py_RETURN_NONE;
}

#define QSA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {QSA_METHOD(bind),          QSA_METHOD(rope),         QSA_METHOD(cache_append),
                         QSA_METHOD(paged_forward), QSA_METHOD(paged_causal), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qsa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qsa_torch(void) { return PyModule_Create(&module); }
