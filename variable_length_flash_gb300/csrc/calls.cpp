// The common case of the decoding and paged entry points as one native call.
//
// A decode step's kernels take microseconds, and so does the host: a Python function that looks at
// ten tensors, allocates its outputs and goes through ctypes costs 13 to 24 us, three to four times
// the kernel; these calls take 5 to 11.  The functions here do the same for plain CUDA tensors and
// library-allocated outputs: test the arguments, allocate with torch's allocator, call the C entry
// point on the current stream of the tensors' device, whichever device is the current one.  They return
// None, having done nothing that counts, for whatever is not such a call or is refused; the Python
// function behind them then takes its own way, which says what was wrong.  What a call has to meet is
// tested on both ways and has to stay alike on both.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "vlf.h"

namespace {

decltype(&vlf_rope) p_rope;
decltype(&vlf_attn_varlen_fwd_prefix) p_prefix;
decltype(&vlf_attn_varlen_fwd_prefix_workspace_size) p_prefix_ws;
decltype(&vlf_attn_key_weights) p_weights;
decltype(&vlf_attn_key_weights_workspace_size) p_weights_ws;
decltype(&vlf_cache_evict) p_evict;
decltype(&vlf_norm_rope) p_norm;
decltype(&vlf_norm_rope_bwd) p_norm_bwd;
decltype(&vlf_norm_rope_bwd_workspace_size) p_norm_ws;
decltype(&vlf_pages_write) p_write;
decltype(&vlf_attn_varlen_fwd_pages) p_pages;
decltype(&vlf_attn_varlen_fwd_pages_workspace_size) p_pages_ws;
decltype(&vlf_pages_copy) p_copy;
decltype(&vlf_pages_fork) p_fork;
decltype(&vlf_pages_fork_workspace_size) p_fork_ws;
decltype(&vlf_pages_compact) p_compact;
decltype(&vlf_pages_compact_workspace_size) p_compact_ws;

// A plain tensor or parameter (no subclass: those have ways of their own).
const at::Tensor *tensor(PyObject *o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }
bool dense(const at::Tensor *t, at::ScalarType type, int dev) {
  return t && t->is_cuda() && t->scalar_type() == type && t->get_device() == dev && t->is_contiguous();
}
int dtype_of(const at::Tensor &t) {
  switch (t.scalar_type()) {
    case at::kHalf: return VLF_F16;
    case at::kBFloat16: return VLF_BF16;
    case at::kFloat: return VLF_F32;
    default: return -1;
  }
}
// A Python int as a C int; false (and no Python error) where it is none or does not fit.
bool whole(PyObject *o, int &x) {
  if (!PyLong_CheckExact(o)) return false;
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  x = (int)v;
  return v >= -0x7fffffffl - 1 && v <= 0x7fffffffl;
}
bool scale_of(PyObject *o, float &x) {
  if (o == Py_None) {
    x = 0.f;
    return true;
  }
  if (!PyFloat_CheckExact(o)) return false;
  x = (float)PyFloat_AS_DOUBLE(o);
  return true;
}
bool window_of(PyObject *o, int &x) {
  if (o == Py_None) {
    x = 0;
    return true;
  }
  return whole(o, x);
}
bool truth(PyObject *o, int &x) {
  x = o == Py_True;
  return o == Py_True || o == Py_False;
}
bool fits(int64_t n) { return n <= 0x7fffffffl; }
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}
vlf_stream_t stream_of(int dev) {
  return reinterpret_cast<vlf_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
}
template <typename... T> PyObject *tuple(T &...t) {
  PyObject *r = PyTuple_New(sizeof...(T));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  bool ok = true;
  auto put = [&](at::Tensor &x) {
    PyObject *o = ok ? THPVariable_Wrap(std::move(x)) : nullptr;
    ok = o != nullptr;
    if (ok) PyTuple_SET_ITEM(r, i++, o);
  };
  (put(t), ...);
  if (!ok) {
    Py_DECREF(r);
    return nullptr;
  }
  return r;
}

// (tokens strided, heads and columns dense; the stride of a single token is its width)
bool rope_rows(const at::Tensor *t, int64_t &stride) {
  if (!t || !t->is_cuda() || t->dim() != 3 || t->stride(2) != 1 || t->stride(1) != t->size(2)) return false;
  stride = t->size(0) > 1 ? t->stride(0) : t->size(1) * t->size(2);
  return fits(t->size(0)) && fits(t->size(1)) && fits(t->size(2));
}

// The position axes, and the sections given (None: one axis).
bool axes_of(const at::Tensor &pos, PyObject *given, int64_t total, int64_t half, int &axes, int (&sections)[4]) {
  if (pos.dim() < 1 || pos.dim() > 2 || pos.size(-1) != total) return false;
  const int64_t n = pos.dim() == 1 ? 1 : pos.size(0);
  axes = (int)n;
  if (given == Py_None) {
    sections[0] = (int)half;
    return n == 1;
  }
  if (!(PyTuple_CheckExact(given) || PyList_CheckExact(given)) || PySequence_Fast_GET_SIZE(given) != n || n < 1 || n > 4)
    return false;
  for (int i = 0; i < n; ++i)
    if (!whole(PySequence_Fast_GET_ITEM(given, i), sections[i])) return false;
  return true;
}

// rope(q, k, positions, inv_freq, sections, interleaved, inverse) -> (q_out, k_out)
PyObject *rope(PyObject *const *a) {
  const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *pos = tensor(a[2]), *f = tensor(a[3]);
  int64_t sq, sk;
  int interleaved, inverse;
  if (!rope_rows(q, sq) || !rope_rows(k, sk) || !truth(a[5], interleaved) || !truth(a[6], inverse)) return nullptr;
  const int dev = q->get_device(), dt = dtype_of(*q);
  const int64_t total = q->size(0), d = q->size(2);
  if (dt < 0 || k->scalar_type() != q->scalar_type() || k->get_device() != dev || k->size(0) != total ||
      k->size(2) != d || !dense(pos, at::kInt, dev) || !dense(f, at::kFloat, dev) || f->dim() != 1 || f->size(0) > d)
    return nullptr;
  int axes, sections[4];
  if (!axes_of(*pos, a[4], total, f->size(0), axes, sections)) return nullptr;
  const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
  at::Tensor qo = fresh(q->sizes(), q->scalar_type(), *q), ko = fresh(k->sizes(), k->scalar_type(), *k);
  if (p_rope(q->const_data_ptr(), sq, k->const_data_ptr(), sk, static_cast<const int32_t *>(pos->const_data_ptr()),
             axes, sections, static_cast<const float *>(f->const_data_ptr()), (int)total, (int)q->size(1),
             (int)k->size(1), (int)d, 2 * (int)f->size(0), dt, interleaved, inverse, qo.mutable_data_ptr(),
             q->size(1) * d, ko.mutable_data_ptr(), k->size(1) * d, stream_of(dev)) != VLF_OK)
    return nullptr;
  return tuple(qo, ko);
}

// prefix(q, k_prefix, v_prefix, k, v, cu_q, cu_kv, max_q, max_kv, scale, causal, window, flags) -> (out, lse)
PyObject *prefix(PyObject *const *a) {
  const at::Tensor *q = tensor(a[0]), *kp = tensor(a[1]), *vp = tensor(a[2]), *k = tensor(a[3]), *v = tensor(a[4]);
  const at::Tensor *cq = tensor(a[5]), *ck = tensor(a[6]);
  int mq, mk, causal, window, flags;
  float scale;
  if (!q || !q->is_cuda() || !whole(a[7], mq) || !whole(a[8], mk) || !scale_of(a[9], scale) || !truth(a[10], causal) ||
      !window_of(a[11], window) || !whole(a[12], flags))
    return nullptr;
  const int dev = q->get_device(), dt = dtype_of(*q);
  const at::ScalarType ty = q->scalar_type();
  if (dt < 0 || !dense(q, ty, dev) || !dense(kp, ty, dev) || !dense(vp, ty, dev) || !dense(k, ty, dev) ||
      !dense(v, ty, dev) || !dense(cq, at::kInt, dev) || !dense(ck, at::kInt, dev))
    return nullptr;
  if (q->dim() != 3 || k->dim() != 3 || v->dim() != 3 || kp->dim() != 3 || vp->dim() != 3) return nullptr;
  const int64_t tq = q->size(0), hq = q->size(1), dqk = q->size(2), tk = v->size(0), hkv = v->size(1), dv = v->size(2);
  const int64_t n = kp->size(0), seqs = cq->numel() - 1;
  if (k->size(0) != tk || k->size(1) != hkv || k->size(2) != dqk || kp->size(1) != hkv || kp->size(2) != dqk ||
      vp->size(0) != n || vp->size(1) != hkv || vp->size(2) != dv || seqs < 0 || ck->numel() - 1 != seqs)
    return nullptr;
  if (!fits(tq) || !fits(hq) || !fits(dqk) || !fits(tk) || !fits(hkv) || !fits(dv) || !fits(n) || !fits(seqs)) return nullptr;
  const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
  const size_t need = p_prefix_ws((int)seqs, (int)tq, mq, mk, (int)n, (int)hq, (int)hkv, (int)dqk, (int)dv, dt,
                                  (unsigned)flags, 0);
  at::Tensor out = fresh({tq, hq, dv}, ty, *q), lse = fresh({hq, tq}, at::kFloat, *q), ws;
  if (need) ws = fresh({(int64_t)need}, at::kByte, *q);
  if (p_prefix(q->const_data_ptr(), kp->const_data_ptr(), vp->const_data_ptr(), (int)n, k->const_data_ptr(),
               v->const_data_ptr(), static_cast<const int32_t *>(cq->const_data_ptr()),
               static_cast<const int32_t *>(ck->const_data_ptr()), (int)seqs, (int)tq, (int)tk, mq, mk, (int)hq,
               (int)hkv, (int)dqk, (int)dv, dt, scale, causal, window, out.mutable_data_ptr(),
               static_cast<float *>(lse.mutable_data_ptr()), need ? ws.mutable_data_ptr() : nullptr, need,
               stream_of(dev), (unsigned)flags) != VLF_OK)
    return nullptr;
  return tuple(out, lse);
}

// weights(q, k, lse, cu_q, cu_kv, max_q, max_kv, scale, causal, window, prev, flags) -> weights
PyObject *weights(PyObject *const *a) {
  const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *lse = tensor(a[2]), *cq = tensor(a[3]), *ck = tensor(a[4]);
  const at::Tensor *prev = a[10] == Py_None ? nullptr : tensor(a[10]);
  int mq, mk, causal, window, flags;
  float scale;
  if (!q || !q->is_cuda() || !whole(a[5], mq) || !whole(a[6], mk) || !scale_of(a[7], scale) || !truth(a[8], causal) ||
      !window_of(a[9], window) || !whole(a[11], flags))
    return nullptr;
  const int dev = q->get_device(), dt = dtype_of(*q);
  const at::ScalarType ty = q->scalar_type();
  if (dt < 0 || !dense(q, ty, dev) || !dense(k, ty, dev) || !dense(lse, at::kFloat, dev) || !dense(cq, at::kInt, dev) ||
      !dense(ck, at::kInt, dev) || (a[10] != Py_None && !dense(prev, at::kFloat, dev)))
    return nullptr;
  if (q->dim() != 3 || k->dim() != 3 || lse->dim() != 2 || (prev && prev->dim() != 2)) return nullptr;
  const int64_t tq = q->size(0), hq = q->size(1), d = q->size(2), tk = k->size(0), hkv = k->size(1), seqs = cq->numel() - 1;
  if (k->size(2) != d || lse->size(0) != hq || lse->size(1) != tq || seqs < 0 || ck->numel() - 1 != seqs ||
      (prev && (prev->size(0) != hkv || prev->size(1) != tk)))
    return nullptr;
  if (!fits(tq) || !fits(hq) || !fits(d) || !fits(tk) || !fits(hkv) || !fits(seqs)) return nullptr;
  const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
  const size_t need = p_weights_ws((int)seqs, (int)tk, mq, mk, (int)hq, (int)hkv, (int)d, dt, (unsigned)flags, 0);
  at::Tensor out = fresh({hkv, tk}, at::kFloat, *q), ws;
  if (need) ws = fresh({(int64_t)need}, at::kByte, *q);
  if (p_weights(q->const_data_ptr(), k->const_data_ptr(), static_cast<const float *>(lse->const_data_ptr()),
                static_cast<const int32_t *>(cq->const_data_ptr()), static_cast<const int32_t *>(ck->const_data_ptr()),
                (int)seqs, (int)tq, (int)tk, mq, mk, (int)hq, (int)hkv, (int)d, dt, scale, causal, window,
                prev ? static_cast<const float *>(prev->const_data_ptr()) : nullptr,
                static_cast<float *>(out.mutable_data_ptr()), need ? ws.mutable_data_ptr() : nullptr, need,
                stream_of(dev), (unsigned)flags) != VLF_OK)
    return nullptr;
  return THPVariable_Wrap(std::move(out));
}

// evict(k, v, weights, cu_kv, budget, sink, recent, max_kv, total_out) -> (k, v, weights, index, cu)
PyObject *evict(PyObject *const *a) {
  const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *w = tensor(a[2]), *cu = tensor(a[3]);
  int budget, sink, recent, mk, total;
  if (!k || !k->is_cuda() || !whole(a[4], budget) || !whole(a[5], sink) || !whole(a[6], recent) || !whole(a[7], mk) ||
      !whole(a[8], total) || total < 0)
    return nullptr;
  const int dev = k->get_device(), dt = dtype_of(*k);
  const at::ScalarType ty = k->scalar_type();
  if (dt < 0 || !dense(k, ty, dev) || !dense(v, ty, dev) || !dense(w, at::kFloat, dev) || !dense(cu, at::kInt, dev) ||
      k->dim() != 3 || v->dim() != 3 || w->dim() != 2 || cu->numel() < 2)
    return nullptr;  // (no sequences: cu_out is then the caller's to write)
  const int64_t tk = k->size(0), h = k->size(1), dk = k->size(2), dv = v->size(2), n = cu->numel() - 1;
  if (v->size(0) != tk || v->size(1) != h || w->size(0) != h || w->size(1) != tk) return nullptr;
  if (!fits(tk) || !fits(h) || !fits(dk) || !fits(dv) || !fits(n)) return nullptr;
  const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
  at::Tensor ko = fresh({total, h, dk}, ty, *k), vo = fresh({total, h, dv}, ty, *k);
  at::Tensor wo = fresh({h, total}, at::kFloat, *k), io = fresh({h, total}, at::kInt, *k), co = fresh({n + 1}, at::kInt, *k);
  if (p_evict(k->const_data_ptr(), v->const_data_ptr(), static_cast<const float *>(w->const_data_ptr()),
              static_cast<const int32_t *>(cu->const_data_ptr()), (int)n, (int)tk, mk, (int)h, (int)dk, (int)dv, dt, budget,
              sink, recent, total, ko.mutable_data_ptr(), vo.mutable_data_ptr(), static_cast<float *>(wo.mutable_data_ptr()),
              static_cast<int32_t *>(io.mutable_data_ptr()), static_cast<int32_t *>(co.mutable_data_ptr()),
              stream_of(dev)) != VLF_OK)
    return nullptr;
  return tuple(ko, vo, wo, io, co);
}

// What norm_rope and its gradients share: q, k, their weights (tensors), positions, frequencies, sections,
// interleaved, eps from a[0] on.
struct Norm {
  const at::Tensor *q, *k, *wq, *wk, *pos, *f;
  int64_t sq, sk;
  int dev, dt, wd, axes, sections[4], interleaved;
  float eps;
  bool get(PyObject *const *a) {
    q = tensor(a[0]), k = tensor(a[1]), wq = tensor(a[2]), wk = tensor(a[3]), pos = tensor(a[4]), f = tensor(a[5]);
    if (!rope_rows(q, sq) || !rope_rows(k, sk) || !wq || !wk || !truth(a[7], interleaved) || !scale_of(a[8], eps) ||
        a[8] == Py_None)
      return false;
    dev = q->get_device(), dt = dtype_of(*q), wd = dtype_of(*wq);
    const int64_t d = q->size(2);
    return dt >= 0 && k->scalar_type() == q->scalar_type() && k->get_device() == dev && k->size(0) == q->size(0) &&
           k->size(2) == d && dense(wq, wq->scalar_type(), dev) && dense(wk, wq->scalar_type(), dev) &&
           wq->dim() == 1 && wk->dim() == 1 && wq->size(0) == d && wk->size(0) == d && (wd == dt || wd == VLF_F32) &&
           dense(pos, at::kInt, dev) && dense(f, at::kFloat, dev) && f->dim() == 1 && f->size(0) <= d &&
           axes_of(*pos, a[6], q->size(0), f->size(0), axes, sections);
  }
};

// norm_rope(q, k, q_weight, k_weight, positions, inv_freq, sections, interleaved, eps) -> (q_out, k_out)
PyObject *norm_rope(PyObject *const *a) {
  Norm n;
  if (!n.get(a)) return nullptr;
  const c10::cuda::CUDAGuard on((c10::DeviceIndex)n.dev);
  const int64_t total = n.q->size(0), hq = n.q->size(1), hk = n.k->size(1), d = n.q->size(2);
  at::Tensor qo = fresh(n.q->sizes(), n.q->scalar_type(), *n.q), ko = fresh(n.k->sizes(), n.k->scalar_type(), *n.k);
  if (p_norm(n.q->const_data_ptr(), n.sq, n.k->const_data_ptr(), n.sk, n.wq->const_data_ptr(), n.wk->const_data_ptr(), n.wd,
             n.eps, static_cast<const int32_t *>(n.pos->const_data_ptr()), n.axes, n.sections,
             static_cast<const float *>(n.f->const_data_ptr()), (int)total, (int)hq, (int)hk, (int)d,
             2 * (int)n.f->size(0), n.dt, n.interleaved, qo.mutable_data_ptr(), hq * d, ko.mutable_data_ptr(), hk * d,
             stream_of(n.dev)) != VLF_OK)
    return nullptr;
  return tuple(qo, ko);
}

// norm_rope_bwd(dq_out, dk_out, q, ..., eps as above) -> (dq, dk, dq_weight, dk_weight)
PyObject *norm_rope_bwd(PyObject *const *a) {
  Norm n;
  const at::Tensor *gq = tensor(a[0]), *gk = tensor(a[1]);
  int64_t sgq, sgk;
  if (!n.get(a + 2) || !rope_rows(gq, sgq) || !rope_rows(gk, sgk)) return nullptr;
  if (gq->scalar_type() != n.q->scalar_type() || gk->scalar_type() != n.q->scalar_type() || gq->get_device() != n.dev ||
      gk->get_device() != n.dev || gq->sizes() != n.q->sizes() || gk->sizes() != n.k->sizes())
    return nullptr;
  const c10::cuda::CUDAGuard on((c10::DeviceIndex)n.dev);
  const int64_t total = n.q->size(0), hq = n.q->size(1), hk = n.k->size(1), d = n.q->size(2);
  const size_t need = p_norm_ws((int)d);
  at::Tensor dq = fresh(n.q->sizes(), n.q->scalar_type(), *n.q), dk = fresh(n.k->sizes(), n.k->scalar_type(), *n.k);
  at::Tensor dwq = fresh(n.wq->sizes(), n.wq->scalar_type(), *n.wq), dwk = fresh(n.wk->sizes(), n.wk->scalar_type(), *n.wk);
  at::Tensor ws = fresh({(int64_t)need}, at::kByte, *n.q);
  if (p_norm_bwd(gq->const_data_ptr(), sgq, gk->const_data_ptr(), sgk, n.q->const_data_ptr(), n.sq, n.k->const_data_ptr(),
                 n.sk, n.wq->const_data_ptr(), n.wk->const_data_ptr(), n.wd, n.eps,
                 static_cast<const int32_t *>(n.pos->const_data_ptr()), n.axes, n.sections,
                 static_cast<const float *>(n.f->const_data_ptr()), (int)total, (int)hq, (int)hk, (int)d,
                 2 * (int)n.f->size(0), n.dt, n.interleaved, dq.mutable_data_ptr(), hq * d, dk.mutable_data_ptr(), hk * d,
                 dwq.mutable_data_ptr(), dwk.mutable_data_ptr(), ws.mutable_data_ptr(), need, stream_of(n.dev)) != VLF_OK)
    return nullptr;
  return tuple(dq, dk, dwq, dwk);
}

// A layer's pages and scales, from a[0] on, on the device of `dev`.
struct Pool {
  const at::Tensor *k, *v, *ks, *vs;
  int n, h, page, dk, dv;
  bool get(PyObject *const *a, int dev) {
    k = tensor(a[0]), v = tensor(a[1]), ks = tensor(a[2]), vs = tensor(a[3]);
    auto bytes = [&](const at::Tensor *t) {
      return t && (t->scalar_type() == at::kByte || t->scalar_type() == at::kFloat8_e4m3fn) && t->dim() == 4 &&
             dense(t, t->scalar_type(), dev) && fits(t->size(0)) && fits(t->size(1)) && fits(t->size(2)) && fits(t->size(3));
    };
    if (!bytes(k) || !bytes(v) || !dense(ks, at::kFloat, dev) || !dense(vs, at::kFloat, dev)) return false;
    n = (int)k->size(0), h = (int)k->size(1), page = (int)k->size(2), dk = (int)k->size(3), dv = (int)v->size(3);
    auto scale = [&](const at::Tensor *t) { return t->dim() == 2 && t->size(0) == n && t->size(1) == h; };
    return v->size(0) == n && v->size(1) == h && v->size(2) == page && scale(ks) && scale(vs);
  }
  float *k_scale() const { return static_cast<float *>(ks->mutable_data_ptr()); }
  float *v_scale() const { return static_cast<float *>(vs->mutable_data_ptr()); }
};
// int32 tensors: [n], and [n, most].
bool list(const at::Tensor *t, int dev, int64_t n) { return dense(t, at::kInt, dev) && t->dim() == 1 && t->size(0) == n; }
bool table(const at::Tensor *t, int dev) {
  return dense(t, at::kInt, dev) && t->dim() == 2 && fits(t->size(0) + 1) && fits(t->size(1));
}
int32_t *ints(const at::Tensor *t) { return static_cast<int32_t *>(t->mutable_data_ptr()); }

// pages_write(k, v, k_pages, v_pages, k_scale, v_scale, page_table, cu, kv_lens) -> True
PyObject *pages_write(PyObject *const *a) {
  const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *t = tensor(a[6]), *cu = tensor(a[7]), *len = tensor(a[8]);
  int64_t sk, sv;
  Pool p;
  if (!rope_rows(k, sk) || !rope_rows(v, sv)) return nullptr;
  const int dev = k->get_device(), dt = dtype_of(*k);
  if (dt < 0 || v->scalar_type() != k->scalar_type() || v->get_device() != dev || !p.get(a + 2, dev) || !table(t, dev))
    return nullptr;
  const int64_t n = t->size(0);
  if (!list(cu, dev, n + 1) || !list(len, dev, n) || v->size(0) != k->size(0) || k->size(1) != p.h || v->size(1) != p.h ||
      k->size(2) != p.dk || v->size(2) != p.dv)
    return nullptr;
  const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
  if (p_write(k->const_data_ptr(), sk, v->const_data_ptr(), sv, p.k->mutable_data_ptr(), p.v->mutable_data_ptr(),
              p.k_scale(), p.v_scale(), ints(t), ints(cu), ints(len), (int)n, (int)k->size(0), (int)t->size(1), p.n, p.page,
              p.h, p.dk, p.dv, dt, stream_of(dev)) != VLF_OK)
    return nullptr;
  Py_RETURN_TRUE;
}

// pages_attn(q, k_pages, v_pages, k_scale, v_scale, page_table, cu_q, kv_lens, max_q, scale, causal, window, flags)
//   -> (out, lse)
PyObject *pages_attn(PyObject *const *a) {
  const at::Tensor *q = tensor(a[0]), *t = tensor(a[5]), *cu = tensor(a[6]), *len = tensor(a[7]);
  int mq, causal, window, flags;
  float scale;
  Pool p;
  if (!q || !q->is_cuda() || !whole(a[8], mq) || !scale_of(a[9], scale) || !truth(a[10], causal) ||
      !window_of(a[11], window) || !whole(a[12], flags))
    return nullptr;
  const int dev = q->get_device(), dt = dtype_of(*q);
  if (dt < 0 || !dense(q, q->scalar_type(), dev) || q->dim() != 3 || !p.get(a + 1, dev) || !table(t, dev)) return nullptr;
  const int64_t tq = q->size(0), hq = q->size(1), n = t->size(0);
  if (q->size(2) != p.dk || !list(cu, dev, n + 1) || !list(len, dev, n) || !fits(tq) || !fits(hq)) return nullptr;
  const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
  const size_t need = p_pages_ws((int)n, (int)tq, mq, (int)hq, p.h, p.dk, p.dv, dt, (unsigned)flags, 0);
  at::Tensor out = fresh({tq, hq, p.dv}, q->scalar_type(), *q), lse = fresh({hq, tq}, at::kFloat, *q), ws;
  if (need) ws = fresh({(int64_t)need}, at::kByte, *q);
  if (p_pages(q->const_data_ptr(), p.k->const_data_ptr(), p.v->const_data_ptr(), p.k_scale(), p.v_scale(), ints(t), ints(cu),
              ints(len), (int)n, (int)tq, mq, (int)t->size(1), p.n, p.page, (int)hq, p.h, p.dk, p.dv, dt, scale, causal,
              window, out.mutable_data_ptr(), static_cast<float *>(lse.mutable_data_ptr()),
              need ? ws.mutable_data_ptr() : nullptr, need, stream_of(dev), (unsigned)flags) != VLF_OK)
    return nullptr;
  return tuple(out, lse);
}

// pages_copy(k_pages, v_pages, k_scale, v_scale, src, dst) -> True
PyObject *pages_copy(PyObject *const *a) {
  const at::Tensor *src = tensor(a[4]), *dst = tensor(a[5]);
  Pool p;
  if (!src || !src->is_cuda() || src->dim() != 1 || !fits(src->size(0))) return nullptr;
  const int dev = src->get_device();
  if (!p.get(a, dev) || !list(src, dev, src->size(0)) || !list(dst, dev, src->size(0))) return nullptr;
  const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
  if (p_copy(p.k->mutable_data_ptr(), p.v->mutable_data_ptr(), p.k_scale(), p.v_scale(), ints(src), ints(dst),
             (int)src->size(0), p.n, p.page, p.h, p.dk, p.dv, stream_of(dev)) != VLF_OK)
    return nullptr;
  Py_RETURN_TRUE;
}

// Several int32 outputs of a call from one allocation, each on 256 bytes, in the order they are taken (an allocation
// costs the host 1.1 us, a fork has six outputs and a workspace): plain tensors that share its memory.  `behind`
// bytes of workspace come after them where that is little; memory that is much is an allocation of its own, so
// that an output that is kept does not keep it.
struct Pieces {
  static constexpr int64_t kLittle = 1 << 18;
  at::Tensor all, apart;
  int64_t at = 0, behind;
  static int64_t room(int64_t n) { return (n + 63) / 64 * 64; }
  Pieces(std::initializer_list<int64_t> counts, size_t workspace, const at::Tensor &like) : behind((int64_t)workspace) {
    int64_t n = 0;
    for (const int64_t c : counts) n += room(c);
    if (behind > kLittle) apart = fresh({behind}, at::kByte, like);
    else n += (behind + 3) / 4;
    all = fresh({n}, at::kInt, like);
  }
  at::Tensor take(at::IntArrayRef shape) {
    int64_t n = 1;
    for (const int64_t x : shape) n *= x;
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    at += room(n);
    return t;
  }
  void *workspace() { return behind > kLittle ? apart.mutable_data_ptr() : static_cast<int32_t *>(all.mutable_data_ptr()) + at; }
};

// pages_fork(page_table, seqlens, refs, parents, grow, page) -> (table, seqlens, refs, src, dst, left)
PyObject *pages_fork(PyObject *const *a) {
  const at::Tensor *t = tensor(a[0]), *len = tensor(a[1]), *refs = tensor(a[2]), *par = tensor(a[3]), *grow = tensor(a[4]);
  int page;
  if (!t || !t->is_cuda() || !refs || !par || refs->dim() != 1 || par->dim() != 1 || !whole(a[5], page)) return nullptr;
  const int dev = t->get_device();
  const int64_t pool = refs->size(0), m = par->size(0);
  if (!table(t, dev) || !list(len, dev, t->size(0)) || !list(refs, dev, pool) || !list(par, dev, m) || !list(grow, dev, m) ||
      !fits(pool) || !fits(m))
    return nullptr;
  const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
  const size_t need = p_fork_ws((int)pool, (int)m);
  Pieces all({m * t->size(1), m, pool, m, m, 1}, need, *t);
  at::Tensor to = all.take({m, t->size(1)}), lo = all.take({m}), ro = all.take({pool}), src = all.take({m}), dst = all.take({m});
  at::Tensor left = all.take({1});
  if (p_fork(ints(t), ints(len), ints(refs), ints(par), ints(grow), (int)t->size(0), (int)m, (int)t->size(1), (int)pool, page,
             ints(&to), ints(&lo), ints(&ro), ints(&src), ints(&dst), ints(&left), all.workspace(), need,
             stream_of(dev)) != VLF_OK)
    return nullptr;
  return tuple(to, lo, ro, src, dst, left);
}

// pages_compact(page_table, refs) -> (table, refs, to, src, dst, used)
PyObject *pages_compact(PyObject *const *a) {
  const at::Tensor *t = tensor(a[0]), *refs = tensor(a[1]);
  if (!t || !t->is_cuda() || !refs || refs->dim() != 1) return nullptr;
  const int dev = t->get_device();
  const int64_t pool = refs->size(0);
  if (!table(t, dev) || !list(refs, dev, pool) || !fits(pool)) return nullptr;
  const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
  const size_t need = p_compact_ws((int)pool);
  Pieces all({t->numel(), pool, pool, pool / 2, pool / 2, 1}, need, *t);
  at::Tensor table_out = all.take(t->sizes()), ro = all.take({pool}), to = all.take({pool}), src = all.take({pool / 2});
  at::Tensor dst = all.take({pool / 2}), used = all.take({1});
  if (p_compact(ints(t), ints(refs), (int)t->size(0), (int)t->size(1), (int)pool, ints(&table_out), ints(&ro), ints(&to),
                ints(&src), ints(&dst), ints(&used), all.workspace(), need, stream_of(dev)) != VLF_OK)
    return nullptr;
  return tuple(table_out, ro, to, src, dst, used);
}

// No C++ exception leaves (an allocation that failed: the Python function meets it again and raises).
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n == N && p_rope) {
    try {
      if (PyObject *r = F(args)) return r;
      if (PyErr_Occurred()) return nullptr;
    } catch (...) {
      PyErr_Clear();
    }
  }
  Py_RETURN_NONE;
}

// bind(addresses of the entry points, in the order of their declaration above)
PyObject *bind(PyObject *, PyObject *args) {
  constexpr int N = 17;
  void *p[N];
  if (PyTuple_GET_SIZE(args) != N) {
    PyErr_SetString(PyExc_TypeError, "bind takes the address of every entry point");
    return nullptr;
  }
  for (int i = 0; i < N; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args, i));
    if (!p[i] && PyErr_Occurred()) return nullptr;
  }
  auto set = [](auto &f, void *address) { f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(address); };
  set(p_prefix, p[1]), set(p_prefix_ws, p[2]), set(p_weights, p[3]), set(p_weights_ws, p[4]), set(p_evict, p[5]);
  set(p_norm, p[6]), set(p_norm_bwd, p[7]), set(p_norm_ws, p[8]), set(p_write, p[9]), set(p_pages, p[10]);
  set(p_pages_ws, p[11]), set(p_copy, p[12]), set(p_fork, p[13]), set(p_fork_ws, p[14]), set(p_compact, p[15]);
  set(p_compact_ws, p[16]);
  set(p_rope, p[0]);
  Py_RETURN_NONE;
}

#define FAST(F, N) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F, N>)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         {"rope", FAST(rope, 7)},
                         {"prefix", FAST(prefix, 13)},
                         {"weights", FAST(weights, 12)},
                         {"evict", FAST(evict, 9)},
                         {"norm_rope", FAST(norm_rope, 9)},
                         {"norm_rope_bwd", FAST(norm_rope_bwd, 11)},
                         {"pages_write", FAST(pages_write, 9)},
                         {"pages_attn", FAST(pages_attn, 13)},
                         {"pages_copy", FAST(pages_copy, 6)},
                         {"pages_fork", FAST(pages_fork, 6)},
                         {"pages_compact", FAST(pages_compact, 2)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// (TORCH: the version it was built against, given by the build; the package binds no other)
PyMODINIT_FUNC PyInit__calls() {
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "TORCH", VLF_TORCH) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
