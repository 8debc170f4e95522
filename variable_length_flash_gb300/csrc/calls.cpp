// The common case of the decoding entry points as one native call.
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
  if (pos->dim() < 1 || pos->dim() > 2 || pos->size(-1) != total) return nullptr;
  const int64_t axes = pos->dim() == 1 ? 1 : pos->size(0);
  int sections[4];
  if (a[4] == Py_None) {
    if (axes != 1) return nullptr;
    sections[0] = (int)f->size(0);
  } else {
    if (!(PyTuple_CheckExact(a[4]) || PyList_CheckExact(a[4])) || PySequence_Fast_GET_SIZE(a[4]) != axes || axes < 1 ||
        axes > 4)
      return nullptr;
    for (int i = 0; i < axes; ++i)
      if (!whole(PySequence_Fast_GET_ITEM(a[4], i), sections[i])) return nullptr;
  }
  const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
  at::Tensor qo = fresh(q->sizes(), q->scalar_type(), *q), ko = fresh(k->sizes(), k->scalar_type(), *k);
  if (p_rope(q->const_data_ptr(), sq, k->const_data_ptr(), sk, static_cast<const int32_t *>(pos->const_data_ptr()),
             (int)axes, sections, static_cast<const float *>(f->const_data_ptr()), (int)total, (int)q->size(1),
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

// bind(addresses of the six entry points, in the order of their declaration above)
PyObject *bind(PyObject *, PyObject *args) {
  unsigned long long p[6];
  if (!PyArg_ParseTuple(args, "KKKKKK", p, p + 1, p + 2, p + 3, p + 4, p + 5)) return nullptr;
  p_prefix = reinterpret_cast<decltype(p_prefix)>(p[1]);
  p_prefix_ws = reinterpret_cast<decltype(p_prefix_ws)>(p[2]);
  p_weights = reinterpret_cast<decltype(p_weights)>(p[3]);
  p_weights_ws = reinterpret_cast<decltype(p_weights_ws)>(p[4]);
  p_evict = reinterpret_cast<decltype(p_evict)>(p[5]);
  p_rope = reinterpret_cast<decltype(p_rope)>(p[0]);
  Py_RETURN_NONE;
}

#define FAST(F, N) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F, N>)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         {"rope", FAST(rope, 7)},
                         {"prefix", FAST(prefix, 13)},
                         {"weights", FAST(weights, 12)},
                         {"evict", FAST(evict, 9)},
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
