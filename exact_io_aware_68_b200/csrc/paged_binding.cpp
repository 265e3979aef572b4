// Compiled argument marshalling for paged.py: the checks, the allocations and the call of kv_append and
// attention_paged, which in Python cost 11 (attention) to 13 us (append) of a call, more than a decode step's kernels.  Only the path of a call
// that fits is here: anything else returns None, and paged.py says what does not fit.  No CUDA code; the work is the
// C ABI's (libfa_sm100.so).
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "../../include/fa.h"

namespace {

using at::Tensor;

// A tensor argument; null for None (which only optional ones may be).
struct Arg {
  const Tensor* t = nullptr;
  bool ok = false;
  explicit Arg(PyObject* o, bool optional = false) {
    if (o == Py_None) ok = optional;
    else if (THPVariable_Check(o)) {
      t = &THPVariable_Unpack(o);
      ok = true;
    }
  }
  void* ptr() const { return t ? t->data_ptr() : nullptr; }
};

bool fits(const Tensor& t, at::ScalarType dtype, at::IntArrayRef shape, int dev) {
  return t.is_cuda() && t.get_device() == dev && t.scalar_type() == dtype && t.sizes() == shape && t.is_contiguous();
}

struct Cache {
  int64_t n_pages, heads, page, width;
  int64_t step[2];   // from page to page of k_cache, v_cache
  int dev;
  bool fp8;
};

// What _refuse_cache of paged.py names the faults of.
bool cache_fits(const Tensor& k, const Tensor& v, const Arg& ks, const Arg& vs, const Tensor& table, const Tensor& lens, const Arg& news,
                int64_t B, int64_t d, Cache& c) {
  if (!k.is_cuda() || !v.is_cuda() || k.dim() != 4 || k.size(3) != d || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
    return false;
  c = Cache{k.size(0), k.size(1), k.size(2), 0, {k.stride(0), v.stride(0)}, int(k.get_device()), k.scalar_type() == at::kFloat8_e4m3fn};
  // (the stride of a dimension of size one is never taken)
  for (const Tensor* t : {&k, &v})
    if ((c.heads > 1 && t->stride(1) != c.page * d) || (c.page > 1 && t->stride(2) != d) || (d > 1 && t->stride(3) != 1)) return false;
  if (c.n_pages == 1) c.step[0] = c.step[1] = c.heads * c.page * d;
  if (v.get_device() != c.dev || (!c.fp8 && k.scalar_type() != at::kBFloat16) || c.fp8 != (ks.t != nullptr) || c.fp8 != (vs.t != nullptr))
    return false;
  if (c.fp8 && !(fits(*ks.t, at::kFloat, {c.n_pages, c.heads}, c.dev) && fits(*vs.t, at::kFloat, {c.n_pages, c.heads}, c.dev))) return false;
  if (!fits(lens, at::kInt, {B}, c.dev) || (news.t && !fits(*news.t, at::kInt, {B}, c.dev))) return false;
  if (table.dim() != 2 || table.size(0) != B) return false;
  c.width = table.size(1);
  return fits(table, at::kInt, {B, c.width}, c.dev);
}

bool is_int(int64_t x) { return x >= 0 && x <= INT32_MAX; }

// attention(q, k_cache, v_cache, page_table, key_lens, new_lens, k_scale, v_scale, workspace, o, lse, scale, causal)
// -> (o, lse), the status if the call failed, None if something does not fit; scale None: 1 / sqrt(d).
PyObject* attention_call(PyObject* const* a, Py_ssize_t n) {
  if (n != 13) Py_RETURN_NONE;
  const Arg q(a[0]), k(a[1]), v(a[2]), table(a[3]), lens(a[4]), news(a[5], true), ks(a[6], true), vs(a[7], true), ws(a[8], true),
      o(a[9], true), lse(a[10], true);
  for (const Arg* x : {&q, &k, &v, &table, &lens, &news, &ks, &vs, &ws, &o, &lse})
    if (!x->ok) Py_RETURN_NONE;
  double scale = a[11] == Py_None ? 0.0 : PyFloat_AsDouble(a[11]);
  const int causal = PyObject_IsTrue(a[12]);
  if (PyErr_Occurred()) return nullptr;
  if (q.t->dim() != 4) Py_RETURN_NONE;
  const int64_t B = q.t->size(0), Hq = q.t->size(1), Nq = q.t->size(2), d = q.t->size(3);
  Cache c;
  if (!cache_fits(*k.t, *v.t, ks, vs, *table.t, *lens.t, news, B, d, c) || !fits(*q.t, at::kBFloat16, q.t->sizes(), c.dev)) Py_RETURN_NONE;
  for (const int64_t x : {B, Hq, Nq, d, c.n_pages, c.heads, c.page, c.width})
    if (!is_int(x)) Py_RETURN_NONE;
  if ((o.t && !fits(*o.t, at::kBFloat16, q.t->sizes(), c.dev)) || (lse.t && !fits(*lse.t, at::kFloat, {B, Hq, Nq}, c.dev))) Py_RETURN_NONE;
  if (ws.t && !(ws.t->is_cuda() && ws.t->get_device() == c.dev && ws.t->scalar_type() == at::kByte && ws.t->is_contiguous())) Py_RETURN_NONE;
  {
    const c10::cuda::CUDAGuard guard(c10::DeviceIndex(c.dev));
    const auto opts = q.t->options();
    const Tensor out = o.t ? *o.t : at::empty(q.t->sizes(), opts);
    const Tensor sums = lse.t ? *lse.t : at::empty({B, Hq, Nq}, opts.dtype(at::kFloat));
    const Tensor space =
        ws.t ? *ws.t
             : at::empty({int64_t(fa_fwd_paged_workspace_size(int(B), int(Hq), int(c.heads), int(Nq), int(d)))}, opts.dtype(at::kByte));
    if (a[11] == Py_None) scale = 1.0 / std::sqrt(double(d));
    cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(c.dev)).stream();
    const auto* pt = static_cast<const int32_t*>(table.ptr());
    const auto* kl = static_cast<const int32_t*>(lens.ptr());
    const auto* nl = static_cast<const int32_t*>(news.ptr());
    fa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = c.fp8 ? fa_fwd_paged_e4m3(q.ptr(), k.ptr(), v.ptr(), static_cast<const float*>(ks.ptr()), static_cast<const float*>(vs.ptr()),
                                   out.data_ptr(), sums.data_ptr<float>(), c.step[0], c.step[1], pt, kl, nl, int(B), int(Hq),
                                   int(c.heads), int(Nq), int(d), int(c.n_pages), int(c.page), int(c.width), float(scale), causal,
                                   space.data_ptr(), size_t(space.numel()), stream)
               : fa_fwd_paged(q.ptr(), k.ptr(), v.ptr(), out.data_ptr(), sums.data_ptr<float>(), c.step[0], c.step[1], pt, kl,
                              nl, int(B), int(Hq), int(c.heads), int(Nq), int(d), int(c.n_pages), int(c.page), int(c.width),
                              float(scale), causal, space.data_ptr(), size_t(space.numel()), stream);
    Py_END_ALLOW_THREADS
    if (st != FA_OK) return PyLong_FromLong(st);
    PyObject* first = o.t ? Py_NewRef(a[9]) : THPVariable_Wrap(out);
    PyObject* second = lse.t ? Py_NewRef(a[10]) : THPVariable_Wrap(sums);
    PyObject* both = first && second ? PyTuple_Pack(2, first, second) : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(second);
    return both;
  }
}

// append(k, v, k_cache, v_cache, page_table, key_lens, new_lens, cos, sin, interleaved, q, k_scale, v_scale, q_out)
// -> q_out or True (no queries), the status if the call failed, None if something does not fit
PyObject* append_call(PyObject* const* a, Py_ssize_t n) {
  if (n != 14) Py_RETURN_NONE;
  const Arg k(a[0]), v(a[1]), kc(a[2]), vc(a[3]), table(a[4]), lens(a[5]), news(a[6], true), cos(a[7], true), sin(a[8], true),
      q(a[10], true), ks(a[11], true), vs(a[12], true), qo(a[13], true);
  for (const Arg* x : {&k, &v, &kc, &vc, &table, &lens, &news, &cos, &sin, &q, &ks, &vs, &qo})
    if (!x->ok) Py_RETURN_NONE;
  const int inter = PyObject_IsTrue(a[9]);
  if (PyErr_Occurred()) return nullptr;
  if (k.t->dim() != 4 || v.t->sizes() != k.t->sizes() || (cos.t == nullptr) != (sin.t == nullptr) || (qo.t && !q.t)) Py_RETURN_NONE;
  const int64_t B = k.t->size(0), Hkv = k.t->size(1), Nq = k.t->size(2), d = k.t->size(3);
  Cache c;
  if (!cache_fits(*kc.t, *vc.t, ks, vs, *table.t, *lens.t, news, B, d, c) || c.heads != Hkv) Py_RETURN_NONE;
  int64_t Hq = Hkv;
  if (q.t) {
    if (q.t->dim() != 4 || q.t->size(0) != B || q.t->size(2) != Nq || q.t->size(3) != d) Py_RETURN_NONE;
    Hq = q.t->size(1);
  }
  int64_t strides[9] = {};
  const Arg* x[3] = {&q, &k, &v};
  for (int i = 0; i < 3; ++i) {
    if (!x[i]->t) continue;
    const Tensor& t = *x[i]->t;
    if (!t.is_cuda() || t.get_device() != c.dev || t.scalar_type() != at::kBFloat16 || t.stride(3) != 1) Py_RETURN_NONE;
    for (int z = 0; z < 3; ++z) strides[3 * i + z] = t.size(z) > 1 ? t.stride(z) : 0;   // that of a dimension of size one is never taken
  }
  int64_t max_pos = 0, half = 0;
  if (cos.t) {
    if (cos.t->dim() != 2) Py_RETURN_NONE;
    max_pos = cos.t->size(0);
    half = cos.t->size(1);
    if (!fits(*cos.t, at::kFloat, {max_pos, half}, c.dev) || !fits(*sin.t, at::kFloat, {max_pos, half}, c.dev)) Py_RETURN_NONE;
  }
  if (qo.t && !fits(*qo.t, at::kBFloat16, q.t->sizes(), c.dev)) Py_RETURN_NONE;
  for (const int64_t z : {B, Hq, Hkv, Nq, d, c.n_pages, c.page, c.width, max_pos, 2 * half})
    if (!is_int(z)) Py_RETURN_NONE;
  {
    const c10::cuda::CUDAGuard guard(c10::DeviceIndex(c.dev));
    Tensor out;
    if (q.t) out = qo.t ? *qo.t : at::empty({B, Hq, Nq, d}, k.t->options());
    cudaStream_t stream = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(c.dev)).stream();
    void* q_out = q.t ? out.data_ptr() : nullptr;
    const auto* pt = static_cast<const int32_t*>(table.ptr());
    const auto* kl = static_cast<const int32_t*>(lens.ptr());
    const auto* nl = static_cast<const int32_t*>(news.ptr());
    const auto *cp = static_cast<const float*>(cos.ptr()), *sp = static_cast<const float*>(sin.ptr());
    fa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = c.fp8 ? fa_kv_append_e4m3(q.ptr(), k.ptr(), v.ptr(), strides, q_out, kc.ptr(), vc.ptr(), static_cast<float*>(ks.ptr()),
                                   static_cast<float*>(vs.ptr()), c.step[0], c.step[1], pt, kl, nl, cp, sp, int(max_pos),
                                   int(2 * half), inter, int(B), int(Hq), int(Hkv), int(Nq), int(d), int(c.n_pages), int(c.page),
                                   int(c.width), stream)
               : fa_kv_append(q.ptr(), k.ptr(), v.ptr(), strides, q_out, kc.ptr(), vc.ptr(), c.step[0], c.step[1], pt, kl,
                              nl, cp, sp, int(max_pos), int(2 * half), inter, int(B), int(Hq), int(Hkv), int(Nq), int(d),
                              int(c.n_pages), int(c.page), int(c.width), stream);
    Py_END_ALLOW_THREADS
    if (st != FA_OK) return PyLong_FromLong(st);
    if (!q.t) Py_RETURN_TRUE;
    return qo.t ? Py_NewRef(a[13]) : THPVariable_Wrap(out);
  }
}

// No C++ exception leaves the module: torch's own become what torch raises for them (OutOfMemoryError and the like).
template <PyObject* (*CALL)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return CALL(a, n);
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<attention_call>)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<append_call>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged(void) { return PyModule_Create(&module); }
