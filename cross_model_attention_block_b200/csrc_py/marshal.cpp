// Argument marshalling of the decode calls (mf_rope, mf_kv_append,
// mf_paged_attn) from torch tensors, for mapflow.py.
//
// A decode step makes these calls for every layer, and at one token a
// sequence they take the GPU 3 to 11 us, a launch 2.3 us of the host: the same
// checks, allocations and stream lookup in Python took 9 to 13 us a call, here
// 1 to 2.
//
// Each function makes the call on its tensors' device, whichever is current, and
// returns its outputs, or an int, the status of a call that failed, or None where
// it refuses an argument (wrong type or shape, several devices, not on a GPU):
// mapflow.py then says which, and raises.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mapflow.h"

namespace {

decltype(&mf_rope) p_rope;
decltype(&mf_kv_append) p_append;
decltype(&mf_paged_attn) p_attn;
decltype(&mf_paged_attn_workspace) p_attn_ws;

// A tensor argument; null for None.
const at::Tensor* tensor(PyObject* o, bool& ok) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    ok = false;
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}

void* address(PyObject* o) { return o == Py_None ? nullptr : PyLong_AsVoidPtr(o); }

bool on(const at::Tensor* t, int dev) { return !t || (t->is_cuda() && t->get_device() == dev); }

bool type_of(const at::Tensor& t, mf_dtype* dt) {
  if (t.scalar_type() == at::kBFloat16)
    *dt = MF_BF16;
  else if (t.scalar_type() == at::kFloat)
    *dt = MF_F32;
  else
    return false;
  return true;
}

// [n][H][d] whose heads are d apart; `stride` gets the elements between tokens.
bool rows(const at::Tensor& t, int64_t n, int64_t H, int64_t d, at::ScalarType type,
          int64_t* stride) {
  if (t.dim() != 3 || t.size(0) != n || t.size(1) != H || t.size(2) != d ||
      t.scalar_type() != type || t.stride(2) != 1 || (t.stride(1) != d && H != 1))
    return false;
  *stride = n > 1 ? t.stride(0) : H * d;
  return true;
}

bool index(const at::Tensor* t, int64_t n) {
  return !t ||
         (t->scalar_type() == at::kInt && t->dim() == 1 && t->size(0) == n && t->is_contiguous());
}

const int32_t* ints(const at::Tensor* t) {
  return t ? static_cast<const int32_t*>(t->const_data_ptr()) : nullptr;
}

// A whole number of 32 bits.
bool number(PyObject* o, int32_t* x) {
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(o, &overflow);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *x = int32_t(v);
  return !overflow && *x == v;
}

bool number(PyObject* o, float* x) {
  *x = float(PyFloat_AsDouble(o));
  if (!PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}

// A new contiguous tensor beside `t`, from the same allocator as at::empty (whose
// dispatch takes half of its 1.2 us).
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& t) {
  return at::Tensor(at::detail::empty_cuda(sizes, type, t.device(), std::nullopt));
}

// The given output, or a new one like `t`.
at::Tensor output(const at::Tensor* given, const at::Tensor& t) {
  return given ? *given : fresh(t.sizes(), t.scalar_type(), t);
}

bool batch_of(int64_t ntok, const at::Tensor* start, const at::Tensor* cu, mf_token_batch* b) {
  if (cu && (cu->dim() != 1 || cu->size(0) < 1)) return false;
  const int64_t nseq = cu ? cu->size(0) - 1 : ntok;
  if (nseq > INT32_MAX || !index(cu, nseq + 1) || !index(start, nseq)) return false;
  *b = mf_token_batch{ntok, int32_t(nseq), ints(cu), ints(start)};
  return true;
}

PyObject* wrapped(const at::Tensor& t, PyObject* given) {
  if (given == Py_None) return THPVariable_Wrap(t);
  Py_INCREF(given);
  return given;
}

mf_stream_t stream(int dev) {
  return reinterpret_cast<mf_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
}

// Makes `dev` current for a call, where it is not.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  explicit On(int dev) {
    if (dev != c10::cuda::current_device()) guard.set_index(c10::DeviceIndex(dev));
  }
};

#define EXPECT(cond) \
  if (!(cond)) Py_RETURN_NONE

// kv_cache(K, V, page_table): (npages, page_size, Hkv, d, nseq, max_pages, device index or -1,
// the bytes of the mf_kv_cache, their address)
PyObject* kv_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 3;
  EXPECT(ok);
  const at::Tensor *K = tensor(a[0], ok), *V = tensor(a[1], ok), *table = tensor(a[2], ok);
  EXPECT(ok && K && V && table && K->dim() == 4 && K->sizes() == V->sizes() &&
         K->scalar_type() == V->scalar_type() && K->is_contiguous() && V->is_contiguous() &&
         table->scalar_type() == at::kInt && table->dim() == 2 && table->is_contiguous());
  mf_kv_cache c = {};
  EXPECT(type_of(*K, &c.dt));
  for (int i = 1; i < 4; ++i) EXPECT(K->size(i) <= INT32_MAX);
  for (int i = 0; i < 2; ++i) EXPECT(table->size(i) <= INT32_MAX);
  c.K = K->mutable_data_ptr();
  c.V = V->mutable_data_ptr();
  c.page_table = ints(table);
  c.npages = K->size(0);
  c.page_size = int32_t(K->size(1));
  c.max_pages_per_seq = int32_t(table->size(1));
  c.nseq = int32_t(table->size(0));
  c.Hkv = int32_t(K->size(2));
  c.d = int32_t(K->size(3));
  const bool one = K->is_cuda() && on(V, K->get_device()) && on(table, K->get_device());
  PyObject* bytes = PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&c), sizeof c);
  if (!bytes) return nullptr;
  return Py_BuildValue("LiiiiiiNN", (long long)c.npages, c.page_size, c.Hkv, c.d, c.nseq,
                       c.max_pages_per_seq, one ? int(K->get_device()) : -1, bytes,
                       PyLong_FromVoidPtr(PyBytes_AS_STRING(bytes)));
  END_HANDLE_TH_ERRORS
}

// rope(desc, phases, Q, K, start, cu_seqlens, Q_out, K_out, backward)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 9;
  EXPECT(ok);
  const at::Tensor *phases = tensor(a[1], ok), *Q = tensor(a[2], ok), *K = tensor(a[3], ok),
                   *start = tensor(a[4], ok), *cu = tensor(a[5], ok), *Qo = tensor(a[6], ok),
                   *Ko = tensor(a[7], ok);
  EXPECT(ok && phases && Q && (start || cu) && (K || !Ko) && Q->is_cuda() && Q->dim() == 3);
  const int dev = Q->get_device();
  EXPECT(on(phases, dev) && on(K, dev) && on(start, dev) && on(cu, dev) && on(Qo, dev) &&
         on(Ko, dev));
  const int64_t ntok = Q->size(0), Hq = Q->size(1), d = Q->size(2);
  const at::ScalarType type = Q->scalar_type();
  mf_dtype dt;
  mf_token_batch b;
  int64_t qs = 0, qos = 0, ks = 0, kos = 0, Hk = 0;
  EXPECT(type_of(*Q, &dt) && batch_of(ntok, start, cu, &b) && rows(*Q, ntok, Hq, d, type, &qs));
  if (K) {
    EXPECT(K->dim() == 3 && K->size(1) > 0);
    Hk = K->size(1);
    EXPECT(rows(*K, ntok, Hk, d, type, &ks));
    EXPECT(!Ko || rows(*Ko, ntok, Hk, d, type, &kos));
  }
  EXPECT(!Qo || rows(*Qo, ntok, Hq, d, type, &qos));
  EXPECT(Hq <= INT32_MAX && Hk <= INT32_MAX && d <= INT32_MAX);
  const int backward = PyObject_IsTrue(a[8]);
  if (backward < 0) return nullptr;
  const On here(dev);
  const at::Tensor q = output(Qo, *Q), k = K ? output(Ko, *K) : at::Tensor();
  const mf_status st =
      p_rope(static_cast<const mf_rope_desc*>(address(a[0])), &b, int32_t(d), dt, int32_t(Hq),
             Q->const_data_ptr(), qs, q.mutable_data_ptr(), Qo ? qos : Hq * d, int32_t(Hk),
             K ? K->const_data_ptr() : nullptr, ks, K ? k.mutable_data_ptr() : nullptr,
             Ko ? kos : Hk * d, backward, stream(dev));
  if (st != MF_OK) return PyLong_FromLong(st);
  PyObject* oq = wrapped(q, a[6]);
  if (!K) return oq;
  PyObject* ok_ = wrapped(k, a[7]);
  PyObject* both = PyTuple_Pack(2, oq, ok_);
  Py_DECREF(oq);
  Py_DECREF(ok_);
  return both;
  END_HANDLE_TH_ERRORS
}

// kv_append(cache desc, cache device, K, V, lens, rope desc, phases, Q, Q_out, cu_seqlens):
// Q_out, or True without Q
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 10;
  EXPECT(ok);
  const auto* c = static_cast<const mf_kv_cache*>(address(a[0]));
  const int dev = int(PyLong_AsLong(a[1]));
  const at::Tensor *K = tensor(a[2], ok), *V = tensor(a[3], ok), *lens = tensor(a[4], ok),
                   *phases = tensor(a[6], ok), *Q = tensor(a[7], ok), *Qo = tensor(a[8], ok),
                   *cu = tensor(a[9], ok);
  EXPECT(ok && K && V && (Q || !Qo) && dev >= 0 && K->is_cuda() && K->dim() == 3);
  EXPECT(on(K, dev) && on(V, dev) && on(lens, dev) && on(phases, dev) && on(Q, dev) &&
         on(Qo, dev) && on(cu, dev));
  const at::ScalarType type = c->dt == MF_BF16 ? at::kBFloat16 : at::kFloat;
  const int64_t ntok = K->size(0), d = c->d;
  mf_token_batch b;
  int64_t ks = 0, vs = 0, qs = 0, qos = 0, Hq = 0;
  EXPECT(batch_of(ntok, lens, cu, &b) && rows(*K, ntok, c->Hkv, d, type, &ks) &&
         rows(*V, ntok, c->Hkv, d, type, &vs));
  if (Q) {
    EXPECT(Q->dim() == 3 && Q->size(1) > 0 && Q->size(1) <= INT32_MAX);
    Hq = Q->size(1);
    EXPECT(rows(*Q, ntok, Hq, d, type, &qs));
    EXPECT(!Qo || rows(*Qo, ntok, Hq, d, type, &qos));
  }
  const On here(dev);
  const at::Tensor q = Q ? output(Qo, *Q) : at::Tensor();
  const mf_status st =
      p_append(c, static_cast<const mf_rope_desc*>(address(a[5])), &b, K->const_data_ptr(), ks,
               V->const_data_ptr(), vs, int32_t(Hq), Q ? Q->const_data_ptr() : nullptr, qs,
               Q ? q.mutable_data_ptr() : nullptr, Qo ? qos : Hq * d, stream(dev));
  if (st != MF_OK) return PyLong_FromLong(st);
  if (!Q) Py_RETURN_TRUE;
  return wrapped(q, a[8]);
  END_HANDLE_TH_ERRORS
}

// paged_attn(cache desc, cache device, Q, lens, O, lse, workspace, len_add, scale, band_bias,
// band_width, window): (O, lse)
PyObject* paged_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  bool ok = n == 12;
  EXPECT(ok);
  const auto* c = static_cast<const mf_kv_cache*>(address(a[0]));
  const int dev = int(PyLong_AsLong(a[1]));
  const at::Tensor *Q = tensor(a[2], ok), *lens = tensor(a[3], ok), *O = tensor(a[4], ok),
                   *lse = tensor(a[5], ok), *ws = tensor(a[6], ok);
  EXPECT(ok && Q && lens && dev >= 0 && Q->is_cuda() && Q->dim() == 3);
  EXPECT(on(Q, dev) && on(lens, dev) && on(O, dev) && on(lse, dev) && on(ws, dev));
  const at::ScalarType type = c->dt == MF_BF16 ? at::kBFloat16 : at::kFloat;
  const int64_t nseq = c->nseq, d = c->d, Hq = Q->size(1);
  int64_t qs = 0, os = 0;
  EXPECT(Hq <= INT32_MAX && rows(*Q, nseq, Hq, d, type, &qs) && index(lens, nseq));
  EXPECT(!O || rows(*O, nseq, Hq, d, type, &os));
  EXPECT(!lse || (lse->scalar_type() == at::kFloat && lse->dim() == 2 && lse->size(0) == Hq &&
                  lse->size(1) == nseq && lse->is_contiguous()));
  mf_paged_attn_desc desc;
  desc.Hq = int32_t(Hq);
  EXPECT(number(a[7], &desc.len_add) && number(a[8], &desc.scale) &&
         number(a[9], &desc.band_bias) && number(a[10], &desc.band_width) &&
         number(a[11], &desc.window));
  const On here(dev);
  const size_t bytes = p_attn_ws(c, &desc);
  EXPECT(bytes > 0);
  at::Tensor own;
  if (!ws || size_t(ws->numel()) < bytes + 256) {
    own = fresh({int64_t(bytes) + 256}, at::kByte, *Q);
    ws = &own;
  }
  EXPECT(ws->scalar_type() == at::kByte && ws->is_contiguous());
  const uintptr_t at_ws =
      (reinterpret_cast<uintptr_t>(ws->mutable_data_ptr()) + 255) & ~uintptr_t(255);
  const at::Tensor o = output(O, *Q);
  const at::Tensor l = lse ? *lse : fresh({Hq, nseq}, at::kFloat, *Q);
  const mf_status st = p_attn(c, &desc, ints(lens), Q->const_data_ptr(), qs, o.mutable_data_ptr(),
                              O ? os : Hq * d, static_cast<float*>(l.mutable_data_ptr()),
                              reinterpret_cast<void*>(at_ws), bytes, stream(dev));
  if (st != MF_OK) return PyLong_FromLong(st);
  PyObject *po = wrapped(o, a[4]), *pl = wrapped(l, a[5]);
  PyObject* both = PyTuple_Pack(2, po, pl);
  Py_DECREF(po);
  Py_DECREF(pl);
  return both;
  END_HANDLE_TH_ERRORS
}

// bind(mf_rope, mf_kv_append, mf_paged_attn, mf_paged_attn_workspace): the library's entry points
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
    return nullptr;
  }
  p_rope = reinterpret_cast<decltype(p_rope)>(PyLong_AsVoidPtr(a[0]));
  p_append = reinterpret_cast<decltype(p_append)>(PyLong_AsVoidPtr(a[1]));
  p_attn = reinterpret_cast<decltype(p_attn)>(PyLong_AsVoidPtr(a[2]));
  p_attn_ws = reinterpret_cast<decltype(p_attn_ws)>(PyLong_AsVoidPtr(a[3]));
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL,
          nullptr};
}

PyMethodDef methods[] = {method<bind>("bind"), method<rope>("rope"),
                         method<kv_cache>("kv_cache"), method<kv_append>("kv_append"),
                         method<paged_attn>("paged_attn"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  // the torch and Python it was compiled against: another's objects may lie otherwise
  if (m && PyModule_AddStringConstant(m, "built_for", MF_MARSHAL_KEY) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
