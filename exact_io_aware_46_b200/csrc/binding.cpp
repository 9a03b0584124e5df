// binding.cpp -- the differential calls and the append from Python, for sound arguments.
//
// A small call's kernels take a few microseconds; its checks, allocations and argument marshalling
// in Python took ten to fifteen.  These functions make the same checks on the tensors
// themselves, allocate the outputs that were not passed in and call the C entry points
// (whose addresses bind() receives).  Anything that is not sound, or not the common form (a tensor
// subclass, a stream argument, another device than the current one), returns None before any
// launch: the Python function then makes its own checks, which name what is wrong.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <optional>

#include "attn.h"

namespace {

struct {
  decltype(&attn_fwd_diff) fwd;
  decltype(&attn_bwd_diff) bwd;
  decltype(&attn_fwd_splitkv_decode_diff) decode;
  decltype(&attn_fwd_splitkv_decode_diff_paged) decode_paged;
  decltype(&attn_kv_append_paged) append;
  decltype(&attn_bwd_diff_workspace_size) bwd_size;
  decltype(&attn_fwd_diff_workspace_size) fwd_size;
  decltype(&attn_decode_diff_workspace_size) decode_size;
  decltype(&attn_kv_append_paged_workspace_size) append_size;
  decltype(&attn_clear_device_status) clear;
  decltype(&attn_num_sms) num_sms;
} api;
bool bound = false;

constexpr auto BF16 = at::kBFloat16;
constexpr auto F32 = at::kFloat;
constexpr auto I32 = at::kInt;

// One argument that is a tensor: nullptr unless it is exactly that, dense and on `dev`
// (dev < 0: any GPU).
const at::Tensor* tensor(PyObject* o, c10::ScalarType type, int dev) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.layout() != at::kStrided || !t.is_cuda() || t.scalar_type() != type) return nullptr;
  if (dev >= 0 && t.get_device() != dev) return nullptr;
  for (const int64_t n : t.sizes())
    if (n > INT_MAX) return nullptr;
  return &t;
}
const at::Tensor* dense(PyObject* o, c10::ScalarType type, int dev) {
  const at::Tensor* t = tensor(o, type, dev);
  return t && t->is_contiguous() ? t : nullptr;
}
const at::Tensor* shaped(PyObject* o, c10::ScalarType type, int dev, at::IntArrayRef shape) {
  const at::Tensor* t = dense(o, type, dev);
  return t && t->sizes().equals(shape) ? t : nullptr;
}
// An optional one: false if it is there and not sound.
bool optional(PyObject* o, c10::ScalarType type, int dev, at::IntArrayRef shape,
              const at::Tensor** out) {
  *out = nullptr;
  if (o == Py_None) return true;
  return (*out = shaped(o, type, dev, shape)) != nullptr;
}

template <typename T>
T* ptr(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
using bf16 = attn_bf16_t;

// The tensor that was passed in, or a new one.
struct Out {
  const at::Tensor* given;
  at::Tensor made;
  Out(const at::Tensor* g, bool want, at::IntArrayRef shape, c10::ScalarType type, int dev)
      : given(g) {
    if (!g && want)
      made = at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, dev), std::nullopt);
  }
  template <typename T>
  T* data() const {
    return given ? static_cast<T*>(given->data_ptr())
                 : made.defined() ? static_cast<T*>(made.data_ptr()) : nullptr;
  }
  PyObject* object(PyObject* arg) {  // a new reference; None where nothing was wanted
    if (given || !made.defined()) return Py_NewRef(arg);
    return THPVariable_Wrap(std::move(made));
  }
};

// The caller's workspace, or one for this call.
struct Workspace {
  at::Tensor made;
  void* p = nullptr;
  size_t bytes = 0;
  bool ok = true;
  template <typename Size>
  Workspace(PyObject* arg, int dev, void* stream, const Size& size, bool clear) {
    if (arg != Py_None) {
      const at::Tensor* t = dense(arg, at::kByte, dev);
      if (!(ok = t != nullptr)) return;
      p = t->data_ptr();
      bytes = static_cast<size_t>(t->numel());
      return;
    }
    bytes = size();
    made = at::detail::empty_cuda({static_cast<int64_t>(bytes)}, at::kByte,
                                  at::Device(at::kCUDA, dev), std::nullopt);
    p = made.data_ptr();
    // nobody reads its status word: cleared only where the call needs its counters at zero
    if (clear) ok = api.clear(p, stream) == ATTN_OK;
  }
};

struct Heads {
  const at::Tensor *Q, *K, *V;
  int B, Hq, Hkv, Lq, Lk, d, dev;
};
bool current(int dev) { return dev == c10::cuda::current_device(); }
void* stream_of(int dev) {
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
}

// Q [B,Hq,Lq,d], K and V [*,Hkv,Lk,d] (cache: any first dimension) on the current device.
bool heads(PyObject* const* a, Heads* h, bool cache) {
  if (!(h->Q = dense(a[0], BF16, -1)) || h->Q->dim() != 4) return false;
  h->dev = h->Q->get_device();
  const auto q = h->Q->sizes();
  if (!current(h->dev) || !(h->K = dense(a[1], BF16, h->dev)) || h->K->dim() != 4) return false;
  const auto k = h->K->sizes();
  if (k[3] != q[3] || (!cache && k[0] != q[0]) || !(h->V = shaped(a[2], BF16, h->dev, k)))
    return false;
  h->B = static_cast<int>(q[0]);
  h->Hq = static_cast<int>(q[1]);
  h->Lq = static_cast<int>(q[2]);
  h->d = static_cast<int>(q[3]);
  h->Hkv = static_cast<int>(k[1]);
  h->Lk = static_cast<int>(k[2]);
  return h->B > 0 && h->d > 0 && h->Hkv > 0 && h->Hq > 0 && h->Hq % h->Hkv == 0;
}

const at::Tensor* weight(PyObject* o, const Heads& h) {
  const at::Tensor* t = dense(o, F32, h.dev);
  return t && t->dim() == 1 && (t->numel() == 1 || t->numel() == h.Hq) ? t : nullptr;
}

bool scale_of(PyObject* o, int d, float* s) {
  if (o == Py_None) {
    *s = static_cast<float>(1. / std::sqrt(d / 2.));
    return true;
  }
  if (!PyFloat_CheckExact(o)) return false;
  *s = static_cast<float>(PyFloat_AS_DOUBLE(o));
  return true;
}

// Runs `call` without the interpreter lock.  A refusal happened before any launch and
// is left to the Python function (true); any other status is kept.
template <typename F>
bool refused(int* status, const F& call) {
  PyThreadState* st = PyEval_SaveThread();
  *status = call();
  PyEval_RestoreThread(st);
  return *status == ATTN_ERR_INVALID || *status == ATTN_ERR_UNSUPPORTED;
}

// (Q, K, V, lam, scale, causal, k_lens, O, O2, lse, workspace, want_aux)
PyObject* fwd_diff(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Heads h;
  const at::Tensor *lam, *kl, *o, *o2, *ls;
  float scale;
  if (!bound || n != 12 || !heads(a, &h, false) || !(lam = weight(a[3], h)) ||
      !scale_of(a[4], h.d, &scale) || !optional(a[6], I32, h.dev, {h.B}, &kl) ||
      !optional(a[7], BF16, h.dev, h.Q->sizes(), &o) ||
      !optional(a[8], BF16, h.dev, h.Q->sizes(), &o2) ||
      !optional(a[9], F32, h.dev, {h.B, h.Hq, 2, h.Lq}, &ls))
    Py_RETURN_NONE;
  const int causal = PyObject_IsTrue(a[5]), aux = PyObject_IsTrue(a[11]);
  if (causal < 0 || aux < 0) return nullptr;
  void* s = stream_of(h.dev);
  const long long tiles = static_cast<long long>(h.B) * h.Hq * ((h.Lq + 127LL) / 128);
  Workspace ws(
      a[10], h.dev, s, [&] { return api.fwd_size(h.B, h.Hq, h.Hkv, h.Lq, h.Lk, h.d); },
      tiles > api.num_sms());
  if (!ws.ok) Py_RETURN_NONE;
  Out O(o, true, h.Q->sizes(), BF16, h.dev), O2(o2, aux, h.Q->sizes(), BF16, h.dev);
  Out L(ls, aux, {h.B, h.Hq, 2, h.Lq}, F32, h.dev);
  int st;
  if (refused(&st, [&] {
        return api.fwd(ptr<bf16>(h.Q), ptr<bf16>(h.K), ptr<bf16>(h.V), ptr<float>(lam),
                       static_cast<int>(lam->numel()), O.data<bf16>(), O2.data<bf16>(),
                       L.data<float>(), h.B, h.Hq, h.Hkv, h.Lq, h.Lk, h.d, scale,
                       causal ? ATTN_MASK_CAUSAL : ATTN_MASK_NONE, ptr<int32_t>(kl), ws.p, ws.bytes,
                       s);
      }))
    Py_RETURN_NONE;
  if (st != ATTN_OK) return PyLong_FromLong(st);
  return Py_BuildValue("(NNN)", O.object(a[7]), O2.object(a[8]), L.object(a[9]));
  END_HANDLE_TH_ERRORS
}

// (Q, K, V, lam, O, O2, dO, lse, scale, causal, k_lens, dQ, dK, dV, dlam, workspace)
PyObject* bwd_diff(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Heads h;
  const at::Tensor *lam, *o, *o2, *go, *ls, *kl, *gq, *gk, *gv, *gl;
  float scale;
  if (!bound || n != 16 || !heads(a, &h, false) || !(lam = weight(a[3], h)) ||
      !(o = shaped(a[4], BF16, h.dev, h.Q->sizes())) ||
      !(o2 = shaped(a[5], BF16, h.dev, h.Q->sizes())) ||
      !(go = shaped(a[6], BF16, h.dev, h.Q->sizes())) ||
      !(ls = shaped(a[7], F32, h.dev, {h.B, h.Hq, 2, h.Lq})) || !scale_of(a[8], h.d, &scale) ||
      !optional(a[10], I32, h.dev, {h.B}, &kl) ||
      !optional(a[11], BF16, h.dev, h.Q->sizes(), &gq) ||
      !optional(a[12], BF16, h.dev, h.K->sizes(), &gk) ||
      !optional(a[13], BF16, h.dev, h.K->sizes(), &gv) ||
      !optional(a[14], BF16, h.dev, lam->sizes(), &gl))
    Py_RETURN_NONE;
  const int causal = PyObject_IsTrue(a[9]);
  if (causal < 0) return nullptr;
  void* s = stream_of(h.dev);
  Workspace ws(
      a[15], h.dev, s, [&] { return api.bwd_size(h.B, h.Hq, h.Hkv, h.Lq, h.Lk, h.d); },
      h.Lq == 0);
  if (!ws.ok) Py_RETURN_NONE;
  Out dQ(gq, true, h.Q->sizes(), BF16, h.dev), dK(gk, true, h.K->sizes(), BF16, h.dev);
  Out dV(gv, true, h.K->sizes(), BF16, h.dev), dl(gl, true, lam->sizes(), BF16, h.dev);
  int st;
  if (refused(&st, [&] {
        return api.bwd(ptr<bf16>(h.Q), ptr<bf16>(h.K), ptr<bf16>(h.V), ptr<float>(lam),
                       static_cast<int>(lam->numel()), ptr<bf16>(o), ptr<bf16>(o2), ptr<bf16>(go),
                       ptr<float>(ls), dQ.data<bf16>(), dK.data<bf16>(), dV.data<bf16>(),
                       dl.data<bf16>(), h.B, h.Hq, h.Hkv, h.Lq, h.Lk, h.d, scale,
                       causal ? ATTN_MASK_CAUSAL : ATTN_MASK_NONE, ptr<int32_t>(kl), ws.p, ws.bytes,
                       s);
      }))
    Py_RETURN_NONE;
  if (st != ATTN_OK) return PyLong_FromLong(st);
  return Py_BuildValue("(NNNN)", dQ.object(a[11]), dK.object(a[12]), dV.object(a[13]),
                       dl.object(a[14]));
  END_HANDLE_TH_ERRORS
}

// (Q, K, V, block_table or None, lam, k_lens, scale, O, lse, workspace, want_lse)
PyObject* decode_diff(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Heads h;
  const at::Tensor *lam, *kl, *bt = nullptr, *o, *ls;
  float scale;
  if (!bound || n != 11 || !heads(a, &h, true) || h.Lq != 1 || !(lam = weight(a[4], h)) ||
      !(kl = shaped(a[5], I32, h.dev, {h.B})) || !scale_of(a[6], h.d, &scale) ||
      !optional(a[7], BF16, h.dev, h.Q->sizes(), &o) ||
      !optional(a[8], F32, h.dev, {h.B, h.Hq, 2}, &ls))
    Py_RETURN_NONE;
  long long rows = h.Lk;
  if (a[3] != Py_None) {
    if (!(bt = dense(a[3], I32, h.dev)) || bt->dim() != 2 || bt->size(0) != h.B) Py_RETURN_NONE;
    rows *= bt->size(1);
  } else if (h.K->size(0) != h.B) {
    Py_RETURN_NONE;
  }
  if (rows > (1LL << 30)) Py_RETURN_NONE;
  const int want = PyObject_IsTrue(a[10]);
  if (want < 0) return nullptr;
  void* s = stream_of(h.dev);
  Workspace ws(
      a[9], h.dev, s,
      [&] { return api.decode_size(h.B, h.Hq, h.Hkv, static_cast<int>(rows), h.d); }, false);
  if (!ws.ok) Py_RETURN_NONE;
  Out O(o, true, h.Q->sizes(), BF16, h.dev), L(ls, want, {h.B, h.Hq, 2}, F32, h.dev);
  const int n_lam = static_cast<int>(lam->numel());
  int st;
  if (refused(&st, [&] {
        return bt ? api.decode_paged(ptr<bf16>(h.Q), ptr<bf16>(h.K), ptr<bf16>(h.V),
                                     ptr<int32_t>(bt), static_cast<int>(bt->size(1)), h.Lk,
                                     static_cast<int>(h.K->size(0)), ptr<float>(lam), n_lam,
                                     O.data<bf16>(), L.data<float>(), h.B, h.Hq, h.Hkv, h.d, scale,
                                     ptr<int32_t>(kl), ws.p, ws.bytes, s)
                  : api.decode(ptr<bf16>(h.Q), ptr<bf16>(h.K), ptr<bf16>(h.V), ptr<float>(lam),
                               n_lam, O.data<bf16>(), L.data<float>(), h.B, h.Hq, h.Hkv, h.Lk, h.d,
                               scale, ptr<int32_t>(kl), ws.p, ws.bytes, s);
      }))
    Py_RETURN_NONE;
  if (st != ATTN_OK) return PyLong_FromLong(st);
  return Py_BuildValue("(NN)", O.object(a[7]), L.object(a[8]));
  END_HANDLE_TH_ERRORS
}

// New tokens [T, H, d] whose head rows are contiguous within a token.
bool tokens(PyObject* o, int dev, int64_t d, int64_t H, int64_t T, const at::Tensor** out) {
  const at::Tensor* t = tensor(o, BF16, dev);
  if (!t || t->dim() != 3 || t->size(2) != d || t->stride(2) != 1 || t->stride(1) != d ||
      t->stride(0) % 8 != 0 || t->stride(0) < t->size(1) * d || t->size(0) == 0 ||
      (H >= 0 && t->size(1) != H) || (T >= 0 && t->size(0) != T))
    return false;
  *out = t;
  return true;
}

// (K, V, Kp, Vp, block_table, k_lens, cu_seqlens, Q, Q_out, cos, sin, maps, interleaved, workspace)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const at::Tensor *Kp, *K, *V, *Q = nullptr, *bt, *kl, *cu = nullptr, *qo = nullptr;
  const at::Tensor *cs = nullptr, *sn = nullptr;
  if (!bound || n != 14 || !(Kp = dense(a[2], BF16, -1)) || Kp->dim() != 4) Py_RETURN_NONE;
  const int dev = Kp->get_device();
  const int64_t n_pages = Kp->size(0), Hkv = Kp->size(1), page = Kp->size(2), d = Kp->size(3);
  const at::Tensor* Vp;
  if (!current(dev) || !(Vp = shaped(a[3], BF16, dev, Kp->sizes())) || Hkv < 1 ||
      !tokens(a[0], dev, d, Hkv, -1, &K) || !tokens(a[1], dev, d, Hkv, K->size(0), &V) ||
      !(kl = dense(a[5], I32, dev)) || kl->dim() != 1 || kl->numel() < 1)
    Py_RETURN_NONE;
  const int64_t T = K->size(0), B = kl->numel();
  if (a[6] == Py_None ? T != B : !(cu = shaped(a[6], I32, dev, {B + 1}))) Py_RETURN_NONE;
  if (!(bt = dense(a[4], I32, dev)) || bt->dim() != 2 || bt->size(0) != B) Py_RETURN_NONE;
  int64_t Hq = Hkv;
  if (a[7] != Py_None) {
    if (!tokens(a[7], dev, d, -1, T, &Q)) Py_RETURN_NONE;
    Hq = Q->size(1);
    if (Hq < 1 || Hq % Hkv != 0 || !optional(a[8], BF16, dev, {T, Hq, d}, &qo)) Py_RETURN_NONE;
  } else if (a[8] != Py_None) {
    Py_RETURN_NONE;
  }
  if ((a[9] == Py_None) != (a[10] == Py_None)) Py_RETURN_NONE;
  int64_t n_pos = 0, rope = 0;
  if (a[9] != Py_None) {
    if (!(cs = dense(a[9], F32, dev)) || cs->dim() != 2 ||
        !(sn = shaped(a[10], F32, dev, cs->sizes())) || cs->size(1) > d)
      Py_RETURN_NONE;
    n_pos = cs->size(0);
    rope = 2 * cs->size(1);
  }
  if (!PyLong_CheckExact(a[11])) Py_RETURN_NONE;
  int over = 0;
  const long maps = PyLong_AsLongAndOverflow(a[11], &over);
  if (over || maps < 1 || maps > 2) Py_RETURN_NONE;
  const int inter = PyObject_IsTrue(a[12]);
  if (inter < 0) return nullptr;
  void* s = stream_of(dev);
  Workspace ws(a[13], dev, s, [&] { return api.append_size(); }, false);
  if (!ws.ok) Py_RETURN_NONE;
  Out out(qo, Q != nullptr, {T, Hq, d}, BF16, dev);
  int st;
  if (refused(&st, [&] {
        auto i = [](int64_t v) { return static_cast<int>(v); };
        return api.append(ptr<bf16>(Q), Q ? Q->stride(0) : 0, ptr<bf16>(K), K->stride(0),
                          ptr<bf16>(V), V->stride(0), out.data<bf16>(), ptr<bf16>(Kp),
                          ptr<bf16>(Vp), ptr<int32_t>(bt), i(bt->size(1)), i(page), i(n_pages),
                          ptr<int32_t>(cu), ptr<int32_t>(kl), i(B), i(T), i(Hq), i(Hkv), i(d),
                          ptr<float>(cs), ptr<float>(sn), i(n_pos), i(rope), i(maps),
                          inter ? 1 : 0, ws.p, ws.bytes, s);
      }))
    Py_RETURN_NONE;
  if (st != ATTN_OK) return PyLong_FromLong(st);
  return Py_BuildValue("(N)", out.object(a[8]));
  END_HANDLE_TH_ERRORS
}

// bind(addresses of the entry points, in the order of NAMES)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void** slot[] = {reinterpret_cast<void**>(&api.fwd),         reinterpret_cast<void**>(&api.bwd),
                   reinterpret_cast<void**>(&api.decode),      reinterpret_cast<void**>(&api.decode_paged),
                   reinterpret_cast<void**>(&api.append),      reinterpret_cast<void**>(&api.fwd_size),
                   reinterpret_cast<void**>(&api.bwd_size),    reinterpret_cast<void**>(&api.decode_size),
                   reinterpret_cast<void**>(&api.append_size), reinterpret_cast<void**>(&api.clear),
                   reinterpret_cast<void**>(&api.num_sms)};
  constexpr Py_ssize_t N = sizeof(slot) / sizeof(slot[0]);
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "bind takes %zd addresses, got %zd", N, n);
    return nullptr;
  }
  void* v[N];
  for (Py_ssize_t i = 0; i < N; ++i) {
    v[i] = PyLong_AsVoidPtr(a[i]);
    if (!v[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  for (Py_ssize_t i = 0; i < N; ++i) *slot[i] = v[i];
  bound = true;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {
    {"fwd_diff", fast<fwd_diff>(), METH_FASTCALL, nullptr},
    {"bwd_diff", fast<bwd_diff>(), METH_FASTCALL, nullptr},
    {"decode_diff", fast<decode_diff>(), METH_FASTCALL, nullptr},
    {"append", fast<append>(), METH_FASTCALL, nullptr},
    {"bind", fast<bind>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  // what it was compiled against, compared when it is loaded
  if (m && PyModule_AddStringConstant(m, "BUILT_FOR", BINDING_TAG) < 0) Py_CLEAR(m);
  return m;
}
