// The Python calls that are made per layer and per token, without Python's own
// time: a CPython module that checks a call's tensors, allocates its outputs and
// workspace, and calls libstreamkl.  It takes the ordinary case (device tensors
// of the current device, in a layout the library reads in place) and returns
// None for everything else: _lib.py then goes through the same call step by
// step, copies what has to be copied, and reports what is wrong.  A call's host
// time against the ctypes path's: attention forward 7 to 8 us against 24, its
// backward 13 to 14 against 37, log probabilities 9 to 10 against 24, their gradient
// 4 to 5 against 18; the short calls' kernels take 6 to 14 us.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <climits>

#include "streamkl.h"

namespace {

const at::Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on_device(const at::Tensor& t, int index) { return t.is_cuda() && t.get_device() == index; }

struct Strides {
  long long b, h, n;
};

// A [B, H, N, D] bf16 tensor that the library reads in place: heads by rows or rows by heads, 16-byte granules.
bool layout(const at::Tensor& t, Strides* s) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 4 || t.numel() == 0) return false;
  const auto size = t.sizes(), st = t.strides();
  const long long sb = st[0], sh = st[1], sn = st[2], H = size[1], N = size[2], D = size[3];
  if (st[3] != 1 || (reinterpret_cast<uintptr_t>(t.const_data_ptr()) & 15) || ((sb | sh | sn) & 7)) return false;
  const bool by_head = D <= sn && sn * N <= sh && sh * H <= sb, by_row = D <= sh && sh * H <= sn && sn * N <= sb;
  if (!(by_head || by_row) || sb >= (1ll << 38)) return false;
  *s = Strides{sb, sh, sn};
  return true;
}

// None or int32 [B] on the device; false where the ordinary path does not take it.
bool lengths(PyObject* o, int64_t B, int index, const int** out) {
  *out = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != at::kInt || t->dim() != 1 || t->size(0) != B || !on_device(*t, index) || !t->is_contiguous())
    return false;
  *out = t->const_data_ptr<int>();
  return true;
}

// fp32 of `like`'s leading sizes (or all of them), contiguous; null for None.
bool rows(PyObject* o, at::IntArrayRef size, int index, const float** out) {
  *out = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != at::kFloat || t->sizes() != size || !on_device(*t, index) || !t->is_contiguous()) return false;
  *out = t->const_data_ptr<float>();
  return true;
}

at::TensorOptions options(at::ScalarType type, int index) {
  return at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(index)));
}

struct Attention {
  const at::Tensor *q, *k, *v;
  int index;
  Strides qs, ks, vs;
  streamkl_attn_shape s;
};

// q, k, v, scale, causal, q_lens, k_lens at args[0], [1], [2], `at`, at + 1, at + 2, at + 3.
bool attention(PyObject* const* args, int at, Attention* a) {
  a->q = tensor(args[0]);
  a->k = tensor(args[1]);
  a->v = tensor(args[2]);
  if (!a->q || !a->k || !a->v || !a->q->is_cuda()) return false;
  a->index = a->q->get_device();
  if (a->index != c10::cuda::current_device() || !on_device(*a->k, a->index) || !on_device(*a->v, a->index)) return false;
  if (!layout(*a->q, &a->qs) || !layout(*a->k, &a->ks) || !layout(*a->v, &a->vs)) return false;
  const auto q = a->q->sizes(), k = a->k->sizes();
  if (k != a->v->sizes() || q[0] != k[0] || q[3] != k[3] || q[1] % k[1]) return false;
  for (int i = 0; i < 3; ++i)
    if (q[i] > INT_MAX || k[i] > INT_MAX) return false;
  double scale = 0;
  if (args[at] != Py_None) {
    if (!PyFloat_Check(args[at])) return false;
    scale = PyFloat_AS_DOUBLE(args[at]);
  }
  if (!PyBool_Check(args[at + 1])) return false;
  const int *ql, *kl;
  if (!lengths(args[at + 2], q[0], a->index, &ql) || !lengths(args[at + 3], q[0], a->index, &kl)) return false;
  a->s = streamkl_attn_shape{(int)q[0], (int)q[1], (int)k[1], (int)q[2], (int)k[2], (int)q[3], (float)scale,
                             args[at + 1] == Py_True, ql, kl, a->qs.b, a->qs.h, a->qs.n, a->ks.b, a->ks.h, a->ks.n,
                             a->vs.b, a->vs.h, a->vs.n, a->qs.b, a->qs.h, a->qs.n};
  return true;
}

at::Tensor like(const at::Tensor& t, const Strides& s, int index) {
  return at::empty_strided(t.sizes(), {s.b, s.h, s.n, 1}, options(at::kBFloat16, index));
}

at::Tensor workspace(size_t bytes, int index) {
  return bytes ? at::empty({static_cast<int64_t>(bytes)}, options(at::kByte, index)) : at::Tensor();
}

void* data(const at::Tensor& t) { return t.defined() ? t.mutable_data_ptr() : nullptr; }

// Other Python threads run while outputs are allocated and kernels launched, as they do in a call through ctypes.
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

void* stream(int index) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream(); }

PyObject* tuple(std::initializer_list<at::Tensor> tensors) {
  THPObjectPtr t(PyTuple_New(static_cast<Py_ssize_t>(tensors.size())));
  if (!t) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& x : tensors) PyTuple_SET_ITEM(t.get(), i++, THPVariable_Wrap(x));
  return t.release();
}

// attn_fwd(q, k, v, scale, causal, q_lens, k_lens[, return_rest])
PyObject* attn_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Attention a;
  if ((n != 7 && n != 8) || !attention(args, 3, &a) || (n == 8 && !PyBool_Check(args[7]))) Py_RETURN_NONE;
  const bool with_rest = n == 8 && args[7] == Py_True;
  at::Tensor o, lse, rest;
  int status;
  {
    NoGil no_gil;
    size_t bytes = 0;
    if (with_rest) {
      rest = like(*a.q, a.qs, a.index);
      a.s.o_rest = data(rest);
    }
    status = streamkl_attn_fwd_workspace(a.s, &bytes);
    if (status == STREAMKL_OK) {
      const at::Tensor ws = workspace(bytes, a.index);
      o = like(*a.q, a.qs, a.index);
      lse = at::empty({a.s.B, a.s.H, a.s.NQ}, options(at::kFloat, a.index));
      status = streamkl_attn_fwd(a.q->const_data_ptr(), a.k->const_data_ptr(), a.v->const_data_ptr(), a.s, data(o),
                                 static_cast<float*>(data(lse)), data(ws), bytes, stream(a.index));
    }
  }
  if (status != STREAMKL_OK) Py_RETURN_NONE;
  return with_rest ? tuple({o, lse, rest}) : tuple({o, lse});
  END_HANDLE_TH_ERRORS
}

// attn_bwd(q, k, v, o, lse, do, dlse, scale, causal, q_lens, k_lens, bwd_mode[, o_rest])
PyObject* attn_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Attention a;
  if ((n != 12 && n != 13) || !attention(args, 7, &a)) Py_RETURN_NONE;
  const at::Tensor *o = tensor(args[3]), *go = tensor(args[5]);
  Strides os, gs;
  if (!o || !go || !on_device(*o, a.index) || !on_device(*go, a.index) || o->sizes() != a.q->sizes() ||
      go->sizes() != a.q->sizes() || !layout(*o, &os) || !layout(*go, &gs) || os.b != gs.b || os.h != gs.h || os.n != gs.n)
    Py_RETURN_NONE;
  a.s.o_stride_b = os.b;
  a.s.o_stride_h = os.h;
  a.s.o_stride_n = os.n;
  if (n == 13 && args[12] != Py_None) {
    const at::Tensor* rest = tensor(args[12]);
    Strides rs;
    if (!rest || !on_device(*rest, a.index) || rest->sizes() != a.q->sizes() || !layout(*rest, &rs) || rs.b != os.b ||
        rs.h != os.h || rs.n != os.n)
      Py_RETURN_NONE;
    a.s.o_rest = const_cast<void*>(rest->const_data_ptr());  // read only
  }
  const float *lse, *dlse;
  const auto row_sizes = a.q->sizes().slice(0, 3);
  if (args[4] == Py_None || !rows(args[4], row_sizes, a.index, &lse) || !rows(args[6], row_sizes, a.index, &dlse) ||
      !PyLong_Check(args[11]))
    Py_RETURN_NONE;
  const long mode = PyLong_AsLong(args[11]);
  if (mode < 0 || mode > INT_MAX) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  at::Tensor dq, dk, dv;
  int status;
  {
    NoGil no_gil;
    size_t bytes = 0;
    status = streamkl_attn_bwd_workspace(a.s, (int)mode, &bytes);
    if (status == STREAMKL_OK) {
      const at::Tensor ws = workspace(bytes, a.index);
      dq = like(*a.q, a.qs, a.index);
      dk = like(*a.k, a.ks, a.index);
      dv = like(*a.v, a.vs, a.index);
      status = streamkl_attn_bwd(a.q->const_data_ptr(), a.k->const_data_ptr(), a.v->const_data_ptr(), o->const_data_ptr(),
                                 lse, go->const_data_ptr(), dlse, a.s, data(dq), data(dk), data(dv), (int)mode, data(ws),
                                 bytes, stream(a.index));
    }
  }
  if (status != STREAMKL_OK) Py_RETURN_NONE;
  return tuple({dq, dk, dv});
  END_HANDLE_TH_ERRORS
}

struct Logits {
  const at::Tensor* x;
  int index, type;
  long long rows, V, stride;
  const long long* tokens;
  at::IntArrayRef token_sizes, lead;
  int T;
  double scale;
};

// logits, tokens and scale at args[0], [1] and `at`.
bool logits(PyObject* const* args, int at, Logits* l) {
  l->x = tensor(args[0]);
  if (!l->x || !l->x->is_cuda() || l->x->dim() < 1 || l->x->numel() == 0) return false;
  l->index = l->x->get_device();
  if (l->index != c10::cuda::current_device()) return false;
  const auto type = l->x->scalar_type();
  if (type != at::kBFloat16 && type != at::kHalf && type != at::kFloat) return false;
  l->type = type == at::kBFloat16 ? STREAMKL_BF16 : type == at::kHalf ? STREAMKL_FP16 : STREAMKL_FP32;
  const auto size = l->x->sizes();
  l->lead = size.slice(0, size.size() - 1);
  l->V = size.back();
  l->rows = l->x->numel() / l->V;
  l->stride = l->V;
  if (!l->x->is_contiguous()) {
    if (size.size() != 2 || l->x->stride(1) != 1 || l->x->stride(0) < l->V) return false;
    l->stride = l->x->stride(0);
  }
  l->T = 0;
  l->tokens = nullptr;
  if (args[1] != Py_None) {
    const at::Tensor* t = tensor(args[1]);
    if (!t || t->scalar_type() != at::kLong || !on_device(*t, l->index) || !t->is_contiguous()) return false;
    l->token_sizes = t->sizes();
    if (t->sizes() == l->lead)
      l->T = 1;
    else if (t->dim() == l->x->dim() && t->sizes().slice(0, t->dim() - 1) == l->lead && t->sizes().back() <= INT_MAX)
      l->T = (int)t->sizes().back();
    else
      return false;
    if (l->T == 0) return false;
    l->tokens = reinterpret_cast<const long long*>(t->const_data_ptr());
  }
  if (!PyFloat_Check(args[at])) return false;
  l->scale = PyFloat_AS_DOUBLE(args[at]);
  return true;
}

// logprobs_fwd(logits, tokens, scale, top_k)
PyObject* logprobs_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Logits l;
  if (n != 4 || !logits(args, 2, &l) || l.T == 0 || !PyLong_Check(args[3])) Py_RETURN_NONE;
  const long k = PyLong_AsLong(args[3]);
  if (k < 0 || k > STREAMKL_LOGPROBS_MAX_TOP_K || k > l.V) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  c10::SmallVector<int64_t, 8> top_sizes(l.lead.begin(), l.lead.end());
  top_sizes.push_back(k);
  const auto f32 = options(at::kFloat, l.index);
  at::Tensor logp, entropy, lse, top, index;
  int status;
  {
    NoGil no_gil;
    logp = at::empty(l.token_sizes, f32);
    entropy = at::empty(l.lead, f32);
    lse = at::empty(l.lead, f32);
    top = at::empty(top_sizes, f32);
    index = at::empty(top_sizes, options(at::kLong, l.index));
    status = streamkl_logprobs_fwd(l.x->const_data_ptr(), l.type, l.rows, l.V, l.stride, l.tokens, l.T, (float)l.scale,
                                   (int)k, static_cast<float*>(data(logp)), static_cast<float*>(data(entropy)),
                                   static_cast<float*>(data(lse)), static_cast<float*>(data(top)),
                                   static_cast<long long*>(data(index)), stream(l.index));
  }
  if (status != STREAMKL_OK) Py_RETURN_NONE;
  return tuple({logp, entropy, lse, top, index});
  END_HANDLE_TH_ERRORS
}

// logprobs_bwd(logits, tokens, lse, entropy, g_logp, g_entropy, scale)
PyObject* logprobs_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Logits l;
  if (n != 7 || !logits(args, 6, &l) || l.T == 0) Py_RETURN_NONE;
  const float *lse, *entropy = nullptr, *g, *gh;
  if (args[2] == Py_None || args[4] == Py_None || !rows(args[2], l.lead, l.index, &lse) ||
      !rows(args[4], l.token_sizes, l.index, &g) || !rows(args[5], l.lead, l.index, &gh))
    Py_RETURN_NONE;
  if (gh && (args[3] == Py_None || !rows(args[3], l.lead, l.index, &entropy))) Py_RETURN_NONE;
  at::Tensor out;
  int status;
  {
    NoGil no_gil;
    out = at::empty(l.x->sizes(), options(l.x->scalar_type(), l.index));
    status = streamkl_logprobs_bwd(l.x->const_data_ptr(), l.type, l.rows, l.V, l.stride, l.tokens, l.T, (float)l.scale, lse,
                                   entropy, g, gh, data(out), l.V, stream(l.index));
  }
  if (status != STREAMKL_OK) Py_RETURN_NONE;
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(F));
}

PyMethodDef kMethods[] = {{"attn_fwd", fast<attn_fwd>(), METH_FASTCALL, nullptr},
                          {"attn_bwd", fast<attn_bwd>(), METH_FASTCALL, nullptr},
                          {"logprobs_fwd", fast<logprobs_fwd>(), METH_FASTCALL, nullptr},
                          {"logprobs_bwd", fast<logprobs_bwd>(), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&kModule); }
