// The Python calls that are made per layer and per token, without Python's own
// time: a CPython module that checks a call's tensors, allocates its outputs and
// workspace, and calls libstreamkl.  It takes the ordinary case (device tensors
// of the current device, in a layout the library reads in place) and returns
// None for everything else: _lib.py then goes through the same call step by
// step, copies what has to be copied, and reports what is wrong.  A call's host
// time against the ctypes path's: attention forward 7 to 8 us against 24, its
// backward 13 to 14 against 37, log probabilities 9 to 10 against 24, their gradient
// 4 to 5 against 18, rotary positions 8 against 22, differential attention 7 against 36 and its
// backward 15 against 56, the vocabulary's cross entropy 10 against 30 and its gradients
// 14 against 39; the short calls' kernels take 4 to 18 us.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
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

// The difference's head count, weights and layout: H differences of two maps each in a.s.  lam is read with the strides that
// broadcasting it gives.
bool difference(const Attention& a, PyObject* lam, streamkl_diff_attn_shape* s) {
  const at::Tensor* l = tensor(lam);
  const int64_t size[3] = {a.s.B, a.s.H / 2, a.s.NQ};
  if (!l || l->scalar_type() != at::kFloat || !on_device(*l, a.index) || l->dim() > 3 || l->dim() < 1 || a.s.H % 2 ||
      a.s.H / 2 % a.s.HK)
    return false;
  long long stride[3] = {0, 0, 0};
  for (int64_t i = 0; i < l->dim(); ++i) {
    const int64_t to = 3 - l->dim() + i;
    if (l->size(i) == size[to])
      stride[to] = l->stride(i);
    else if (l->size(i) != 1)
      return false;
  }
  *s = streamkl_diff_attn_shape{a.s, l->const_data_ptr<float>(), stride[0], stride[1], stride[2], 0, 0, 0};
  return true;
}

// diff_attn_fwd(q, k, v, lam, scale, causal, q_lens, k_lens, return_maps)
PyObject* diff_attn_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Attention a;
  streamkl_diff_attn_shape s;
  if (n != 9 || !attention(args, 4, &a) || !difference(a, args[3], &s) || !PyBool_Check(args[8])) Py_RETURN_NONE;
  const bool with_maps = args[8] == Py_True;
  at::Tensor d, lse, maps, rest;
  int status;
  {
    NoGil no_gil;
    size_t bytes = 0;
    if (with_maps) {
      maps = like(*a.q, a.qs, a.index);
      rest = like(*a.q, a.qs, a.index);
      s.maps.o_rest = data(rest);
    }
    const auto bf16 = options(at::kBFloat16, a.index);
    const long long B = a.s.B, H = a.s.H / 2, N = a.s.NQ, D = a.s.D;
    if (H > 1 && a.qs.h < a.qs.n) {  // rows before heads, as q has them
      d = at::empty_strided({B, H, N, D}, {N * H * D, D, H * D, 1}, bf16);
      s.d_stride_b = N * H * D;
      s.d_stride_h = D;
      s.d_stride_n = H * D;
    } else {
      d = at::empty({B, H, N, D}, bf16);
    }
    status = streamkl_diff_attn_fwd_workspace(s, &bytes);
    if (status == STREAMKL_OK) {
      const at::Tensor ws = workspace(bytes, a.index);
      lse = at::empty({a.s.B, a.s.H, a.s.NQ}, options(at::kFloat, a.index));
      status = streamkl_diff_attn_fwd(a.q->const_data_ptr(), a.k->const_data_ptr(), a.v->const_data_ptr(), s, data(d), data(maps),
                                      static_cast<float*>(data(lse)), data(ws), bytes, stream(a.index));
    }
  }
  if (status != STREAMKL_OK) Py_RETURN_NONE;
  return with_maps ? tuple({d, lse, maps, rest}) : tuple({d, lse});
  END_HANDLE_TH_ERRORS
}

// diff_attn_bwd(q, k, v, lam, maps, lse, do, dlse, scale, causal, q_lens, k_lens, bwd_mode, maps_rest)
PyObject* diff_attn_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Attention a;
  streamkl_diff_attn_shape s;
  if (n != 14 || !attention(args, 8, &a) || !difference(a, args[3], &s)) Py_RETURN_NONE;
  const at::Tensor *maps = tensor(args[4]), *go = tensor(args[6]), *rest = tensor(args[13]);
  Strides os, rs, gs;
  if (!maps || !go || !rest || !on_device(*maps, a.index) || !on_device(*go, a.index) || !on_device(*rest, a.index) ||
      maps->sizes() != a.q->sizes() || rest->sizes() != a.q->sizes() || !layout(*maps, &os) || !layout(*rest, &rs) ||
      os.b != rs.b || os.h != rs.h || os.n != rs.n || !layout(*go, &gs))
    Py_RETURN_NONE;
  const int64_t d_sizes[4] = {a.s.B, a.s.H / 2, a.s.NQ, a.s.D};
  if (go->sizes() != at::IntArrayRef(d_sizes, 4)) Py_RETURN_NONE;
  s.maps.o_stride_b = os.b;
  s.maps.o_stride_h = os.h;
  s.maps.o_stride_n = os.n;
  s.maps.o_rest = const_cast<void*>(rest->const_data_ptr());  // read only
  s.d_stride_b = gs.b;
  s.d_stride_h = gs.h;
  s.d_stride_n = gs.n;
  const float *lse, *dlse;
  const auto row_sizes = a.q->sizes().slice(0, 3);
  if (args[5] == Py_None || !rows(args[5], row_sizes, a.index, &lse) || !rows(args[7], row_sizes, a.index, &dlse) ||
      !PyLong_Check(args[12]))
    Py_RETURN_NONE;
  const long mode = PyLong_AsLong(args[12]);
  if (mode < 0 || mode > INT_MAX) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  at::Tensor dq, dk, dv, dlam;
  int status;
  {
    NoGil no_gil;
    size_t bytes = 0;
    status = streamkl_diff_attn_bwd_workspace(s, (int)mode, &bytes);
    if (status == STREAMKL_OK) {
      const at::Tensor ws = workspace(bytes, a.index);
      dq = like(*a.q, a.qs, a.index);
      dk = like(*a.k, a.ks, a.index);
      dv = like(*a.v, a.vs, a.index);
      dlam = at::empty({a.s.B, a.s.H / 2, a.s.NQ}, options(at::kFloat, a.index));
      status = streamkl_diff_attn_bwd(a.q->const_data_ptr(), a.k->const_data_ptr(), a.v->const_data_ptr(), maps->const_data_ptr(),
                                      lse, go->const_data_ptr(), dlse, s, data(dq), data(dk), data(dv),
                                      static_cast<float*>(data(dlam)), (int)mode, data(ws), bytes, stream(a.index));
    }
  }
  if (status != STREAMKL_OK) Py_RETURN_NONE;
  return tuple({dq, dk, dv, dlam});
  END_HANDLE_TH_ERRORS
}

bool real_type(at::ScalarType type, int* out) {
  *out = type == at::kBFloat16 ? STREAMKL_BF16 : type == at::kHalf ? STREAMKL_FP16 : STREAMKL_FP32;
  return type == at::kBFloat16 || type == at::kHalf || type == at::kFloat;
}

// rotary(q, k, turns, dim, amplitude, positions, offset, interleaved, inverse), q and k both there
PyObject* rotary(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) Py_RETURN_NONE;
  const at::Tensor *x[2] = {tensor(args[0]), tensor(args[1])}, *turns = tensor(args[2]);
  if (!x[0] || !x[1] || !turns || !x[0]->is_cuda()) Py_RETURN_NONE;
  const int index = x[0]->get_device();
  streamkl_rotary_shape s{};
  if (index != c10::cuda::current_device() || !on_device(*x[1], index) || !on_device(*turns, index) ||
      !real_type(x[0]->scalar_type(), &s.dtype) || x[1]->scalar_type() != x[0]->scalar_type() || turns->scalar_type() != at::kLong)
    Py_RETURN_NONE;
  for (const at::Tensor* t : x) {
    if (t->dim() != 4 || t->numel() == 0 || t->stride(3) != 1) Py_RETURN_NONE;
    for (int i = 0; i < 4; ++i)
      if (t->size(i) > INT_MAX || t->stride(i) <= 0 || t->size(i) != (i == 1 ? t->size(i) : x[0]->size(i))) Py_RETURN_NONE;
  }
  if (!PyLong_Check(args[3]) || !PyFloat_Check(args[4]) || !PyLong_Check(args[6]) || !PyBool_Check(args[7]) || !PyBool_Check(args[8]))
    Py_RETURN_NONE;
  const long dim = PyLong_AsLong(args[3]);
  const long long offset = PyLong_AsLongLong(args[6]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  s.B = (int)x[0]->size(0);
  s.HQ = (int)x[0]->size(1);
  s.HK = (int)x[1]->size(1);
  s.N = (int)x[0]->size(2);
  s.D = (int)x[0]->size(3);
  if (dim <= 0 || dim > s.D || turns->numel() != dim / 2 || !turns->is_contiguous()) Py_RETURN_NONE;
  s.dim = (int)dim;
  s.interleaved = args[7] == Py_True;
  s.amplitude = (float)PyFloat_AS_DOUBLE(args[4]);
  s.offset = offset;
  if (args[5] != Py_None) {
    const at::Tensor* p = tensor(args[5]);
    if (!p || offset || !on_device(*p, index) || (p->scalar_type() != at::kLong && p->scalar_type() != at::kInt) || p->dim() < 1 ||
        p->dim() > 2 || p->size(p->dim() - 1) != s.N || (p->dim() == 2 && p->size(0) != s.B) ||
        (s.N > 1 && p->stride(p->dim() - 1) != 1))
      Py_RETURN_NONE;
    s.positions = p->const_data_ptr();
    s.positions_bytes = p->scalar_type() == at::kLong ? 8 : 4;
    s.positions_stride = p->dim() == 2 && s.B > 1 ? p->stride(0) : 0;
  }
  at::Tensor out[2];
  int status;
  {
    NoGil no_gil;
    for (int i = 0; i < 2; ++i)
      out[i] = x[i]->is_contiguous() ? at::empty(x[i]->sizes(), options(x[i]->scalar_type(), index)) : at::empty_like(*x[i]);
    auto put = [](const at::Tensor& t, long long* b, long long* h, long long* r) {
      *b = t.stride(0);
      *h = t.stride(1);
      *r = t.stride(2);
    };
    put(*x[0], &s.q_stride_b, &s.q_stride_h, &s.q_stride_n);
    put(*x[1], &s.k_stride_b, &s.k_stride_h, &s.k_stride_n);
    put(out[0], &s.q_out_stride_b, &s.q_out_stride_h, &s.q_out_stride_n);
    put(out[1], &s.k_out_stride_b, &s.k_out_stride_h, &s.k_out_stride_n);
    status = streamkl_rotary(x[0]->const_data_ptr(), x[1]->const_data_ptr(), s,
                             reinterpret_cast<const unsigned long long*>(turns->const_data_ptr()), data(out[0]), data(out[1]),
                             args[8] == Py_True, stream(index));
  }
  if (status != STREAMKL_OK) Py_RETURN_NONE;
  return tuple({out[0], out[1]});
  END_HANDLE_TH_ERRORS
}

struct Xent {
  const at::Tensor *hidden, *weight;
  const long long* tokens;
  at::IntArrayRef lead;
  int index;
  streamkl_xent_shape s;
};

// hidden, weight, tokens at args[0..2], scale at args[`at`].
bool xent(PyObject* const* args, int at, Xent* x) {
  x->hidden = tensor(args[0]);
  x->weight = tensor(args[1]);
  const at::Tensor* t = tensor(args[2]);
  if (!x->hidden || !x->weight || !t || !x->hidden->is_cuda() || x->hidden->numel() == 0 || x->hidden->dim() < 1) return false;
  x->index = x->hidden->get_device();
  const auto type = x->hidden->scalar_type();
  if (x->index != c10::cuda::current_device() || !on_device(*x->weight, x->index) || !on_device(*t, x->index) ||
      (type != at::kBFloat16 && type != at::kHalf) || x->weight->scalar_type() != type || x->weight->dim() != 2)
    return false;
  const auto size = x->hidden->sizes();
  x->lead = size.slice(0, size.size() - 1);
  const int64_t C = size.back();
  if (x->weight->size(1) != C || x->weight->size(0) == 0 || C > INT_MAX || t->scalar_type() != at::kLong || t->sizes() != x->lead ||
      !t->is_contiguous() || !PyFloat_Check(args[at]))
    return false;
  auto place = [](const at::Tensor& m) { return (reinterpret_cast<uintptr_t>(m.const_data_ptr()) & 15) == 0; };
  long long hs = C;
  if (!x->hidden->is_contiguous()) {
    if (size.size() != 2 || x->hidden->stride(1) != 1 || x->hidden->stride(0) < C || x->hidden->stride(0) % 8) return false;
    hs = x->hidden->stride(0);
  }
  const long long ws = x->weight->is_contiguous() ? C : x->weight->stride(0);
  if (x->weight->stride(1) != 1 || ws < C || ws % 8 || C % 8 || !place(*x->hidden) || !place(*x->weight)) return false;
  x->tokens = reinterpret_cast<const long long*>(t->const_data_ptr());
  x->s = streamkl_xent_shape{x->hidden->numel() / C, x->weight->size(0), (int)C, type == at::kHalf ? STREAMKL_FP16 : STREAMKL_BF16,
                             (float)PyFloat_AS_DOUBLE(args[at]), hs, ws};
  return true;
}

// vocab_xent_fwd(hidden, weight, tokens, scale)
PyObject* vocab_xent_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Xent x;
  if (n != 4 || !xent(args, 3, &x)) Py_RETURN_NONE;
  at::Tensor loss, lse;
  int status;
  {
    NoGil no_gil;
    size_t bytes = 0;
    status = streamkl_vocab_xent_fwd_workspace(x.s, &bytes);
    if (status == STREAMKL_OK) {
      const at::Tensor ws = workspace(bytes, x.index);
      loss = at::empty(x.lead, options(at::kFloat, x.index));
      lse = at::empty(x.lead, options(at::kFloat, x.index));
      status = streamkl_vocab_xent_fwd(x.hidden->const_data_ptr(), x.weight->const_data_ptr(), x.tokens, x.s,
                                       static_cast<float*>(data(loss)), static_cast<float*>(data(lse)), data(ws), bytes,
                                       stream(x.index));
    }
  }
  if (status != STREAMKL_OK) Py_RETURN_NONE;
  return tuple({loss, lse});
  END_HANDLE_TH_ERRORS
}

// vocab_xent_bwd(hidden, weight, tokens, lse, g_loss, g_lse, scale), both gradients
PyObject* vocab_xent_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Xent x;
  if (n != 7 || !xent(args, 6, &x)) Py_RETURN_NONE;
  const float *lse, *g, *gl;
  if (args[3] == Py_None || args[4] == Py_None || !rows(args[3], x.lead, x.index, &lse) || !rows(args[4], x.lead, x.index, &g) ||
      !rows(args[5], x.lead, x.index, &gl))
    Py_RETURN_NONE;
  at::Tensor dh, dw;
  int status;
  {
    NoGil no_gil;
    size_t bytes = 0;
    status = streamkl_vocab_xent_bwd_workspace(x.s, 1, 1, &bytes);
    if (status == STREAMKL_OK) {
      const at::Tensor ws = workspace(bytes, x.index);
      dh = at::empty(x.hidden->sizes(), options(x.hidden->scalar_type(), x.index));
      dw = at::empty(x.weight->sizes(), options(x.hidden->scalar_type(), x.index));
      status = streamkl_vocab_xent_bwd(x.hidden->const_data_ptr(), x.weight->const_data_ptr(), x.tokens, lse, g, gl, x.s, data(dh),
                                       data(dw), data(ws), bytes, stream(x.index));
    }
  }
  if (status != STREAMKL_OK) Py_RETURN_NONE;
  return tuple({dh, dw});
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
                          {"diff_attn_fwd", fast<diff_attn_fwd>(), METH_FASTCALL, nullptr},
                          {"diff_attn_bwd", fast<diff_attn_bwd>(), METH_FASTCALL, nullptr},
                          {"rotary", fast<rotary>(), METH_FASTCALL, nullptr},
                          {"vocab_xent_fwd", fast<vocab_xent_fwd>(), METH_FASTCALL, nullptr},
                          {"vocab_xent_bwd", fast<vocab_xent_bwd>(), METH_FASTCALL, nullptr},
                          {"logprobs_fwd", fast<logprobs_fwd>(), METH_FASTCALL, nullptr},
                          {"logprobs_bwd", fast<logprobs_bwd>(), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&kModule); }
