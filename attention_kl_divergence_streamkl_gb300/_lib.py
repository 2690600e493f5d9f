"""Python binding of libstreamkl (argument marshalling only), through ctypes.

Every step of the computation runs in the CUDA kernels of ``libstreamkl.so``;
this module only checks tensor metadata, allocates outputs and workspaces
through PyTorch's CUDA allocator, and passes raw pointers and the current CUDA
stream to the C entry points of the same names.  There is no CPU fallback: if
the library is missing, every call raises.  The entry points that a model calls
per layer and per token (attn_fwd, attn_bwd, diff_attn_fwd, diff_attn_bwd, rotary_fwd,
rotary_bwd, logprobs_fwd, logprobs_bwd, vocab_xent_fwd, vocab_xent_bwd) go to
the native caller first (csrc/calls.cpp, _calls.so), which does the same for
tensors that need no copy in a third of the time, and come back here for the rest.

Inputs given as CPU tensors are copied to the current CUDA device on the
current stream (non-blocking from pinned memory) and the results are copied
back, so a host caller uses the same functions.

Device inputs need not be contiguous: any [B, H, N, D] view whose D is
contiguous, whose other strides are multiples of 8 elements and whose rows do
not overlap (a [B, N, H, D] tensor permuted, a slice of a packed QKV tensor) is
passed as it is, with its strides; the gradients come back with the strides of
the input they belong to.  Other views are copied to a contiguous tensor first.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libstreamkl.so")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_SCRATCH_LIMIT = range(7)
BWD_AUTO, BWD_FUSED, BWD_SEPARATE, BWD_DQ_ONLY, BWD_DK_ONLY = 0, 1, 2, 3, 4
SPLITK_MAX_NQ = 16
LOGPROBS_MAX_TOP_K = 32
ATTN_EXACT_KEYS = 64  # up to so many keys (N_K) the attention backward forms its row sums without o
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # streamkl_dtype


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("NQ", ctypes.c_int), ("NK", ctypes.c_int),
                ("D", ctypes.c_int), ("scale", ctypes.c_float), ("causal", ctypes.c_int),
                ("q_stride_b", ctypes.c_longlong), ("q_stride_h", ctypes.c_longlong),
                ("q_stride_n", ctypes.c_longlong), ("k_stride_b", ctypes.c_longlong),
                ("k_stride_h", ctypes.c_longlong), ("k_stride_n", ctypes.c_longlong)]


class AttnShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("HK", ctypes.c_int), ("NQ", ctypes.c_int), ("NK", ctypes.c_int),
                ("D", ctypes.c_int), ("scale", ctypes.c_float), ("causal", ctypes.c_int), ("q_lens", ctypes.c_void_p),
                ("k_lens", ctypes.c_void_p)] + [(f"{t}_stride_{x}", ctypes.c_longlong) for t in "qkvo" for x in "bhn"] + [("o_rest", ctypes.c_void_p)]


class DiffAttnShape(ctypes.Structure):
    _fields_ = [("maps", AttnShape), ("lam", ctypes.c_void_p)] + [
        (f"{t}_stride_{x}", ctypes.c_longlong) for t in ("lam", "d") for x in "bhn"]


class RotaryShape(ctypes.Structure):
    _fields_ = [(x, ctypes.c_int) for x in ("B", "HQ", "HK", "N", "D", "dim", "dtype", "interleaved")] + [
        ("amplitude", ctypes.c_float), ("offset", ctypes.c_longlong), ("positions", ctypes.c_void_p),
        ("positions_bytes", ctypes.c_int), ("positions_stride", ctypes.c_longlong)] + [
        (f"{t}_stride_{x}", ctypes.c_longlong) for t in ("q", "k", "q_out", "k_out") for x in "bhn"]


class XentShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("vocab", ctypes.c_longlong), ("channels", ctypes.c_int), ("dtype", ctypes.c_int),
                ("scale", ctypes.c_float), ("hidden_stride", ctypes.c_longlong), ("weight_stride", ctypes.c_longlong)]


class StreamKLError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


_P, _F, _S, _I, _SZ = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_LL = ctypes.c_longlong
# name -> (restype, argtypes); also the list of symbols include/streamkl.h declares
SIGNATURES = {
    "streamkl_fwd": (_I, [_P, _P, _P, _P, Shape, _F, _F, _F, _S]),
    "streamkl_fwd_splitk_workspace": (_I, [Shape, _I, ctypes.POINTER(_SZ)]),
    "streamkl_fwd_splitk": (_I, [_P, _P, _P, _P, Shape, _I, _P, _SZ, _F, _F, _F, _S]),
    "streamkl_fwd_splitk_plan": (_I, [Shape, _I, ctypes.POINTER(_I)]),
    "streamkl_fwd_splitk_noalloc": (_I, [_P, _P, _P, _P, Shape, _I, _F, _F, _F, _S]),
    "streamkl_fwd_partials": (_I, [_P, _P, _P, _P, Shape, _LL, _LL, _F, _S]),
    "streamkl_merge_partials": (_I, [_F, _I, Shape, _F, _F, _F, _S]),
    "streamkl_bwd_keyshard_workspace": (_I, [Shape, _LL, _LL, ctypes.POINTER(_SZ)]),
    "streamkl_bwd_keyshard": (_I, [_I, _P, _P, _P, _P, Shape, _LL, _LL, _F, _F, _F, _F, _F, _P, _P, _SZ, _S]),
    "streamkl_dq_from_partial": (_I, [_F, Shape, _P, _S]),
    "streamkl_bwd_workspace": (_I, [Shape, _I, ctypes.POINTER(_SZ)]),
    "streamkl_bwd_select": (_I, [Shape, _SZ, _I]),
    "streamkl_bwd_fused_plan": (_I, [Shape, _SZ, _I, ctypes.POINTER(_I), ctypes.POINTER(_SZ)]),
    "streamkl_bwd_s1": (_I, [_P, _P, _P, _P, Shape, _F, _F, _F, _P, _P, _I, _P, _SZ, _S]),
    "streamkl_bwd_s2": (_I, [_P, _P, _P, _P, Shape, _F, _F, _F, _F, _P, _P, _I, _P, _SZ, _S]),
    "streamkl_bwd_mutual": (_I, [_P, _P, _P, _P, Shape, _F, _F, _F, _F, _P, _P, _P, _P, _I, _P, _SZ, _S]),
    "streamkl_bwd_mutual_select": (_I, [Shape, _SZ, _I]),
    "streamkl_bwd_mutual_workspace": (_I, [Shape, _I, ctypes.POINTER(_SZ)]),
    "streamkl_attn_fwd_workspace": (_I, [AttnShape, ctypes.POINTER(_SZ)]),
    "streamkl_attn_fwd_plan": (_I, [AttnShape, _I, ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "streamkl_attn_fwd": (_I, [_P, _P, _P, AttnShape, _P, _F, _P, _SZ, _S]),
    "streamkl_attn_bwd_plan": (_I, [AttnShape, _I, _I, *[ctypes.POINTER(_I)] * 3, ctypes.POINTER(_SZ)]),
    "streamkl_attn_bwd_workspace": (_I, [AttnShape, _I, ctypes.POINTER(_SZ)]),
    "streamkl_attn_bwd": (_I, [_P, _P, _P, _P, _F, _P, _F, AttnShape, _P, _P, _P, _I, _P, _SZ, _S]),
    "streamkl_logprobs_fwd": (_I, [_P, _I, _LL, _LL, _LL, _P, _I, ctypes.c_float, _I, _F, _F, _F, _F, _P, _S]),
    "streamkl_logprobs_bwd": (_I, [_P, _I, _LL, _LL, _LL, _P, _I, ctypes.c_float, _F, _F, _F, _F, _P, _LL, _S]),
    "streamkl_diff_attn_fwd_plan": (_I, [DiffAttnShape, _I, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_SZ)]),
    "streamkl_diff_attn_fwd_workspace": (_I, [DiffAttnShape, ctypes.POINTER(_SZ)]),
    "streamkl_diff_attn_fwd": (_I, [_P, _P, _P, DiffAttnShape, _P, _P, _F, _P, _SZ, _S]),
    "streamkl_diff_attn_bwd_workspace": (_I, [DiffAttnShape, _I, ctypes.POINTER(_SZ)]),
    "streamkl_diff_attn_bwd": (_I, [_P, _P, _P, _P, _F, _P, _F, DiffAttnShape, _P, _P, _P, _F, _I, _P, _SZ, _S]),
    "streamkl_rotary": (_I, [_P, _P, RotaryShape, _P, _P, _P, _I, _S]),
    "streamkl_vocab_xent_fwd_plan": (_I, [XentShape, _I, ctypes.POINTER(_I), ctypes.POINTER(_SZ)]),
    "streamkl_vocab_xent_fwd_workspace": (_I, [XentShape, ctypes.POINTER(_SZ)]),
    "streamkl_vocab_xent_fwd": (_I, [_P, _P, _P, XentShape, _F, _F, _P, _SZ, _S]),
    "streamkl_vocab_xent_bwd_plan": (_I, [XentShape, _I, _I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_SZ)]),
    "streamkl_vocab_xent_bwd_workspace": (_I, [XentShape, _I, _I, ctypes.POINTER(_SZ)]),
    "streamkl_vocab_xent_bwd": (_I, [_P, _P, _P, _F, _F, _F, XentShape, _P, _P, _P, _SZ, _S]),
    "streamkl_status_string": (ctypes.c_char_p, [_I]),
    "streamkl_check_device_status": (_I, [_S]),
    "streamkl_debug_wait_timeout": (_I, [_I, _S]),
    "streamkl_version": (_I, []),
}

_lib: Optional[ctypes.CDLL] = None
_calls = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libstreamkl.so not found at {LIB_PATH}: build it with "
                               "attention_kl_divergence_streamkl_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def calls():
    """The native caller of the per-layer entry points (csrc/calls.cpp); raises if it has not been built."""
    global _calls
    if _calls is None:
        lib()
        try:
            from . import _calls as module
        except ImportError as e:
            raise RuntimeError("_calls.so is missing or does not load: build it with "
                               f"attention_kl_divergence_streamkl_gb300.build.build() ({e})") from e
        _calls = module
    return _calls


def status_string(status: int) -> str:
    return lib().streamkl_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != OK:
        raise StreamKLError(status, where)


def make_shape(B, H, NQ, NK, D, scale=None, causal=False, q_strides=(0, 0, 0), k_strides=(0, 0, 0)) -> Shape:
    """The C shape; q_strides / k_strides are element strides along (b, h, n), zeros = contiguous."""
    return Shape(int(B), int(H), int(NQ), int(NK), int(D), float(scale or 0.0), int(bool(causal)),
                 *(int(x) for x in q_strides), *(int(x) for x in k_strides))


def _bhn_strides(t: torch.Tensor):
    """(b, h, n) element strides under which the library can read `t` in place, else None.

    D must be contiguous, the start 16-byte aligned, each stride of an extent > 1
    a positive multiple of 8 elements and the rows pairwise disjoint (sorted by
    stride, each stride covers the extent below it).  The stride of an extent-1
    dimension is never used to address anything; it is replaced by a valid one.
    """
    B, H, N, D = t.shape
    if t.numel() == 0:  # nothing is read; any valid strides do
        return max(H, 1) * max(N, 1) * D, max(N, 1) * D, D
    if t.stride(3) != 1 or t.data_ptr() % 16:
        return None
    dims = [(t.stride(i), t.size(i)) for i in range(4) if t.size(i) > 1]
    if any(st <= 0 for st, _ in dims):
        return None
    span = 0
    for st, n in sorted(dims):
        if st < span:
            return None
        span = st * n
    sn = t.stride(2) if t.size(2) > 1 else D
    sh = t.stride(1) if t.size(1) > 1 else 8
    sb = t.stride(0) if t.size(0) > 1 else 8
    if sn < D or any(x % 8 for x in (sb, sh, sn)):
        return None
    return sb, sh, sn


def _pair(a: torch.Tensor, b: torch.Tensor):
    """The two tensors of a pair (Q1/Q2 or K1/K2) and their shared (b, h, n) strides."""
    sa, sb = _bhn_strides(a), _bhn_strides(b)
    if sa is None or sa != sb:
        a, b = a.contiguous(), b.contiguous()
        sa = _bhn_strides(a)
        if sa is None:
            raise ValueError("inputs must be 16-byte aligned")
    return a, b, sa


def _grad_like(t: torch.Tensor, strides, rows) -> torch.Tensor:
    """A bf16 output with the (b, h, n) strides the library writes `t`'s gradient with."""
    B, H, _, D = t.shape
    return torch.empty_strided((B, H, rows, D), (strides[0], strides[1], strides[2], 1), dtype=torch.bfloat16,
                               device=t.device)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _prep(q1, k1, q2, k2):
    """Validates the four inputs; returns (device tensors, was_host, q strides, k strides)."""
    ts = [q1, k1, q2, k2]
    for t in ts:
        if t.dtype != torch.bfloat16:
            raise TypeError("Q1, K1, Q2, K2 must be bfloat16")
        if t.dim() != 4:
            raise ValueError("Q1, K1, Q2, K2 must be [B, H, N, D]")
    if q1.shape != q2.shape or k1.shape != k2.shape or q1.shape[:2] != k1.shape[:2] or q1.shape[3] != k1.shape[3]:
        raise ValueError(f"shape mismatch: Q1 {tuple(q1.shape)} K1 {tuple(k1.shape)} "
                         f"Q2 {tuple(q2.shape)} K2 {tuple(k2.shape)}")
    host = q1.device.type == "cpu"
    if host:
        dev = torch.device("cuda", torch.cuda.current_device())
        ts = [t.contiguous().to(dev, non_blocking=True) for t in ts]
    elif any(t.device != ts[0].device for t in ts):
        raise ValueError("inputs on different devices")
    q1, q2, qs = _pair(ts[0], ts[2])
    k1, k2, ks = _pair(ts[1], ts[3])
    return [q1, k1, q2, k2], host, qs, ks


def _rows(t: Optional[torch.Tensor], dev, shape3, name):
    if t is None:
        return None
    if t.dtype != torch.float32 or tuple(t.shape) != tuple(shape3):
        raise ValueError(f"{name} must be float32 of shape {tuple(shape3)}")
    return t.to(dev, non_blocking=True).contiguous()


def _back(ts, host):
    if not host:
        return ts
    out = tuple(t.to("cpu", non_blocking=True) for t in ts)
    torch.cuda.current_stream().synchronize()
    return out


def fwd(q1, k1, q2, k2, scale=None, causal=False):
    """KL, LSE1, LSE2 fp32 [B, H, N_Q] (one-pass forward)."""
    (q1, k1, q2, k2), host, qs, ks = _prep(q1, k1, q2, k2)
    B, H, NQ, D = q1.shape
    s = make_shape(B, H, NQ, k1.shape[2], D, scale, causal, qs, ks)
    kl, l1, l2 = (torch.empty((B, H, NQ), dtype=torch.float32, device=q1.device) for _ in range(3))
    _check(lib().streamkl_fwd(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), s, _ptr(kl), _ptr(l1), _ptr(l2),
                              _stream(q1.device)), "streamkl_fwd")
    return _back((kl, l1, l2), host)


def splitk_plan(B, H, NQ, NK, D, num_sms=0, causal=False) -> int:
    n = ctypes.c_int(0)
    _check(lib().streamkl_fwd_splitk_plan(make_shape(B, H, NQ, NK, D, None, causal), int(num_sms),
                                          ctypes.byref(n)), "streamkl_fwd_splitk_plan")
    return n.value


def fwd_splitk(q1, k1, q2, k2, scale=None, causal=False, num_splits=0):
    """Split-K forward for N_Q <= 16: KL, LSE1, LSE2 fp32 [B, H, N_Q]."""
    (q1, k1, q2, k2), host, qs, ks = _prep(q1, k1, q2, k2)
    B, H, NQ, D = q1.shape
    s = make_shape(B, H, NQ, k1.shape[2], D, scale, causal, qs, ks)
    nbytes = ctypes.c_size_t(0)
    _check(lib().streamkl_fwd_splitk_workspace(s, int(num_splits), ctypes.byref(nbytes)),
           "streamkl_fwd_splitk_workspace")
    ws = torch.empty(max(16, nbytes.value), dtype=torch.uint8, device=q1.device)
    kl, l1, l2 = (torch.empty((B, H, NQ), dtype=torch.float32, device=q1.device) for _ in range(3))
    _check(lib().streamkl_fwd_splitk(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), s, int(num_splits), _ptr(ws),
                                     nbytes.value, _ptr(kl), _ptr(l1), _ptr(l2), _stream(q1.device)),
           "streamkl_fwd_splitk")
    return _back((kl, l1, l2), host)


def fwd_partials(q1, k1, q2, k2, key_offset, nk_total, scale=None, causal=False):
    """Five scalars per row fp32 [B, H, N_Q, 5] over a key shard.

    k1, k2 hold the shard's keys, at global positions [key_offset, key_offset +
    k1.shape[2]) of a sequence of nk_total keys (the causal frontier is the
    global one).  Merge the shards' partials with merge_partials."""
    (q1, k1, q2, k2), host, qs, ks = _prep(q1, k1, q2, k2)
    B, H, NQ, D = q1.shape
    s = make_shape(B, H, NQ, k1.shape[2], D, scale, causal, qs, ks)
    part = torch.empty((B, H, NQ, 5), dtype=torch.float32, device=q1.device)
    _check(lib().streamkl_fwd_partials(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), s, int(key_offset), int(nk_total),
                                       _ptr(part), _stream(q1.device)), "streamkl_fwd_partials")
    return _back((part,), host)[0]


def merge_partials(parts, D, scale=None):
    """KL, LSE1, LSE2 fp32 [B, H, N_Q] from partial sets stacked as [S, B, H, N_Q, 5] (device)."""
    if parts.dtype != torch.float32 or parts.dim() != 5 or parts.shape[-1] != 5:
        raise ValueError("partials must be float32 [S, B, H, N_Q, 5]")
    parts = parts.contiguous()
    S, B, H, NQ, _ = parts.shape
    s = make_shape(B, H, NQ, 1, D, scale, False)
    kl, l1, l2 = (torch.empty((B, H, NQ), dtype=torch.float32, device=parts.device) for _ in range(3))
    _check(lib().streamkl_merge_partials(_ptr(parts), int(S), s, _ptr(kl), _ptr(l1), _ptr(l2),
                                         _stream(parts.device)), "streamkl_merge_partials")
    return kl, l1, l2


def bwd_keyshard(setting, q1, k1, q2, k2, key_offset, nk_total, lse1, lse2, kl, g, scale=None, causal=False):
    """Backward over a key shard: (unscaled fp32 dQ contribution [B, H, N_Q, D], bf16 dK of the shard's keys).

    lse1, lse2, kl are the merged values of the whole sequence; summing the
    dQ contributions of every shard and passing the sum to dq_from_partial gives dQ."""
    (q1, k1, q2, k2), host, qs, ks = _prep(q1, k1, q2, k2)
    B, H, NQ, D = q1.shape
    NK = k1.shape[2]
    dev = q1.device
    s = make_shape(B, H, NQ, NK, D, scale, causal, qs, ks)
    lse1 = _rows(lse1, dev, (B, H, NQ), "lse1")
    lse2 = _rows(lse2, dev, (B, H, NQ), "lse2")
    g = _rows(g, dev, (B, H, NQ), "g")
    kl = _rows(kl, dev, (B, H, NQ), "kl") if setting == 2 else None
    nbytes = ctypes.c_size_t(0)
    _check(lib().streamkl_bwd_keyshard_workspace(s, int(key_offset), int(nk_total), ctypes.byref(nbytes)),
           "streamkl_bwd_keyshard_workspace")
    ws = torch.empty(max(16, nbytes.value), dtype=torch.uint8, device=dev)
    dq = torch.empty((B, H, NQ, D), dtype=torch.float32, device=dev)
    dk = _grad_like(k1, ks, NK)
    _check(lib().streamkl_bwd_keyshard(int(setting), _ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), s, int(key_offset),
                                       int(nk_total), _ptr(lse1), _ptr(lse2), _ptr(kl), _ptr(g), _ptr(dq), _ptr(dk),
                                       _ptr(ws), nbytes.value, _stream(dev)), "streamkl_bwd_keyshard")
    return _back((dq, dk), host)


def dq_from_partial(dq_partial, q_like, scale=None):
    """bf16 dQ = scale * dq_partial, with the layout the library gives q_like's gradient."""
    if dq_partial.dtype != torch.float32 or dq_partial.dim() != 4:
        raise ValueError("dq_partial must be float32 [B, H, N_Q, D]")
    dq_partial = dq_partial.contiguous()
    B, H, NQ, D = dq_partial.shape
    qs = _bhn_strides(q_like) or (H * NQ * D, NQ * D, D)
    s = make_shape(B, H, NQ, 1, D, scale, False, qs)
    out = _grad_like(q_like, qs, NQ) if _bhn_strides(q_like) else torch.empty(
        (B, H, NQ, D), dtype=torch.bfloat16, device=dq_partial.device)
    _check(lib().streamkl_dq_from_partial(_ptr(dq_partial), s, _ptr(out), _stream(dq_partial.device)),
           "streamkl_dq_from_partial")
    return out


def bwd_select(B, H, NQ, NK, D, l2_bytes, num_sms, causal=False) -> int:
    return lib().streamkl_bwd_select(make_shape(B, H, NQ, NK, D, None, causal), int(l2_bytes), int(num_sms))


def bwd_fused_plan(B, H, NQ, NK, D, l2_bytes, num_sms, causal=False):
    """(key ranges, workspace bytes) of the fused backward on a device with this L2 and SM count."""
    n, ws = ctypes.c_int(0), ctypes.c_size_t(0)
    _check(lib().streamkl_bwd_fused_plan(make_shape(B, H, NQ, NK, D, None, causal), int(l2_bytes), int(num_sms),
                                         ctypes.byref(n), ctypes.byref(ws)), "streamkl_bwd_fused_plan")
    return n.value, ws.value


def bwd_workspace_bytes(B, H, NQ, NK, D, bwd_mode=BWD_AUTO, causal=False) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().streamkl_bwd_workspace(make_shape(B, H, NQ, NK, D, None, causal), int(bwd_mode),
                                        ctypes.byref(n)), "streamkl_bwd_workspace")
    return n.value


def _bwd(setting, q1, k1, q2, k2, lse1, lse2, kl, g, scale, causal, bwd_mode):
    (q1, k1, q2, k2), host, qs, ks = _prep(q1, k1, q2, k2)
    B, H, NQ, D = q1.shape
    NK = k1.shape[2]
    dev = q1.device
    s = make_shape(B, H, NQ, NK, D, scale, causal, qs, ks)
    lse1 = _rows(lse1, dev, (B, H, NQ), "lse1")
    lse2 = _rows(lse2, dev, (B, H, NQ), "lse2")
    g = _rows(g, dev, (B, H, NQ), "g")
    kl = _rows(kl, dev, (B, H, NQ), "kl") if setting == 2 else None
    nbytes = ctypes.c_size_t(0)
    _check(lib().streamkl_bwd_workspace(s, int(bwd_mode), ctypes.byref(nbytes)), "streamkl_bwd_workspace")
    ws = torch.empty(max(16, nbytes.value), dtype=torch.uint8, device=dev)
    dq = _grad_like(q1, qs, NQ) if bwd_mode != BWD_DK_ONLY else None
    dk = _grad_like(k1, ks, NK) if bwd_mode != BWD_DQ_ONLY else None
    if setting == 1:
        st = lib().streamkl_bwd_s1(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), s, _ptr(lse1), _ptr(lse2), _ptr(g),
                                   _ptr(dq), _ptr(dk), int(bwd_mode), _ptr(ws), nbytes.value, _stream(dev))
    else:
        st = lib().streamkl_bwd_s2(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), s, _ptr(lse1), _ptr(lse2), _ptr(kl),
                                   _ptr(g), _ptr(dq), _ptr(dk), int(bwd_mode), _ptr(ws), nbytes.value,
                                   _stream(dev))
    _check(st, f"streamkl_bwd_s{setting}")
    got = iter(_back(tuple(t for t in (dq, dk) if t is not None), host))
    return tuple(None if t is None else next(got) for t in (dq, dk))


def bwd_s1(q1, k1, q2, k2, lse1, lse2, g, scale=None, causal=False, bwd_mode=BWD_AUTO):
    """Setting 1 (P1 fixed): (dQ2, dK2) bf16."""
    return _bwd(1, q1, k1, q2, k2, lse1, lse2, None, g, scale, causal, bwd_mode)


def bwd_s2(q1, k1, q2, k2, lse1, lse2, kl, g, scale=None, causal=False, bwd_mode=BWD_AUTO):
    """Setting 2 (P2 fixed): (dQ1, dK1) bf16."""
    return _bwd(2, q1, k1, q2, k2, lse1, lse2, kl, g, scale, causal, bwd_mode)


def bwd_mutual_select(B, H, NQ, NK, D, l2_bytes, num_sms, causal=False) -> int:
    """AUTO's path for the mutual case (BWD_SEPARATE = the mutual kernels, BWD_FUSED = a fused pass per setting)."""
    return lib().streamkl_bwd_mutual_select(make_shape(B, H, NQ, NK, D, None, causal), int(l2_bytes), int(num_sms))


def bwd_mutual(q1, k1, q2, k2, lse1, lse2, kl, g, scale=None, causal=False, bwd_mode=BWD_AUTO):
    """Gradients of all four inputs (the mutual case): (dQ1, dK1, dQ2, dK2) bf16.

    bwd_mode BWD_SEPARATE rebuilds each logit tile pair once for both settings;
    BWD_FUSED runs one fused pass per setting; BWD_AUTO picks by shape.
    """
    (q1, k1, q2, k2), host, qs, ks = _prep(q1, k1, q2, k2)
    B, H, NQ, D = q1.shape
    NK = k1.shape[2]
    dev = q1.device
    s = make_shape(B, H, NQ, NK, D, scale, causal, qs, ks)
    lse1 = _rows(lse1, dev, (B, H, NQ), "lse1")
    lse2 = _rows(lse2, dev, (B, H, NQ), "lse2")
    kl = _rows(kl, dev, (B, H, NQ), "kl")
    g = _rows(g, dev, (B, H, NQ), "g")
    nbytes = ctypes.c_size_t(0)
    _check(lib().streamkl_bwd_mutual_workspace(s, int(bwd_mode), ctypes.byref(nbytes)),
           "streamkl_bwd_mutual_workspace")
    ws = torch.empty(max(16, nbytes.value), dtype=torch.uint8, device=dev)
    dq1, dq2 = _grad_like(q1, qs, NQ), _grad_like(q2, qs, NQ)
    dk1, dk2 = _grad_like(k1, ks, NK), _grad_like(k2, ks, NK)
    _check(lib().streamkl_bwd_mutual(_ptr(q1), _ptr(k1), _ptr(q2), _ptr(k2), s, _ptr(lse1), _ptr(lse2), _ptr(kl),
                                     _ptr(g), _ptr(dq1), _ptr(dk1), _ptr(dq2), _ptr(dk2), int(bwd_mode), _ptr(ws),
                                     nbytes.value, _stream(dev)),
           "streamkl_bwd_mutual")
    return _back((dq1, dk1, dq2, dk2), host)


def _call(name, index, *args):
    """Calls a C entry point on device `index`'s current stream, with that device current while it runs.

    Tensors go in as addresses (plain integers): these calls are made per layer and per token, where the binding's
    own time counts."""
    f = getattr(_lib or lib(), name)
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch.cuda.current_device():
        st = f(*args, stream)
    else:
        with torch.cuda.device(index):
            st = f(*args, stream)
    if st != OK:
        raise StreamKLError(st, name)


def _layout(t):
    """A [B, H, N, D] tensor the library can read and its (b, h, n) strides (a contiguous copy where it cannot)."""
    B, H, N, D = t.shape
    sb, sh, sn, sd = st = t.stride()
    if sd == 1 and not (t.data_ptr() & 15 or (sb | sh | sn) & 7) and (
            D <= sn and sn * N <= sh and sh * H <= sb or D <= sh and sh * H <= sn and sn * N <= sb) and sb < 1 << 38:
        return t, st[:3]  # heads by rows or rows by heads, the usual orders
    st = _bhn_strides(t)
    if st is None:
        t = t.clone(memory_format=torch.contiguous_format)  # also where only the start is off a 16-byte boundary
        st = _bhn_strides(t)
        if st is None:
            raise ValueError("the last dimension must be a multiple of 8")
    return t, st


def make_attn_shape(B, H, HK, NQ, NK, D, scale=None, causal=False, q_lens=None, k_lens=None, q_strides=(0, 0, 0),
                    k_strides=(0, 0, 0), v_strides=(0, 0, 0), o_strides=(0, 0, 0), o_rest=None) -> AttnShape:
    """The C shape of an attention; lens are int32 device tensors, o_rest one like o (kept alive by the caller), or None."""
    return AttnShape(B, H, HK, NQ, NK, D, scale or 0.0, bool(causal), None if q_lens is None else q_lens.data_ptr(),
                     None if k_lens is None else k_lens.data_ptr(), *q_strides, *k_strides, *v_strides, *o_strides,
                     None if o_rest is None else o_rest.data_ptr())


def _lens(t, B, dev, name):
    if t.dtype is not torch.int32 or t.shape != (B,):
        raise ValueError(f"{name} must be int32 of shape ({B},)")
    if t.device != dev:
        t = t.to(dev, non_blocking=True)
    return t if t.is_contiguous() else t.contiguous()


def _attn_inputs(tensors, q_lens, k_lens):
    """Validates an attention's tensors (q, k, v, and o, do, o_rest in the backward).

    Returns (the tensors on the device, q_lens, k_lens, (B, H, HK, NQ, NK, D), device, was_host)."""
    q, k, v = tensors[:3]
    shape, key_shape, dev = q.shape, k.shape, q.device
    for t in tensors:
        if t.dtype is not torch.bfloat16:
            raise TypeError("q, k, v, o, do, o_rest must be bfloat16")
        if t.device != dev:
            raise ValueError("inputs on different devices")
    if len(shape) != 4 or len(key_shape) != 4:
        raise ValueError("q must be [B, H, N_Q, D], k and v [B, HK, N_K, D]")
    B, H, NQ, D = shape
    Bk, HK, NK, Dk = key_shape
    if key_shape != v.shape or B != Bk or D != Dk:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)}")
    for t in tensors[3:]:
        if t.shape != shape:
            raise ValueError(f"o, do, o_rest must be {tuple(shape)}")
    if HK == 0 or H % HK:
        raise ValueError(f"{H} query heads do not divide over {HK} key heads")
    host = dev.type == "cpu"
    if host:
        dev = torch.device("cuda", torch.cuda.current_device())
        tensors = [t.contiguous().to(dev, non_blocking=True) for t in tensors]
    if q_lens is not None:
        q_lens = _lens(q_lens, B, dev, "q_lens")
    if k_lens is not None:
        k_lens = _lens(k_lens, B, dev, "k_lens")
    return tensors, q_lens, k_lens, (B, H, HK, NQ, NK, D), dev, host


def attn_fwd_plan(B, H, HK, NQ, NK, D, num_sms, causal=False):
    """(packed, key splits) of the attention forward on a device with num_sms SMs."""
    a, b = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().streamkl_attn_fwd_plan(make_attn_shape(B, H, HK, NQ, NK, D, None, causal), int(num_sms),
                                        ctypes.byref(a), ctypes.byref(b)), "streamkl_attn_fwd_plan")
    return bool(a.value), b.value


@functools.lru_cache(maxsize=1024)
def _attn_workspace(name, index, sizes, causal, *mode):
    """Workspace bytes of an attention of these sizes on device `index` (a pure rule of sizes and the device)."""
    n = ctypes.c_size_t(0)
    with torch.cuda.device(index):
        _check(getattr(lib(), name)(make_attn_shape(*sizes, None, causal), *mode, ctypes.byref(n)), name)
    return n.value


def attn_fwd(q, k, v, scale=None, causal=False, q_lens=None, k_lens=None, return_rest=False):
    """Attention: (o bf16 with q's layout, lse fp32 [B, H, N_Q]).

    q: [B, H, N_Q, D], k and v: [B, HK, N_K, D] bf16, H a multiple of HK; q_lens, k_lens: int32 [B] lengths of a
    padded batch's sequences.  Causal masking is aligned at the last query and key of each sequence.  Rows that
    see no key give 0 and -inf.  return_rest adds what rounding o to bf16 left, a bf16 tensor like o, for attn_bwd.
    """
    got = (_calls or calls()).attn_fwd(q, k, v, scale, causal, q_lens, k_lens, return_rest)
    if got is not None:
        return got
    (q, k, v), q_lens, k_lens, sizes, dev, host = _attn_inputs((q, k, v), q_lens, k_lens)
    (q, qs), (k, ks), (v, vs) = _layout(q), _layout(k), _layout(v)
    B, H, _, NQ, _, D = sizes
    rest = torch.empty_strided((B, H, NQ, D), (*qs, 1), dtype=torch.bfloat16, device=dev) if return_rest else None
    s = make_attn_shape(*sizes, scale, causal, q_lens, k_lens, qs, ks, vs, qs, rest)
    nbytes = _attn_workspace("streamkl_attn_fwd_workspace", dev.index, sizes, bool(causal))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    o = torch.empty_strided((B, H, NQ, D), (*qs, 1), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((B, H, NQ), dtype=torch.float32, device=dev)
    _call("streamkl_attn_fwd", dev.index, q.data_ptr(), k.data_ptr(), v.data_ptr(), s, o.data_ptr(), lse.data_ptr(),
          ws.data_ptr() if nbytes else None, nbytes)
    out = (o, lse, rest) if return_rest else (o, lse)
    return _back(out, True) if host else out


def attn_bwd_plan(B, H, HK, NQ, NK, D, num_sms, causal=False, bwd_mode=BWD_AUTO):
    """(path, parts of a dk/dv tile, parts of a dq tile, workspace bytes) of the attention backward on a device with
    num_sms SMs; path is BWD_FUSED or BWD_SEPARATE."""
    path, kv, q, n = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0), ctypes.c_size_t(0)
    _check(lib().streamkl_attn_bwd_plan(make_attn_shape(B, H, HK, NQ, NK, D, None, causal), int(num_sms), int(bwd_mode),
                                        *map(ctypes.byref, (path, kv, q, n))), "streamkl_attn_bwd_plan")
    return path.value, kv.value, q.value, n.value


def attn_bwd(q, k, v, o, lse, do, dlse=None, scale=None, causal=False, q_lens=None, k_lens=None, bwd_mode=BWD_AUTO,
             o_rest=None):
    """Attention's gradients (dq, dk, dv), bf16 with the layouts of q, k, v.

    o, lse: attn_fwd's for the same inputs; do: dLoss/do like o; dlse: dLoss/dlse fp32 [B, H, N_Q] or None.
    o_rest: attn_fwd's too (return_rest).  Without it, and with N_K above 64, dq and dk carry o's rounding: their error grows
    with the part that v's rows have in common, to several times that of their own rounding (attention gives it).
    bwd_mode BWD_SEPARATE gives the same bits on every run; BWD_FUSED (D = 64) visits each tile pair once and adds dq up
    in no fixed order; BWD_AUTO picks by shape, BWD_SEPARATE where torch.use_deterministic_algorithms asks for the same bits.
    """
    if bwd_mode == BWD_AUTO and torch.are_deterministic_algorithms_enabled():
        bwd_mode = BWD_SEPARATE
    got = (_calls or calls()).attn_bwd(q, k, v, o, lse, do, dlse, scale, causal, q_lens, k_lens, bwd_mode, o_rest)
    if got is not None:
        return got
    (q, k, v, *like_o), q_lens, k_lens, sizes, dev, host = _attn_inputs(
        (q, k, v, o, do) if o_rest is None else (q, k, v, o, do, o_rest), q_lens, k_lens)
    (q, qs), (k, ks), (v, vs) = _layout(q), _layout(k), _layout(v)
    like_o = [_layout(t) for t in like_o]
    B, H, HK, NQ, NK, D = sizes
    os_ = like_o[0][1]
    if any(st != os_ for _, st in like_o):  # the library reads them with one set of strides
        like_o = [(t.clone(memory_format=torch.contiguous_format), None) for t, _ in like_o]
        os_ = (H * NQ * D, NQ * D, D)
    o, do, rest = [t for t, _ in like_o] + ([None] if o_rest is None else [])
    lse = _rows(lse, dev, (B, H, NQ), "lse")
    dlse = _rows(dlse, dev, (B, H, NQ), "dlse")
    s = make_attn_shape(*sizes, scale, causal, q_lens, k_lens, qs, ks, vs, os_, rest)
    nbytes = _attn_workspace("streamkl_attn_bwd_workspace", dev.index, sizes, bool(causal), bwd_mode)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    dq = torch.empty_strided((B, H, NQ, D), (*qs, 1), dtype=torch.bfloat16, device=dev)
    dk = torch.empty_strided((B, HK, NK, D), (*ks, 1), dtype=torch.bfloat16, device=dev)
    dv = torch.empty_strided((B, HK, NK, D), (*vs, 1), dtype=torch.bfloat16, device=dev)
    _call("streamkl_attn_bwd", dev.index, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
          do.data_ptr(), None if dlse is None else dlse.data_ptr(), s, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
          bwd_mode, ws.data_ptr() if nbytes else None, nbytes)
    return _back((dq, dk, dv), True) if host else (dq, dk, dv)


def make_diff_attn_shape(maps, lam=None, lam_strides=(0, 0, 0), d_strides=(0, 0, 0)) -> DiffAttnShape:
    """The C shape of a difference: make_attn_shape's of both maps, and lam (kept alive by the caller)."""
    return DiffAttnShape(maps, None if lam is None else lam.data_ptr(), *lam_strides, *d_strides)


def diff_attn_plan(B, H, HK, NQ, NK, D, num_sms, causal=False):
    """(packed, key splits, workspace bytes) of the forward of H differences on a device with num_sms SMs."""
    a, b, n = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_size_t(0)
    s = make_diff_attn_shape(make_attn_shape(B, 2 * H, HK, NQ, NK, D, None, causal))
    _check(lib().streamkl_diff_attn_fwd_plan(s, int(num_sms), *map(ctypes.byref, (a, b, n))), "streamkl_diff_attn_fwd_plan")
    return bool(a.value), b.value, n.value


def _diff_inputs(tensors, like_d, lam, q_lens, k_lens):
    """Validates a difference's tensors (q, k, v, and maps, maps_rest in the backward), what is like its result, and lam."""
    tensors, q_lens, k_lens, sizes, dev, host = _attn_inputs(tensors, q_lens, k_lens)
    B, H, HK, NQ, _, D = sizes
    if H % 2 or H // 2 % HK:
        raise ValueError(f"{H} query heads are not pairs that divide over {HK} key heads")
    for i, t in enumerate(like_d):
        if t.dtype is not torch.bfloat16:
            raise TypeError("do must be bfloat16")
        if t.shape != (B, H // 2, NQ, D):
            raise ValueError(f"do must be {(B, H // 2, NQ, D)}")
        if (t.device.type == "cpu") != host or (not host and t.device != dev):
            raise ValueError("inputs on different devices")
        if host:
            like_d[i] = t.contiguous().to(dev, non_blocking=True)
    if lam.dtype is not torch.float32:
        raise TypeError("lam must be float32")
    if lam.dim() > 3:
        raise ValueError(f"lam {tuple(lam.shape)} must broadcast to {(B, H // 2, NQ)}")
    lam = lam.expand(B, H // 2, NQ)  # raises where it does not
    if lam.device != dev:
        if not host:
            raise ValueError("inputs on different devices")
        lam = lam.to(dev, non_blocking=True)
    return tensors, like_d, lam, q_lens, k_lens, sizes, dev, host


def diff_attn_fwd(q, k, v, lam, scale=None, causal=False, q_lens=None, k_lens=None, return_maps=False):
    """Differential attention: (d, lse), d = softmax(scale Q1 K^T) V - lam softmax(scale Q2 K^T) V.

    q: [B, 2 H, N_Q, D] bf16, heads 2 i and 2 i + 1 the maps of difference i; k and v: [B, HK, N_K, D], H a multiple of HK;
    lam: fp32, any shape that broadcasts to [B, H, N_Q].  d: bf16 [B, H, N_Q, D], stored by heads or by rows as q is; lse: fp32
    [B, 2 H, N_Q] of both maps.  scale, causal and lengths as in attn_fwd.  return_maps adds what diff_attn_bwd reads: each
    map's own result and what its rounding left, two bf16 tensors like q.
    """
    got = (_calls or calls()).diff_attn_fwd(q, k, v, lam, scale, causal, q_lens, k_lens, return_maps)
    if got is not None:
        return got
    (q, k, v), _, lam, q_lens, k_lens, sizes, dev, host = _diff_inputs((q, k, v), [], lam, q_lens, k_lens)
    (q, qs), (k, ks), (v, vs) = _layout(q), _layout(k), _layout(v)
    B, H, _, NQ, _, D = sizes
    maps = rest = None
    if return_maps:
        maps, rest = (torch.empty_strided((B, H, NQ, D), (*qs, 1), dtype=torch.bfloat16, device=dev) for _ in range(2))
    d = _by_order(B, H // 2, NQ, D, qs, dev)
    s = make_diff_attn_shape(make_attn_shape(*sizes, scale, causal, q_lens, k_lens, qs, ks, vs, qs, rest), lam, lam.stride(),
                             d.stride()[:3])
    nbytes = _workspace_bytes("streamkl_diff_attn_fwd_workspace", dev, s)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    lse = torch.empty((B, H, NQ), dtype=torch.float32, device=dev)
    _call("streamkl_diff_attn_fwd", dev.index, q.data_ptr(), k.data_ptr(), v.data_ptr(), s, d.data_ptr(),
          maps.data_ptr() if return_maps else None, lse.data_ptr(), ws.data_ptr() if nbytes else None, nbytes)
    out = (d, lse, maps, rest) if return_maps else (d, lse)
    return _back(out, True) if host else out


def _by_order(B, H, N, D, strides, dev):
    """A dense bf16 [B, H, N, D] tensor, its rows before its heads where `strides` has them so."""
    if H > 1 and strides[1] < strides[2]:
        return torch.empty((B, N, H, D), dtype=torch.bfloat16, device=dev).transpose(1, 2)
    return torch.empty((B, H, N, D), dtype=torch.bfloat16, device=dev)


def _workspace_bytes(name, dev, *args):
    n = ctypes.c_size_t(0)
    with torch.cuda.device(dev):
        _check(getattr(lib(), name)(*args, ctypes.byref(n)), name)
    return n.value


def diff_attn_bwd(q, k, v, lam, maps, lse, do, dlse=None, scale=None, causal=False, q_lens=None, k_lens=None, bwd_mode=BWD_AUTO,
                  maps_rest=None):
    """Differential attention's gradients (dq, dk, dv, dlam): bf16 with the layouts of q, k, v, and fp32 [B, H, N_Q], a value
    for each row whatever shape lam has.

    maps, lse, maps_rest: diff_attn_fwd's for the same inputs (return_maps), whose 16 bits dlam is as exact as; do: dLoss/dd
    like d; dlse: dLoss/dlse fp32 [B, 2 H, N_Q] or None.  bwd_mode as in attn_bwd.
    """
    if bwd_mode == BWD_AUTO and torch.are_deterministic_algorithms_enabled():
        bwd_mode = BWD_SEPARATE
    got = (_calls or calls()).diff_attn_bwd(q, k, v, lam, maps, lse, do, dlse, scale, causal, q_lens, k_lens, bwd_mode, maps_rest)
    if got is not None:
        return got
    if maps_rest is None:
        raise ValueError("maps_rest is needed: diff_attn_fwd gives it with the maps (return_maps)")
    (q, k, v, maps, rest), (do,), lam, q_lens, k_lens, sizes, dev, host = _diff_inputs((q, k, v, maps, maps_rest), [do], lam,
                                                                                     q_lens, k_lens)
    (q, qs), (k, ks), (v, vs), (do, ds) = _layout(q), _layout(k), _layout(v), _layout(do)
    (maps, os_), (rest, rs) = _layout(maps), _layout(rest)
    B, H, HK, NQ, NK, D = sizes
    if os_ != rs:  # the library reads them with one set of strides
        maps, rest = (t.clone(memory_format=torch.contiguous_format) for t in (maps, rest))
        os_ = (H * NQ * D, NQ * D, D)
    lse, dlse = _rows(lse, dev, (B, H, NQ), "lse"), _rows(dlse, dev, (B, H, NQ), "dlse")
    if lse is None:
        raise ValueError("lse is needed")
    s = make_diff_attn_shape(make_attn_shape(*sizes, scale, causal, q_lens, k_lens, qs, ks, vs, os_, rest), lam, lam.stride(), ds)
    nbytes = _workspace_bytes("streamkl_diff_attn_bwd_workspace", dev, s, int(bwd_mode))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    dq = torch.empty_strided((B, H, NQ, D), (*qs, 1), dtype=torch.bfloat16, device=dev)
    dk = torch.empty_strided((B, HK, NK, D), (*ks, 1), dtype=torch.bfloat16, device=dev)
    dv = torch.empty_strided((B, HK, NK, D), (*vs, 1), dtype=torch.bfloat16, device=dev)
    dlam = torch.empty((B, H // 2, NQ), dtype=torch.float32, device=dev)
    _call("streamkl_diff_attn_bwd", dev.index, q.data_ptr(), k.data_ptr(), v.data_ptr(), maps.data_ptr(), lse.data_ptr(),
          do.data_ptr(), None if dlse is None else dlse.data_ptr(), s, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
          dlam.data_ptr(), bwd_mode, ws.data_ptr() if nbytes else None, nbytes)
    return _back((dq, dk, dv, dlam), True) if host else (dq, dk, dv, dlam)


def _logits_rows(logits, tokens):
    """Validates logits [..., V] and tokens [...] or [..., T]; returns (device logits as strided [R, V] rows,
    contiguous int64 device tokens or None, T, the leading shape, device, was_host)."""
    shape, dev = logits.shape, logits.device
    if logits.dtype not in DTYPES:
        raise TypeError("logits must be bfloat16, float16 or float32")
    if len(shape) < 1 or shape[-1] == 0:
        raise ValueError("logits must be [..., V] with V > 0")
    V, lead, T = shape[-1], shape[:-1], 0
    if tokens is not None:
        if tokens.dtype is not torch.int64 and tokens.dtype is not torch.int32:
            raise TypeError("tokens must be int64 or int32")
        given = tokens.shape
        if given == lead:
            T = 1
        elif len(given) == len(shape) and given[:-1] == lead:
            T = given[-1]
        else:
            raise ValueError(f"tokens {tuple(given)} do not fit logits {tuple(shape)}")
        if tokens.device != dev:
            raise ValueError("inputs on different devices")
    host = dev.type == "cpu"
    if host:
        dev = torch.device("cuda", torch.cuda.current_device())
        logits = logits.to(dev, non_blocking=True)
    x = logits if len(shape) == 2 else logits.reshape(-1, V)
    if not x.is_contiguous() and ((V > 1 and x.stride(1) != 1) or (x.shape[0] > 1 and x.stride(0) < V)):
        x = x.contiguous()
    if not T:
        return x, None, 0, lead, dev, host
    if host or tokens.dtype is not torch.int64:
        tokens = tokens.to(device=dev, dtype=torch.int64, non_blocking=True)
    return x, tokens if tokens.is_contiguous() else tokens.contiguous(), T, lead, dev, host


def _row_stride(x):
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def logprobs_fwd(logits, tokens=None, scale=1.0, top_k=0):
    """Log probabilities of given tokens: (logp, entropy, lse, top_logp, top_index).

    logits: [..., V] bf16, fp16 or fp32, multiplied by scale > 0; tokens: [...] or [..., T], int64 or int32, a
    negative one is no token (its logp is 0).  logp has the shape of tokens; entropy and lse are [...];
    top_logp fp32 and top_index int64 are [..., top_k], the largest logits (equal ones: the lowest index first).
    """
    got = (_calls or calls()).logprobs_fwd(logits, tokens, scale, top_k)
    if got is not None:
        return got
    x, tok, T, lead, dev, host = _logits_rows(logits, tokens)
    R, V = x.shape
    if not 0 <= top_k <= min(LOGPROBS_MAX_TOP_K, V):
        raise ValueError(f"top_k must be between 0 and min({LOGPROBS_MAX_TOP_K}, V)")
    logp = torch.empty(tokens.shape if tokens is not None else (*lead, 0), dtype=torch.float32, device=dev)
    entropy = torch.empty(lead, dtype=torch.float32, device=dev)
    lse = torch.empty(lead, dtype=torch.float32, device=dev)
    top = torch.empty((*lead, top_k), dtype=torch.float32, device=dev)
    idx = torch.empty((*lead, top_k), dtype=torch.int64, device=dev)
    _call("streamkl_logprobs_fwd", dev.index, x.data_ptr(), DTYPES[x.dtype], R, V, _row_stride(x),
          tok.data_ptr() if T else None, T, scale, top_k, logp.data_ptr(), entropy.data_ptr(), lse.data_ptr(),
          top.data_ptr(), idx.data_ptr())
    return _back((logp, entropy, lse, top, idx), True) if host else (logp, entropy, lse, top, idx)


def logprobs_bwd(logits, tokens, lse, entropy, g_logp, g_entropy=None, scale=1.0):
    """Gradient of the logits, contiguous and of their type, for upstream gradients g_logp (tokens' shape) and
    g_entropy ([...] or None); lse and entropy are logprobs_fwd's (entropy may be None without g_entropy)."""
    got = (_calls or calls()).logprobs_bwd(logits, tokens, lse, entropy, g_logp, g_entropy, scale)
    if got is not None:
        return got
    x, tok, T, lead, dev, host = _logits_rows(logits, tokens)
    R, V = x.shape
    lse = _rows(lse, dev, lead, "lse")
    ent = None
    if g_entropy is not None:
        if entropy is None:
            raise ValueError("g_entropy needs the forward's entropy")
        g_entropy, ent = _rows(g_entropy, dev, lead, "g_entropy"), _rows(entropy, dev, lead, "entropy")
    g_logp = _rows(g_logp, dev, tokens.shape, "g_logp") if T else None
    if T and g_logp is None:
        raise ValueError("tokens need g_logp")
    out = torch.empty(logits.shape, dtype=x.dtype, device=dev)
    _call("streamkl_logprobs_bwd", dev.index, x.data_ptr(), DTYPES[x.dtype], R, V, _row_stride(x),
          tok.data_ptr() if T else None, T, scale, lse.data_ptr(), None if ent is None else ent.data_ptr(),
          g_logp.data_ptr() if T else None, None if ent is None else g_entropy.data_ptr(), out.data_ptr(), V)
    return _back((out,), True)[0] if host else out


def _rotary(tensors, plan, positions, offset, interleaved, inverse, out):
    """Turns q and k (either may be None) by their positions; see rotary_fwd."""
    q, k = tensors
    one = q if q is not None else k
    if one is None:
        raise ValueError("q or k is needed")
    B, _, N, D = _rotary_sizes(one)
    dtype, dev = one.dtype, one.device
    if dtype not in DTYPES:
        raise TypeError("q and k must be bfloat16, float16 or float32")
    if D % 2 or plan.dim > D:
        raise ValueError(f"{plan.dim} channels do not turn in {D}: D must be even and at least the plan's dim")
    host = dev.type == "cpu"
    if host:
        if out is not None:
            raise ValueError("out is for device tensors")
        dev = torch.device("cuda", torch.cuda.current_device())
    if plan.turns.device != dev:
        raise ValueError(f"the plan is on {plan.turns.device}, the tensors on {dev}")
    given, stride, size = None, 0, 0
    if positions is not None:
        if offset:
            raise ValueError("positions or an offset, not both")
        if positions.dtype is not torch.int64 and positions.dtype is not torch.int32:
            raise TypeError("positions must be int64 or int32")
        if positions.shape != (N,) and positions.shape != (B, N):
            raise ValueError(f"positions {tuple(positions.shape)} must be [{N}] or [{B}, {N}]")
        given = positions.to(dev, non_blocking=True) if positions.device != dev else positions
        if N > 1 and given.stride(-1) != 1:
            given = given.contiguous()
        size, stride = given.element_size(), given.stride(0) if given.dim() == 2 and B > 1 else 0
    outs = (None, None) if out is None else tuple(out)
    if len(outs) != 2:
        raise ValueError("out must be (q_out, k_out)")
    ins, outs, strides, ptrs = [], list(outs), [], []
    for i, (t, o) in enumerate(zip(tensors, list(outs))):
        if t is None:
            if o is not None:
                raise ValueError("an output without its input")
            ins.append(None)
            continue
        if t.dtype != dtype or t.device != one.device:
            raise ValueError("q and k must have the same type and device")
        b, h, n, d = _rotary_sizes(t)
        if (b, n, d) != (B, N, D):
            raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)}")
        if host:
            t = t.to(dev, non_blocking=True)
        if t.stride(3) != 1:
            t = t.contiguous()
        if o is None:
            outs[i] = torch.empty_like(t) if t.stride(3) == 1 and all(s > 0 for s in t.stride()) else t.new_empty(t.shape)
        elif o.shape != t.shape or o.dtype != dtype or o.device != dev or o.stride(3) != 1:
            raise ValueError("an output must have its input's shape, type and device, and contiguous channels")
        elif o.requires_grad and torch.is_grad_enabled():
            raise ValueError("out has no gradient: an output that requires one is not written to")
        elif not o.is_inference():
            torch.autograd.graph.increment_version(o)  # what was saved of it for a backward is no longer there
        ins.append(t)
    for t in (*ins, *outs):
        strides += [0, 0, 0] if t is None else t.stride()[:3]
        ptrs.append(None if t is None else t.data_ptr())
    s = RotaryShape(B, 0 if q is None else q.shape[1], 0 if k is None else k.shape[1], N, D, plan.dim, DTYPES[dtype],
                    bool(interleaved), plan.amplitude, int(offset), None if given is None else given.data_ptr(), size, stride,
                    *strides)
    _call("streamkl_rotary", dev.index, ptrs[0], ptrs[1], s, plan.turns.data_ptr(), ptrs[2], ptrs[3], bool(inverse))
    if not host:
        return tuple(outs)
    got = iter(_back(tuple(t for t in outs if t is not None), True))
    return tuple(None if t is None else next(got) for t in outs)


def _rotary_sizes(t):
    if t.dim() != 4:
        raise ValueError("q and k must be [B, H, N, D]")
    return t.shape


def rotary_fwd(q, k, plan, positions=None, offset=0, interleaved=False, out=None):
    """Rotary positions: (q, k) with the first plan.dim of D channels turned by each row's position.

    q: [B, HQ, N, D], k: [B, HK, N, D], bf16, fp16 or fp32, either may be None; plan: rotary_plan's, on their device.
    positions: int64 or int32 [N] or [B, N]; without them row n is at offset + n.  Pairs are the channels i and dim / 2 + i,
    with interleaved 2 i and 2 i + 1.  out: (q_out, k_out) to write to, for example q and k themselves or a cache's rows
    (it may overlap nothing else, and require no gradient); an entry may be None.
    """
    if out is None:
        got = (_calls or calls()).rotary(q, k, plan.turns, plan.dim, plan.amplitude, positions, offset, interleaved, False)
        if got is not None:
            return got
    return _rotary((q, k), plan, positions, offset, interleaved, False, out)


def rotary_bwd(dq, dk, plan, positions=None, offset=0, interleaved=False, out=None):
    """The gradients of rotary_fwd's q and k from those of its results: turned back by the same positions."""
    if out is None:
        got = (_calls or calls()).rotary(dq, dk, plan.turns, plan.dim, plan.amplitude, positions, offset, interleaved, True)
        if got is not None:
            return got
    return _rotary((dq, dk), plan, positions, offset, interleaved, True, out)


def make_xent_shape(rows, vocab, channels, dtype=0, scale=1.0, hidden_stride=None, weight_stride=None) -> XentShape:
    """The C shape of a vocabulary's cross entropy; dtype is a streamkl_dtype, strides default to contiguous rows."""
    return XentShape(rows, vocab, channels, dtype, scale, channels if hidden_stride is None else hidden_stride,
                     channels if weight_stride is None else weight_stride)


def _matrix(t):
    """A 2-D matrix that the library reads in place (a contiguous copy where it cannot) and its row stride."""
    if t.stride(1) != 1 or t.data_ptr() & 15 or (t.shape[0] > 1 and (t.stride(0) % 8 or t.stride(0) < t.shape[1])):
        t = t.clone(memory_format=torch.contiguous_format)
    return t, t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _xent_inputs(hidden, weight, tokens, scale):
    """Validates hidden [..., C], weight [V, C] and tokens [...]; returns (hidden as [R, C], weight, contiguous int64
    tokens, the C shape, the leading shape, device, was_host)."""
    if hidden.dtype is not torch.bfloat16 and hidden.dtype is not torch.float16:
        raise TypeError("hidden must be bfloat16 or float16")
    if weight.dtype is not hidden.dtype:
        raise TypeError("hidden and weight must have the same type")
    if hidden.dim() < 1 or weight.dim() != 2 or hidden.shape[-1] != weight.shape[1]:
        raise ValueError(f"shape mismatch: hidden {tuple(hidden.shape)} weight {tuple(weight.shape)}")
    V, C = weight.shape
    if V == 0 or C == 0 or C % 8:
        raise ValueError("weight must be [V, C] with V > 0 and C a positive multiple of 8")
    lead, dev = hidden.shape[:-1], hidden.device
    if tokens.dtype is not torch.int64 and tokens.dtype is not torch.int32:
        raise TypeError("tokens must be int64 or int32")
    if tokens.shape != lead:
        raise ValueError(f"tokens {tuple(tokens.shape)} do not fit hidden {tuple(hidden.shape)}")
    if weight.device != dev or tokens.device != dev:
        raise ValueError("inputs on different devices")
    host = dev.type == "cpu"
    if host:
        dev = torch.device("cuda", torch.cuda.current_device())
        hidden, weight = hidden.to(dev, non_blocking=True), weight.to(dev, non_blocking=True)
    if host or tokens.dtype is not torch.int64:
        tokens = tokens.to(device=dev, dtype=torch.int64, non_blocking=True)
    (x, xs), (w, ws) = _matrix(hidden if hidden.dim() == 2 else hidden.reshape(-1, C)), _matrix(weight)
    s = make_xent_shape(x.shape[0], V, C, DTYPES[x.dtype], scale, xs, ws)
    return x, w, tokens if tokens.is_contiguous() else tokens.contiguous(), s, lead, dev, host


def vocab_xent_fwd_plan(rows, vocab, channels, num_sms):
    """(columns of a tile, workspace bytes) of the forward on a device with num_sms SMs."""
    w, n = ctypes.c_int(0), ctypes.c_size_t(0)
    _check(lib().streamkl_vocab_xent_fwd_plan(make_xent_shape(rows, vocab, channels), int(num_sms), ctypes.byref(w), ctypes.byref(n)),
           "streamkl_vocab_xent_fwd_plan")
    return w.value, n.value


def vocab_xent_plan(rows, vocab, channels, num_sms, want_dhidden=True, want_dweight=True):
    """(pieces of the vocabulary, splits of dhidden's sums, workspace bytes) of the backward on a device with num_sms SMs."""
    a, b, n = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_size_t(0)
    _check(lib().streamkl_vocab_xent_bwd_plan(make_xent_shape(rows, vocab, channels), int(num_sms), bool(want_dhidden),
                                              bool(want_dweight), *map(ctypes.byref, (a, b, n))), "streamkl_vocab_xent_bwd_plan")
    return a.value, b.value, n.value


def vocab_xent_fwd(hidden, weight, tokens, scale=1.0):
    """Cross entropy of the rows softmax(scale hidden weight^T) at given tokens, without the logits in memory:
    (loss, lse), fp32 like tokens.

    hidden: [..., C], weight: [V, C], both bf16 or both fp16, C a multiple of 8; tokens: [...], int64 or int32, a negative
    one is no token (its loss is 0), one past the vocabulary gives NaN.
    """
    got = (_calls or calls()).vocab_xent_fwd(hidden, weight, tokens, scale)
    if got is not None:
        return got
    x, w, tok, s, lead, dev, host = _xent_inputs(hidden, weight, tokens, scale)
    nbytes = _workspace_bytes("streamkl_vocab_xent_fwd_workspace", dev, s)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    loss, lse = (torch.empty(lead, dtype=torch.float32, device=dev) for _ in range(2))
    _call("streamkl_vocab_xent_fwd", dev.index, x.data_ptr(), w.data_ptr(), tok.data_ptr(), s, loss.data_ptr(),
          lse.data_ptr(), ws.data_ptr(), nbytes)
    return _back((loss, lse), True) if host else (loss, lse)


def vocab_xent_bwd(hidden, weight, tokens, lse, g_loss, g_lse=None, scale=1.0, want_dhidden=True, want_dweight=True):
    """Gradients (dhidden, dweight) of vocab_xent_fwd's outputs, contiguous and of the inputs' type, for upstream
    gradients g_loss and g_lse (fp32 like tokens; g_lse may be None); lse is the forward's.  One that is not wanted is None.

    The same bits on every run.  Rows without a gradient have none whatever they hold, NaN included; weight has to be finite.
    """
    if want_dhidden and want_dweight:
        got = (_calls or calls()).vocab_xent_bwd(hidden, weight, tokens, lse, g_loss, g_lse, scale)
        if got is not None:
            return got
    x, w, tok, s, lead, dev, host = _xent_inputs(hidden, weight, tokens, scale)
    lse, g_loss, g_lse = _rows(lse, dev, lead, "lse"), _rows(g_loss, dev, lead, "g_loss"), _rows(g_lse, dev, lead, "g_lse")
    if lse is None or g_loss is None:
        raise ValueError("lse and g_loss are needed")
    if not want_dhidden and not want_dweight:
        return None, None
    nbytes = _workspace_bytes("streamkl_vocab_xent_bwd_workspace", dev, s, bool(want_dhidden), bool(want_dweight))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    dh = torch.empty(hidden.shape, dtype=x.dtype, device=dev) if want_dhidden else None
    dw = torch.empty(weight.shape, dtype=x.dtype, device=dev) if want_dweight else None
    _call("streamkl_vocab_xent_bwd", dev.index, x.data_ptr(), w.data_ptr(), tok.data_ptr(), lse.data_ptr(), g_loss.data_ptr(),
          None if g_lse is None else g_lse.data_ptr(), s, None if dh is None else dh.data_ptr(),
          None if dw is None else dw.data_ptr(), ws.data_ptr() if nbytes else None, nbytes)
    if not host:
        return dh, dw
    got = iter(_back(tuple(t for t in (dh, dw) if t is not None), True))
    return tuple(None if t is None else next(got) for t in (dh, dw))


def check_device_status(device=None) -> int:
    """Synchronises the current stream and returns (and clears) the device status."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return lib().streamkl_check_device_status(_stream(dev))


def debug_wait_timeout(timeout_us: int) -> int:
    dev = torch.device("cuda", torch.cuda.current_device())
    return lib().streamkl_debug_wait_timeout(int(timeout_us), _stream(dev))
