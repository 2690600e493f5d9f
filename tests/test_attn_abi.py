"""Attention: what the entry points refuse and how the forward is planned, on the host before anything is launched."""
import ctypes

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib as K
from attention_kl_divergence_streamkl_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return K.lib()


def ptr(off=0):
    return ctypes.c_void_p(0x10000000 + off)


OK = dict(B=2, H=8, HK=2, NQ=100, NK=100, D=64)
BAD = [
    (dict(B=0), K.ERR_INVALID), (dict(H=0), K.ERR_INVALID), (dict(HK=0), K.ERR_INVALID), (dict(HK=3), K.ERR_INVALID),
    (dict(NQ=-1), K.ERR_INVALID), (dict(NK=-1), K.ERR_INVALID), (dict(D=0), K.ERR_INVALID),
    (dict(D=96), K.ERR_UNSUPPORTED), (dict(D=256), K.ERR_UNSUPPORTED), (dict(NK=2**31 - 1), K.ERR_UNSUPPORTED),
    (dict(scale=float("nan")), K.ERR_INVALID), (dict(scale=float("inf")), K.ERR_INVALID),
    (dict(B=1 << 15, H=1 << 15, HK=1), K.ERR_UNSUPPORTED),
    (dict(q_strides=(8, 8, 32)), K.ERR_INVALID), (dict(k_strides=(6400, 6401, 64)), K.ERR_INVALID),
    (dict(v_strides=(-6400, 6400, 64)), K.ERR_INVALID), (dict(o_strides=(6400, 6400, 63)), K.ERR_INVALID),
]


@pytest.mark.parametrize("change,code", BAD)
def test_fwd_refuses_shapes(lib, change, code):
    s = K.make_attn_shape(**{**OK, **change})
    assert lib.streamkl_attn_fwd(ptr(), ptr(), ptr(), s, ptr(), ptr(), None, 0, None) == code
    assert lib.streamkl_attn_fwd_workspace(s, ctypes.byref(ctypes.c_size_t())) == code


def test_fwd_refuses_pointers(lib):
    s = K.make_attn_shape(**OK)
    a = [ptr(64 * i) for i in range(5)]
    for i in range(5):
        for bad in (None, ptr(64 * i + 2)):
            b = list(a)
            b[i] = bad
            assert lib.streamkl_attn_fwd(*b[:3], s, *b[3:], None, 0, None) == K.ERR_INVALID
    s.q_lens = 0x1002
    assert lib.streamkl_attn_fwd(*a[:3], s, *a[3:], None, 0, None) == K.ERR_INVALID


def test_no_queries_is_no_work(lib):
    s = K.make_attn_shape(**{**OK, "NQ": 0})
    assert lib.streamkl_attn_fwd(None, None, None, s, None, None, None, 0, None) == K.OK


@pytest.mark.parametrize("shape,want", [
    (dict(B=1, H=32, HK=8, NQ=4096, NK=4096, D=128), (False, 1)),   # enough query tiles
    (dict(B=1, H=8, HK=2, NQ=1, NK=129, D=64), (True, 1)),          # too short to split
    (dict(B=1, H=8, HK=1, NQ=17, NK=300, D=64), (False, 1)),        # 136 packed rows do not fit one tile
])
def test_plan(lib, shape, want):
    assert skl.attn_fwd_plan(**shape, num_sms=152) == want


@pytest.mark.parametrize("NQ,H,HK,B,NK", [(1, 32, 8, 8, 131072), (1, 8, 8, 1, 131072), (4, 32, 8, 1, 4096), (300, 4, 4, 1, 65536)])
def test_few_tiles_split_the_keys(lib, NQ, H, HK, B, NK):
    """The launch fills the SMs without leaving a nearly empty last wave, and every split has keys."""
    packed, splits = skl.attn_fwd_plan(B, H, HK, NQ, NK, 128, 152)
    assert packed == (H // HK * NQ <= 128)
    blocks = B * (HK if packed else H * -(-NQ // 256)) * splits
    assert splits > 1 and -(-NK // 128) // splits >= 1
    assert blocks / (152 * -(-blocks // 152)) > 0.6 or blocks < 152


@pytest.mark.parametrize("q,k,v,lens,error", [
    ((1, 4, 3, 64), (1, 3, 3, 64), (1, 3, 3, 64), None, ValueError),   # heads do not divide
    ((1, 4, 3, 64), (1, 2, 3, 64), (1, 2, 4, 64), None, ValueError),   # k and v differ
    ((1, 4, 3, 64), (2, 2, 3, 64), (2, 2, 3, 64), None, ValueError),   # batches differ
    ((1, 4, 3, 64), (1, 2, 3, 128), (1, 2, 3, 128), None, ValueError),
    ((4, 3, 64), (1, 2, 3, 64), (1, 2, 3, 64), None, ValueError),
])
def test_binding_refuses(q, k, v, lens, error):
    q, k, v = (torch.zeros(x, dtype=torch.bfloat16) for x in (q, k, v))
    with pytest.raises(error):
        skl.attn_fwd(q, k, v)


def test_binding_refuses_types():
    q = torch.zeros(1, 2, 3, 64)
    with pytest.raises(TypeError):
        skl.attn_fwd(q, q, q)


def bwd_args(s, drop=None, off=None, ws=1 << 30, mode=K.BWD_SEPARATE):
    names = ["q", "k", "v", "o", "lse", "go", "dlse", "s", "dq", "dk", "dv", "mode", "ws"]
    a = {n: ptr(64 * i) for i, n in enumerate(names)}
    a["s"], a["mode"] = s, mode
    if drop:
        a[drop] = None
    if off:
        a[off] = ptr(2)
    return [*a.values(), ws, None]


@pytest.mark.parametrize("change,code", BAD)
def test_bwd_refuses_shapes(lib, change, code):
    s = K.make_attn_shape(**{**OK, **change})
    assert lib.streamkl_attn_bwd(*bwd_args(s)) == code
    out = [ctypes.byref(ctypes.c_int()) for _ in range(3)] + [ctypes.byref(ctypes.c_size_t())]
    assert lib.streamkl_attn_bwd_plan(s, 152, K.BWD_AUTO, *out) == code
    assert lib.streamkl_attn_bwd_workspace(s, K.BWD_AUTO, out[-1]) == code


def test_bwd_refuses_pointers_and_small_workspaces(lib):
    s = K.make_attn_shape(**OK)
    for name in ("q", "k", "v", "o", "lse", "go", "dq", "dk", "dv"):
        assert lib.streamkl_attn_bwd(*bwd_args(s, drop=name)) == K.ERR_INVALID, name
        assert lib.streamkl_attn_bwd(*bwd_args(s, off=name)) == K.ERR_INVALID, name
    assert lib.streamkl_attn_bwd(*bwd_args(s, off="dlse")) == K.ERR_INVALID
    for mode in (-1, K.BWD_DQ_ONLY, K.BWD_DK_ONLY, 5):
        assert lib.streamkl_attn_bwd(*bwd_args(s, mode=mode)) == K.ERR_INVALID
        with pytest.raises(skl.StreamKLError):
            skl.attn_bwd_plan(**OK, num_sms=152, bwd_mode=mode)
    wide = K.make_attn_shape(**{**OK, "D": 128})
    assert lib.streamkl_attn_bwd(*bwd_args(wide, mode=K.BWD_FUSED)) == K.ERR_UNSUPPORTED
    for ws in (0, 2 * 8 * 100 * 32 - 1):
        assert lib.streamkl_attn_bwd(*bwd_args(s, ws=ws)) == K.ERR_WORKSPACE
    assert lib.streamkl_attn_bwd(*bwd_args(s, drop="ws")) == K.ERR_WORKSPACE
    assert lib.streamkl_attn_bwd(*bwd_args(s, off="ws")) == K.ERR_WORKSPACE


def test_bwd_binding_refuses():
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    lse = torch.zeros(1, 2, 3)
    with pytest.raises(TypeError):
        skl.attn_bwd(q, q, q, q, lse, q.float())
    with pytest.raises(ValueError):
        skl.attn_bwd(q, q, q, q[:, :, :2], lse, q)


def test_bwd_plan(lib):
    """The path, the parts and the workspace: 32 bytes a row (queries rounded up to 128), 4 D more when fused, and 3 D
    fp32 accumulators of 128 rows for a part of both kinds."""
    rows = 2 * 8 * 128
    assert skl.attn_bwd_plan(**OK, num_sms=152) == (K.BWD_SEPARATE, 1, 1, rows * 32)
    assert skl.attn_bwd_plan(**OK, num_sms=152, bwd_mode=K.BWD_FUSED)[3] == rows * (32 + 4 * 64)
    # D = 64, key tiles fill the SMs: fused; its last wave of 512 - 3 * 152 = 56 tiles in two parts each
    path, kv, q, ws = skl.attn_bwd_plan(1, 8, 8, 8192, 8192, 64, 152)
    assert (path, kv, q) == (K.BWD_FUSED, 2, 1)
    assert ws == 8 * 8192 * (32 + 256) + 56 * 2 * 128 * 128 * 4 + 56 * 4
    # causal: its own short blocks fill the end
    assert skl.attn_bwd_plan(1, 8, 8, 8192, 8192, 64, 152, True)[:2] == (K.BWD_FUSED, 1)
    assert skl.attn_bwd_plan(1, 8, 8, 8192, 8192, 64, 152, bwd_mode=K.BWD_SEPARATE)[0] == K.BWD_SEPARATE
    # many blocks: none is dealt out
    assert skl.attn_bwd_plan(2, 32, 8, 4096, 4096, 128, 152, True)[:3] == (K.BWD_SEPARATE, 1, 1)
    # 64 key tiles, each read by four heads of 16 tiles, leave most SMs idle
    assert skl.attn_bwd_plan(1, 16, 4, 2048, 2048, 128, 152, True)[1:3] == (2, 1)
    # so do 4 query tiles over 512 key tiles
    assert skl.attn_bwd_plan(1, 4, 4, 128, 65536, 128, 152)[2] > 1
