"""Differential attention: what the entry points refuse and how they plan, on the host before anything is launched."""
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


MAPS = dict(B=2, H=8, HK=2, NQ=16, NK=32, D=64, scale=0.0, causal=0, q_lens=None, k_lens=None, qb=0, qh=0, qn=0, kb=0, kh=0, kn=0,
            vb=0, vh=0, vn=0, ob=0, oh=0, on=0, o_rest=None)
REST = dict(lam=ptr(1024), lb=0, lh=0, ln=0, db=0, dh=0, dn=0)


def shape(**change):
    maps = K.AttnShape(*{k: change.get(k, v) for k, v in MAPS.items()}.values())
    return K.DiffAttnShape(maps, *{k: change.get(k, v) for k, v in REST.items()}.values())


def fwd(lib, q=ptr(), k=ptr(16), v=ptr(32), d=ptr(64), maps=None, lse=ptr(128), ws=ptr(4096), nbytes=1 << 24, **change):
    return lib.streamkl_diff_attn_fwd(q, k, v, shape(**change), d, maps, lse, ws, nbytes, None)


def bwd(lib, q=ptr(), k=ptr(16), v=ptr(32), maps=ptr(48), lse=ptr(64), go=ptr(80), dlse=None, dq=ptr(96), dk=ptr(112), dv=ptr(128),
        dlam=ptr(144), mode=0, ws=ptr(4096), nbytes=1 << 24, **change):
    return lib.streamkl_diff_attn_bwd(q, k, v, maps, lse, go, dlse, shape(**{"o_rest": ptr(160), **change}), dq, dk, dv, dlam, mode,
                                      ws, nbytes, None)


SHAPES = [(dict(B=0), K.ERR_INVALID), (dict(H=7, HK=7), K.ERR_INVALID), (dict(H=8, HK=8), K.ERR_INVALID), (dict(H=12, HK=4), K.ERR_INVALID),
          (dict(HK=0), K.ERR_INVALID), (dict(NQ=-1), K.ERR_INVALID), (dict(D=96), K.ERR_UNSUPPORTED), (dict(scale=float("nan")), K.ERR_INVALID),
          (dict(lam=ptr(2)), K.ERR_INVALID), (dict(lb=-1), K.ERR_INVALID), (dict(dn=32, dh=512, db=4096), K.ERR_INVALID),
          (dict(dn=68, dh=2048, db=8192), K.ERR_INVALID), (dict(qn=60, qh=1024, qb=8192), K.ERR_INVALID), (dict(NQ=2**31 - 1), K.ERR_UNSUPPORTED)]


@pytest.mark.parametrize("change,code", SHAPES)
def test_shapes_that_are_refused(lib, change, code):
    i, n = ctypes.c_int(0), ctypes.c_size_t(0)
    assert fwd(lib, **change) == code
    assert bwd(lib, **change) == code
    assert lib.streamkl_diff_attn_fwd_plan(shape(**change), 152, ctypes.byref(i), ctypes.byref(i), ctypes.byref(n)) == code
    assert lib.streamkl_diff_attn_bwd_workspace(shape(**change), 0, ctypes.byref(n)) == code


@pytest.mark.parametrize("change", [dict(q=None), dict(k=ptr(8)), dict(v=None), dict(d=None), dict(d=ptr(8)), dict(lse=None),
                                    dict(maps=ptr(48)), dict(o_rest=ptr(48)), dict(lam=None)])
def test_forward_refuses_pointers(lib, change):
    """Each map's own result and its rest are wanted together or not at all."""
    assert fwd(lib, **change) == K.ERR_INVALID


@pytest.mark.parametrize("change,code", [
    (dict(q=None), K.ERR_INVALID), (dict(maps=None), K.ERR_INVALID), (dict(o_rest=None), K.ERR_INVALID), (dict(go=None), K.ERR_INVALID),
    (dict(go=ptr(8)), K.ERR_INVALID), (dict(lse=None), K.ERR_INVALID), (dict(dlse=ptr(2)), K.ERR_INVALID), (dict(dq=None), K.ERR_INVALID),
    (dict(dk=None), K.ERR_INVALID), (dict(dv=ptr(8)), K.ERR_INVALID), (dict(dlam=None), K.ERR_INVALID), (dict(lam=None), K.ERR_INVALID),
    (dict(mode=3), K.ERR_INVALID), (dict(mode=1, D=128), K.ERR_UNSUPPORTED), (dict(ws=None), K.ERR_WORKSPACE),
    (dict(ws=ptr(8)), K.ERR_WORKSPACE), (dict(nbytes=100), K.ERR_WORKSPACE),
])
def test_backward_refuses(lib, change, code):
    assert bwd(lib, **change) == code


def test_no_queries_is_no_work(lib):
    assert fwd(lib, NQ=0, q=None, d=None, lse=None) == K.OK


@pytest.mark.parametrize("B_,H,HK,NQ,NK,D", [(1, 8, 4, 1, 65536, 128), (8, 16, 8, 1, 131072, 128), (2, 16, 8, 4096, 4096, 128),
                                             (1, 1, 1, 1, 1, 64), (4, 8, 4, 64, 100, 64), (1, 4, 2, 33, 5000, 128)])
def test_plan(B_, H, HK, NQ, NK, D):
    """Packed where both maps of all heads of a key head fit one tile; otherwise a block has 128 rows of both maps."""
    B.build()
    packed, splits, nbytes = skl.diff_attn_plan(B_, H, HK, NQ, NK, D, 152)
    assert packed == (2 * H // HK * NQ <= 128)
    assert 1 <= splits <= -(-NK // 128)
    assert nbytes == (splits * B_ * 2 * H * NQ * (D + 2) * 4 if splits > 1 else 0)
    if B_ * (HK if packed else H * -(-NQ // 128)) >= 152:
        assert splits <= 4 * 152


def q_like(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("q,k,lam,error", [
    (q_like(1, 4, 8, 64, dtype=torch.float16), q_like(1, 2, 8, 64), torch.zeros(1), TypeError),
    (q_like(1, 3, 8, 64), q_like(1, 3, 8, 64), torch.zeros(1), ValueError),
    (q_like(1, 4, 8, 64), q_like(1, 4, 8, 64), torch.zeros(1), ValueError),
    (q_like(4, 8, 64), q_like(1, 2, 8, 64), torch.zeros(1), ValueError),
])
def test_binding_refuses(q, k, lam, error):
    B.build()
    if q.dim() == 4 and q.dtype is torch.bfloat16 and q.shape[1] != 3 and not torch.cuda.is_available():
        pytest.skip("host tensors go to the device first")
    if q.dim() == 4 and q.shape[1] == 3 and not torch.cuda.is_available():
        pytest.skip("host tensors go to the device first")
    with pytest.raises(error):
        skl.diff_attn_fwd(q, k, k, lam)
