"""Token log probabilities: what the entry points refuse, checked on the host before anything is launched."""
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


FWD = dict(logits=ptr(), dtype=0, rows=4, vocab=100, stride=100, tokens=ptr(64), T=2, scale=1.0, top_k=5, logp=ptr(128),
           entropy=ptr(192), lse=ptr(256), top=ptr(320), index=ptr(384))
BWD = dict(logits=ptr(), dtype=0, rows=4, vocab=100, stride=100, tokens=ptr(64), T=2, scale=1.0, lse=ptr(128),
           entropy=ptr(192), g=ptr(256), gh=ptr(320), out=ptr(384), out_stride=100)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), K.ERR_INVALID), (dict(vocab=0), K.ERR_INVALID), (dict(stride=99), K.ERR_INVALID),
    (dict(T=-1), K.ERR_INVALID), (dict(top_k=-1), K.ERR_INVALID), (dict(top_k=101), K.ERR_INVALID),
    (dict(top_k=33), K.ERR_UNSUPPORTED), (dict(dtype=3), K.ERR_INVALID), (dict(dtype=-1), K.ERR_INVALID),
    (dict(scale=0.0), K.ERR_INVALID), (dict(scale=-1.0), K.ERR_INVALID), (dict(scale=float("nan")), K.ERR_INVALID),
    (dict(scale=float("inf")), K.ERR_INVALID), (dict(vocab=2**31, stride=2**31), K.ERR_UNSUPPORTED),
    (dict(rows=2**31), K.ERR_UNSUPPORTED), (dict(logits=None), K.ERR_INVALID), (dict(logits=ptr(1)), K.ERR_INVALID),
    (dict(dtype=2, logits=ptr(2)), K.ERR_INVALID), (dict(tokens=ptr(4)), K.ERR_INVALID), (dict(logp=None), K.ERR_INVALID),
    (dict(lse=None), K.ERR_INVALID), (dict(entropy=ptr(2)), K.ERR_INVALID), (dict(index=ptr(4)), K.ERR_INVALID),
    (dict(top=None), K.ERR_INVALID),
])
def test_fwd_refuses(lib, change, code):
    assert lib.streamkl_logprobs_fwd(*{**FWD, **change}.values(), None) == code


@pytest.mark.parametrize("change,code", [
    (dict(out_stride=99), K.ERR_INVALID), (dict(out=None), K.ERR_INVALID), (dict(out=ptr(1)), K.ERR_INVALID),
    (dict(out=ptr()), K.ERR_INVALID),  # onto the logits, with tokens
    (dict(out=ptr(), out_stride=104, T=0), K.ERR_INVALID),  # onto the logits, rows on other rows
    (dict(lse=None), K.ERR_INVALID), (dict(g=None), K.ERR_INVALID), (dict(tokens=None), K.ERR_INVALID),
    (dict(entropy=None), K.ERR_INVALID), (dict(scale=0.0), K.ERR_INVALID), (dict(rows=2**31), K.ERR_UNSUPPORTED),
])
def test_bwd_refuses(lib, change, code):
    assert lib.streamkl_logprobs_bwd(*{**BWD, **change}.values(), None) == code


def test_no_rows_is_no_work(lib):
    assert lib.streamkl_logprobs_fwd(*{**FWD, "rows": 0, "logits": None}.values(), None) == K.OK
    assert lib.streamkl_logprobs_bwd(*{**BWD, "rows": 0, "logits": None}.values(), None) == K.OK


@pytest.mark.parametrize("logits,tokens,error", [
    (torch.zeros(3, 5, dtype=torch.float64), torch.zeros(3, dtype=torch.int64), TypeError),
    (torch.zeros(3, 5), torch.zeros(3), TypeError),
    (torch.zeros(3, 5), torch.zeros(4, dtype=torch.int64), ValueError),
    (torch.zeros(3, 5), torch.zeros(4, 2, dtype=torch.int64), ValueError),
    (torch.zeros(3, 0), torch.zeros(3, dtype=torch.int64), ValueError),
    (torch.zeros(()), None, ValueError),
])
def test_binding_refuses(logits, tokens, error):
    with pytest.raises(error):
        skl.logprobs_fwd(logits, tokens)
