"""Cross entropy over a vocabulary of no rows: an empty tensor has no address, and its gradient is empty."""
import ctypes

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib as K
from attention_kl_divergence_streamkl_gb300 import build as B


def bwd(lib, dh, dw, rows=0):
    at = ctypes.c_void_p(0x10000000)
    return lib.streamkl_vocab_xent_bwd(at, at, at, at, at, None, K.make_xent_shape(rows, 100, 64), dh, dw, None, 0, None)


def test_an_empty_dhidden_has_no_address():
    B.build()
    lib = K.lib()
    assert bwd(lib, None, None) == K.OK
    assert bwd(lib, ctypes.c_void_p(0x10000100), None) == K.OK
    assert bwd(lib, ctypes.c_void_p(0x10000108), None) == K.ERR_INVALID
    assert bwd(lib, None, ctypes.c_void_p(0x10000108)) == K.ERR_INVALID
    assert bwd(lib, None, None, rows=1) == K.ERR_INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lead", [(0,), (3, 0)])
def test_gradients_of_no_rows(lead, dtype):
    h = torch.empty(*lead, 64, device="cuda", dtype=dtype)
    w = torch.ones(100, 64, device="cuda", dtype=dtype)
    t, none = torch.empty(lead, device="cuda", dtype=torch.int64), torch.empty(lead, device="cuda")
    for want in ((True, True), (True, False), (False, True), (False, False)):
        dh, dw = skl.vocab_xent_bwd(h, w, t, none, none, want_dhidden=want[0], want_dweight=want[1])
        assert dh.shape == h.shape if want[0] else dh is None
        assert dw.shape == w.shape and not bool(dw.any()) if want[1] else dw is None


@pytest.mark.gpu
@pytest.mark.parametrize("frozen", ["weight", "hidden", "none"])
def test_a_mask_that_leaves_no_row(frozen):
    h = torch.randn(20, 64, device="cuda").to(torch.bfloat16).requires_grad_(frozen != "hidden")
    w = torch.randn(100, 64, device="cuda").to(torch.bfloat16).requires_grad_(frozen != "weight")
    t, mask = torch.arange(20, device="cuda"), torch.zeros(20, dtype=torch.bool, device="cuda")
    loss, lse = skl.vocab_cross_entropy(h[mask], w, t[mask], return_lse=True)
    (loss.sum() + lse.sum()).backward()
    for x in (h, w):
        assert x.grad is None if not x.requires_grad else x.grad.shape == x.shape and not bool(x.grad.any())
