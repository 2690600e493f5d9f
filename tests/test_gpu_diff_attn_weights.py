"""Differential attention's backward: nothing is rounded for lam's sake.

With queries of 0 every key has the weight 1 / N_K, exact for 1, 2 and 4 keys.  A lam of whole 128ths below 1.5 leaves |lam| P2
exact in bf16 as well (its exponent is off by a few u = 2^-24, far less than half a step), so that
    dV_j = sum over rows and pairs of (1 - lam) dO / N_K
has no rounding but those of its fp32 sum, n u of the terms' magnitudes for n terms, and of the result, h = 2^-8 of it.  With
-lam dO rounded to bf16 first, a single row's dV at lam = 127/128 would be off by up to half of itself.
"""
import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib as K
from tests import attn_util as A

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,mode", [(64, K.BWD_SEPARATE), (64, K.BWD_FUSED), (128, K.BWD_SEPARATE)])
@pytest.mark.parametrize("B,Hd,HK,NQ", [(1, 1, 1, 1), (2, 3, 3, 1), (1, 4, 2, 2), (2, 2, 1, 130)])
@pytest.mark.parametrize("NK", [1, 2, 4])
@pytest.mark.parametrize("dlse", [False, True])
def test_weights_of_whole_128ths(dlse, NK, B, Hd, HK, NQ, D, mode):
    gen = torch.Generator(device="cuda").manual_seed(D + NQ + NK)
    q = torch.zeros(B, 2 * Hd, NQ, D, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn(B, HK, NK, D, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    do = torch.randn(B, Hd, NQ, D, generator=gen, device="cuda").to(torch.bfloat16)
    lam = torch.randint(2, 192, (B, Hd, NQ), generator=gen, device="cuda") / 128.0  # from 1/64 on
    lam *= torch.where(torch.rand(lam.shape, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    lam[0, 0, 0] = 127 / 128
    z = torch.randn(B, 2 * Hd, NQ, generator=gen, device="cuda") if dlse else None
    d, lse, maps, rest = skl.diff_attn_fwd(q, k, v, lam, return_maps=True)
    _, _, dv, _ = skl.diff_attn_bwd(q, k, v, lam, maps, lse, do, dlse=z, bwd_mode=mode, maps_rest=rest)

    def sums(x):  # over rows and a key head's pairs, for each key
        return x.view(B, HK, Hd // HK, NQ, D).sum((2, 3))[:, :, None].expand(B, HK, NK, D) / NK

    one, two = do.double(), lam.double()[..., None] * do.double()
    ref, size = sums(one - two), sums(one.abs() + two.abs())
    bound = A.H * ref.abs() + (2 * NQ * Hd // HK + 8) * A.U * size + 2.0 ** -126
    A.within(dv, ref, bound, "dv")
    if NQ == 1:  # the bound would show a rounding of lam dO
        planted = sums(one - (lam[..., None] * do.float()).to(torch.bfloat16).double())
        assert bool(((planted - ref).abs() > bound).any())
    assert skl.check_device_status() == K.OK
