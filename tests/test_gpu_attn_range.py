"""Attention forward: values of large size in rows whose logits grow after the first key tile (bounds: attn_util.py)."""
import math

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import build
from tests import attn_util as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    yield
    assert skl.check_device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("NQ,H,HK", [(1, 8, 2), (130, 304, 304), (130, 608, 38)])
@pytest.mark.parametrize("grow", [8.0, 30.0, 43.0])
def test_large_values(grow, NQ, H, HK, D):
    """Keys after the first tile bring logits larger by `grow` (43: a factor of 2^62 of the weights), the values are 2^80 and 2^88;
    with keys split over blocks (one query) and with one block that sees them all."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert (skl.attn_fwd_plan(1, H, HK, NQ, 700, D, sms)[1] == 1) == (NQ > 1)
    gen = torch.Generator(device="cuda").manual_seed(D)
    base = torch.randn(D, generator=gen, device="cuda")
    base *= math.sqrt(D) / base.norm()
    q = (base + 0.1 * torch.randn(1, H, NQ, D, generator=gen, device="cuda")).to(torch.bfloat16)
    k = 0.2 * torch.randn(1, HK, 700, D, generator=gen, device="cuda")
    k[:, :, 200:] += base * (grow / math.sqrt(D)) * torch.linspace(0.5, 1, 500, device="cuda").view(1, 1, -1, 1)
    k = k.to(torch.bfloat16)
    for exponent in (80, 88):
        v = (torch.randn(1, HK, 700, D, generator=gen, device="cuda").clamp(-1, 1) * 2.0 ** exponent).to(torch.bfloat16)
        o, lse = skl.attn_fwd(q, k, v)
        ro, rlse, bo, bl, _, _ = A.forward(q, k, v)
        A.within(lse, rlse, bl, "lse")
        A.within(o, ro, bo, "o")
