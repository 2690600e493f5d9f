"""The native caller of rotary positions, differential attention and the vocabulary's cross entropy against the
step-by-step path: the same tensors, bit for bit, and the ordinary calls are taken."""
import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import build
from tests import attn_util as A
from tests.test_gpu_calls import both, lens

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    yield
    assert skl.check_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, torch.float16, torch.float32])
@pytest.mark.parametrize("rows_first", [False, True])
@pytest.mark.parametrize("given", [None, "wide", "narrow", "one"])
def test_rotary(monkeypatch, dtype, rows_first, given):
    q, k, _, _ = A.tensors(3, 4, 2, 17, 17, 64, 1, rows_first)
    q, k = q.to(dtype), k.to(dtype)
    plan = skl.rotary_plan(32, scaling="parts", factor=4.0, trained_length=512)
    at = torch.randint(0, 5000, (3, 17), device="cuda")
    kw = dict(positions=None if given is None else at[0] if given == "one" else at.int() if given == "narrow" else at,
              offset=9 if given is None else 0, interleaved=rows_first)
    assert both(monkeypatch, lambda: skl.rotary_fwd(q, k, plan, **kw)) == [True]
    assert both(monkeypatch, lambda: skl.rotary_bwd(q, k, plan, **kw)) == [True]


def test_rotary_leaves_the_rest_to_the_other_path(monkeypatch):
    q, k, _, _ = A.tensors(2, 4, 2, 9, 9, 64, 2)
    plan = skl.rotary_plan(64)
    assert both(monkeypatch, lambda: skl.rotary_fwd(q.transpose(2, 3).contiguous().transpose(2, 3), k, plan)) == [False]
    assert both(monkeypatch, lambda: skl.rotary_fwd(q[:, :1].expand(2, 4, 9, 64), k, plan)) == [False]
    assert both(monkeypatch, lambda: skl.rotary_fwd(q, k, plan, torch.arange(18, device="cuda")[::2])) == [False]


@pytest.mark.parametrize("rows_first", [False, True])
@pytest.mark.parametrize("shape", [(2, 2, 130), (2, 130), (1, 1), (2, 2, 1), (130,)])
def test_differential_attention(monkeypatch, rows_first, shape):
    q, k, v, do = A.tensors(2, 4, 1, 130, 200, 64, 3, rows_first)
    do = do[:, :2]
    if rows_first:
        do = do.transpose(1, 2).contiguous().transpose(1, 2)
    lam = torch.rand(shape, device="cuda")
    kw = dict(scale=0.3, causal=True, q_lens=lens(130, 129), k_lens=lens(101, 200))
    assert both(monkeypatch, lambda: skl.diff_attn_fwd(q, k, v, lam, **kw)) == [True]
    assert both(monkeypatch, lambda: skl.diff_attn_fwd(q, k, v, lam, return_maps=True, **kw)) == [True]
    _, lse, maps, rest = skl.diff_attn_fwd(q, k, v, lam, return_maps=True, **kw)
    dlse = torch.randn_like(lse)
    do = do.contiguous() if not rows_first else do
    taken = both(monkeypatch, lambda: skl.diff_attn_bwd(q, k, v, lam, maps, lse, do, dlse, bwd_mode=skl.BWD_SEPARATE,
                                                       maps_rest=rest, **kw))
    assert taken == [True]


def test_differential_attention_leaves_the_rest_to_the_other_path(monkeypatch):
    q, k, v, _ = A.tensors(1, 4, 2, 8, 20, 64, 4)
    lam = torch.rand(1, device="cuda")
    assert both(monkeypatch, lambda: skl.diff_attn_fwd(q, k, v, lam[0])) == [False]
    wide = torch.randn(1, 4, 8, 72, device="cuda").to(BF)[..., 4:68]
    assert both(monkeypatch, lambda: skl.diff_attn_fwd(wide, k, v, lam)) == [False]


@pytest.mark.parametrize("dtype", [BF, torch.float16])
@pytest.mark.parametrize("lead", [(50,), (2, 25), ()])
def test_cross_entropy(monkeypatch, dtype, lead):
    gen = torch.Generator(device="cuda").manual_seed(5)
    h = torch.randn(*lead, 72, generator=gen, device="cuda").to(dtype)
    w = (torch.randn(300, 80, generator=gen, device="cuda") / 8).to(dtype)[:, :72]
    t = torch.randint(-1, 300, lead, generator=gen, device="cuda")
    assert both(monkeypatch, lambda: skl.vocab_xent_fwd(h, w, t, 0.5)) == [True]
    _, lse = skl.vocab_xent_fwd(h, w, t, 0.5)
    g = torch.rand_like(lse)
    for gl in (None, torch.rand_like(lse)):
        assert both(monkeypatch, lambda: skl.vocab_xent_bwd(h, w, t, lse, g, gl, 0.5)) == [True]
    assert both(monkeypatch, lambda: skl.vocab_xent_fwd(h, w, t.int(), 0.5)) == [False]
