"""Attention backward where the program has asked PyTorch for deterministic algorithms."""
import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib, build
from tests import attn_util as A


@pytest.fixture
def deterministic():
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(False)


class Modes:
    """A native caller that notes the mode it is called with."""
    def __init__(self):
        self.seen = []

    def attn_bwd(self, *a):
        self.seen.append(a[11])
        return a[0], a[1], a[2]


def modes(monkeypatch):
    calls = Modes()
    monkeypatch.setattr(_lib, "_calls", calls)
    q, lse = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 2)
    for mode in (skl.BWD_AUTO, skl.BWD_FUSED, skl.BWD_SEPARATE):
        skl.attn_bwd(q, q, q, q, lse, q, bwd_mode=mode)
    return calls.seen


def test_auto_takes_the_fixed_order(monkeypatch, deterministic):
    assert modes(monkeypatch) == [skl.BWD_SEPARATE, skl.BWD_FUSED, skl.BWD_SEPARATE]


def test_auto_is_left_to_the_library_otherwise(monkeypatch):
    assert modes(monkeypatch) == [skl.BWD_AUTO, skl.BWD_FUSED, skl.BWD_SEPARATE]


@pytest.mark.gpu
def test_autograd_gives_the_same_bits(deterministic):
    """A shape whose AUTO is the path that adds dq up in no fixed order."""
    build.build()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert skl.attn_bwd_plan(4, 20, 20, 300, 500, 64, sms)[0] == skl.BWD_FUSED
    q, k, v, do = A.tensors(4, 20, 20, 300, 500, 64, 1)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    runs = [torch.autograd.grad(skl.attention(*leaves), leaves, do) for _ in range(3)]
    o, lse, rest = skl.attn_fwd(q, k, v, return_rest=True)
    runs.append(skl.attn_bwd(q, k, v, o, lse, do, bwd_mode=skl.BWD_SEPARATE, o_rest=rest))
    for got in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got, runs[0]))
