"""Differential attention's backward where the program has asked PyTorch for deterministic algorithms."""
import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib, build
from tests.test_gpu_diff_attn import inputs


@pytest.fixture
def deterministic():
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(False)


class Modes:
    """A native caller that notes the mode it is called with."""
    def __init__(self):
        self.seen = []

    def diff_attn_bwd(self, *a):
        self.seen.append(a[12])
        return a[0], a[1], a[2], a[3]


def modes(monkeypatch):
    calls = Modes()
    monkeypatch.setattr(_lib, "_calls", calls)
    q, lse, lam = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 2), torch.zeros(1)
    for mode in (skl.BWD_AUTO, skl.BWD_FUSED, skl.BWD_SEPARATE):
        skl.diff_attn_bwd(q, q[:, :1], q[:, :1], lam, q, lse, q[:, :1], bwd_mode=mode, maps_rest=q)
    return calls.seen


def test_auto_takes_the_fixed_order(monkeypatch, deterministic):
    assert modes(monkeypatch) == [skl.BWD_SEPARATE, skl.BWD_FUSED, skl.BWD_SEPARATE]


def test_auto_is_left_to_the_library_otherwise(monkeypatch):
    assert modes(monkeypatch) == [skl.BWD_AUTO, skl.BWD_FUSED, skl.BWD_SEPARATE]


@pytest.mark.gpu
def test_autograd_gives_the_same_bits(deterministic):
    """A shape whose AUTO is the path that adds dq up in no fixed order; lam has one value to a head."""
    build.build()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert skl.attn_bwd_plan(4, 40, 20, 300, 500, 64, sms)[0] == skl.BWD_FUSED
    q, k, v, lam, do = inputs(4, 20, 20, 300, 500, 64, 1)
    leaves = [t.requires_grad_() for t in (q, k, v, lam[:1, :, :1].clone())]
    runs = [torch.autograd.grad(skl.differential_attention(*leaves), leaves, do) for _ in range(3)]
    for got in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got, runs[0]))
