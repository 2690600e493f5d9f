"""The native caller of rotary positions, differential attention and the vocabulary's cross entropy, on the CPU: what it leaves
to the step-by-step path."""
import pytest
import torch

from attention_kl_divergence_streamkl_gb300 import _lib, build

BF = torch.bfloat16
NAMES = ("rotary", "diff_attn_fwd", "diff_attn_bwd", "vocab_xent_fwd", "vocab_xent_bwd")


@pytest.fixture(scope="module")
def calls():
    build.build()
    return _lib.calls()


def test_host_tensors_are_left_to_the_other_path(calls):
    q, k, lse, lam = torch.zeros(1, 4, 8, 64, dtype=BF), torch.zeros(1, 2, 8, 64, dtype=BF), torch.zeros(1, 4, 8), torch.zeros(1, 2, 8)
    assert calls.rotary(q, k, torch.zeros(32, dtype=torch.int64), 64, 1.0, None, 0, False, False) is None
    assert calls.diff_attn_fwd(q, k, k, lam, None, False, None, None, False) is None
    assert calls.diff_attn_bwd(q, k, k, lam, q, lse, q[:, :2], None, None, False, None, None, 0, q) is None
    h, w, t, r = torch.zeros(3, 8, dtype=BF), torch.zeros(5, 8, dtype=BF), torch.zeros(3, dtype=torch.int64), torch.zeros(3)
    assert calls.vocab_xent_fwd(h, w, t, 1.0) is None
    assert calls.vocab_xent_bwd(h, w, t, r, r, None, 1.0) is None


@pytest.mark.parametrize("args", [(), (1,), *[(None,) * n for n in (4, 7, 9, 14)], *[(object(),) * n for n in (4, 7, 9, 14)],
                                  *[(1 << 70,) * n for n in (4, 7, 9, 14)], (1.5, "a", [], {}, (), None, True, 2, b"")])
def test_other_arguments_are_left_to_the_other_path(calls, args):
    for name in NAMES:
        assert getattr(calls, name)(*args) is None
