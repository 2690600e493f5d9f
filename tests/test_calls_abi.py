"""The native caller on the CPU: what it leaves to the step-by-step path, and that the refusals there are the same."""
import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib, build

BF = torch.bfloat16


@pytest.fixture(scope="module")
def calls():
    build.build()
    return _lib.calls()


def test_host_tensors_are_left_to_the_other_path(calls):
    q, lse = torch.zeros(1, 2, 4, 64, dtype=BF), torch.zeros(1, 2, 4)
    assert calls.attn_fwd(q, q, q, None, False, None, None) is None
    assert calls.attn_bwd(q, q, q, q, lse, q, None, None, False, None, None, 0) is None
    x, t = torch.zeros(3, 10), torch.zeros(3, dtype=torch.int64)
    assert calls.logprobs_fwd(x, t, 1.0, 0) is None
    assert calls.logprobs_bwd(x, t, x[:, 0], None, x[:, 0], None, 1.0) is None


@pytest.mark.parametrize("args", [(), (1,), (None,) * 4, (None,) * 7, (1.5, "a", [], {}, (), None, True), (None,) * 12,
                                  (object(),) * 12, (torch.float32,) * 7, (1 << 70,) * 4])
def test_other_arguments_are_left_to_the_other_path(calls, args):
    for name in ("attn_fwd", "attn_bwd", "logprobs_fwd", "logprobs_bwd"):
        assert getattr(calls, name)(*args) is None


def test_no_keywords(calls):
    with pytest.raises(TypeError):
        calls.attn_fwd(q=None)


def test_missing_module_is_an_error_with_the_way_out(monkeypatch):
    import builtins
    real = builtins.__import__

    def refuse(name, globals=None, locals=None, fromlist=(), level=0):
        if fromlist and "_calls" in fromlist:
            raise ImportError("no _calls here")
        return real(name, globals, locals, fromlist, level)

    monkeypatch.setattr(_lib, "_calls", None)
    monkeypatch.setattr(builtins, "__import__", refuse)
    q = torch.zeros(1, 1, 1, 64, dtype=BF)
    with pytest.raises(RuntimeError, match="build"):
        skl.attn_fwd(q, q, q)
