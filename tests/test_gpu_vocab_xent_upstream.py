"""Cross entropy over a vocabulary: upstream gradients that have no effect have none on the others' digits either.

In fp16 d is multiplied by one power of two for all rows.  It is taken from the gradients that are used: not from g_loss of
a row without a token, whatever it holds, and not from values that are not finite.  So the bits are those of a call with 0
there, and the bounds those of test_gpu_vocab_xent.py with 0 there.
"""
import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib as K
from tests import test_gpu_vocab_xent as X

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("what", [1e4, 1e8, 1e30, INF, -INF, NAN])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("with_lse", [False, True])
@pytest.mark.parametrize("R,C,V", [(64, 72, 5001), (1200, 64, 300)])
def test_rows_without_a_token_have_no_say(R, C, V, with_lse, dtype, what):
    h, w, t = X.inputs(R, C, V, dtype, 31, none=0.3)
    t[3], t[4], t[5], t[6], t[R - 1] = V, 2 ** 40, -2 ** 63, 1, -1
    off = (t < 0) | (t >= V)
    gen = torch.Generator(device="cuda").manual_seed(32)
    g = torch.where(off, 0.0, (torch.rand(R, generator=gen, device="cuda") + 0.5) / 4096)
    gl = torch.randn(R, generator=gen, device="cuda") / 4096 if with_lse else None
    _, lse = skl.vocab_xent_fwd(h, w, t)
    ref = skl.vocab_xent_bwd(h, w, t, lse, g, gl)
    got = skl.vocab_xent_bwd(h, w, t, lse, torch.where(off, what, g), gl)
    for a, b, r, bound, name in zip(got, ref, *zip(*_formulas(h, w, t, g, gl)), ("dhidden", "dweight")):
        X.within(a, r, bound, name)
        assert torch.equal(a, b), name
    assert skl.check_device_status() == K.OK


def _formulas(h, w, t, g, gl):
    rh, rw, bh, bw = X.backward(h, w, t, g, gl, 1.0)
    return (rh, bh), (rw, bw)


@pytest.mark.parametrize("what", [INF, -INF, NAN])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("of_lse", [False, True])
def test_a_gradient_that_is_not_finite_stays_in_its_row(of_lse, dtype, what):
    """dhidden of the other rows; dweight sums over all of them and is not finite."""
    R = 100
    h, w, t = X.inputs(R, 64, 3000, dtype, 33, none=0.0)
    gen = torch.Generator(device="cuda").manual_seed(34)
    g = torch.rand(R, generator=gen, device="cuda") / 4096
    gl = torch.rand(R, generator=gen, device="cuda") / 4096
    g[7] = gl[7] = 0.0
    _, lse = skl.vocab_xent_fwd(h, w, t)
    ref, _ = skl.vocab_xent_bwd(h, w, t, lse, g, gl)
    (gl if of_lse else g)[7] = what
    got, _ = skl.vocab_xent_bwd(h, w, t, lse, g, gl)
    others = torch.arange(R, device="cuda") != 7
    assert torch.equal(got[others], ref[others]) and not bool(got[7].isfinite().any())


def test_a_sequence_without_tokens_in_a_mean_over_sequences():
    """Losses weighted by one over their sequence's tokens, at least 1e-8: the upstream gradient of an empty sequence is 1e8."""
    h, w, t = X.inputs(96, 64, 5001, "fp16", 35, none=0.2)
    t = t.view(4, 24)
    t[2] = -1
    a, b = h.clone().view(4, 24, 64).requires_grad_(), w.clone().requires_grad_()
    count = (t >= 0).sum(1)
    (skl.vocab_cross_entropy(a, b, t).sum(1) / count.clamp(min=1e-8)).sum().backward()
    g = torch.where(t >= 0, 1.0 / count.clamp(min=1e-8)[:, None], 0.0)
    rh, rw, bh, bw = X.backward(h, w, t.view(-1), g.view(-1).float(), None, 1.0)
    X.within(a.grad.view(96, 64), rh, bh, "hidden")
    X.within(b.grad, rw, bw, "weight")
