"""Token log probabilities of logits at the ends of their type's range and far from zero, against 64 bits.

Tolerances.  u = 2^-24.  With m a row's largest logit, everything but the LSE itself is formed from differences to m, so the
bounds below do not grow with |m|: an exponent d = (x - m) c is off by 3 u |d| (its rounding, and c's two), a weight 2^d by
that and 2^-22 (ex2.approx), and the sum of the weights, where sum p |d| <= H + log V in all, by
    E = (16 (1 + log V) + V / 64 + 128) u
with the additions (test_gpu_logprobs.py).  A log probability -- a difference, a product and a sum more -- is within
E + 4 u |log p|, the entropy within (2 + H + log V) E, the LSE within E + 2 u |LSE|.  A gradient's terms are each off by
a relative 4 (2 + log V) E, plus 2 u |LSE| where the LSE is at most 256, above which it is formed again; then half a step of the type.
"""
import ctypes
import math

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib, build

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NEG = float("-inf")
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
HALF = {BF: 2.0 ** -8, HF: 2.0 ** -11, FP: U}
LEAST = {BF: 2.0 ** -126, HF: 2.0 ** -25, FP: 2.0 ** -126}


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def rows(V, dtype):
    """Rows that an ordinary mask or an overflowing head leaves: everything masked, few left, the ends of the range, and
    logits far from zero that differ by little."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    n = torch.randn(10, V, generator=gen, device="cuda")
    x = (n * 3).to(dtype)
    x[0] = low                                  # a mask of the lowest value that leaves nothing
    x[1, 3:] = low                              # ... that leaves three columns
    x[2] = low
    x[2, ::2] = NEG
    x[3] = high
    x[3, V // 2:] = low
    x[4] = low
    x[4, V - 1] = low * 0.75
    x[5, 7] = high
    x[6] = (n[6] * 3 + (5000 if dtype == FP else 0)).to(dtype)
    x[7] = (n[7] * 3 - (200000 if dtype == FP else 300)).to(dtype)
    x[8] = NEG
    x[8, V // 3] = low
    x[9] = NEG
    return x


def plain(x, scale):
    """(LSE, log probabilities, entropy) in 64 bits, from differences to the largest logit."""
    x = x.double()
    m = x.amax(-1, keepdim=True)
    none = m == NEG
    d = (x - torch.where(none, torch.zeros_like(m), m)) * scale
    rest = torch.logsumexp(d, -1, keepdim=True)
    lp = torch.where(none, torch.full_like(d, NEG), d - rest)
    H = -torch.where(lp > NEG, lp.exp() * lp, torch.zeros_like(lp)).sum(-1)
    end = torch.finfo(torch.float32).max
    lse = torch.where(none, m, (m * scale + rest).clamp(-end, end))
    return lse.squeeze(-1), lp, H


def near(got, ref, tol, what):
    got, tol = got.double(), torch.broadcast_to(tol, ref.shape)
    assert torch.equal(got == NEG, ref == NEG), what
    err = (got - ref).abs()
    fin = ref != NEG
    assert bool((err <= tol)[fin].all()), f"{what}: {(err / tol)[fin].max().item():.2f} of the tolerance"


@pytest.mark.parametrize("scale", [1.0, 0.7, 3.0])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("V", [13, 40, 5001, 131072])
def test_ends_of_the_range(V, dtype, scale):
    x = rows(V, dtype)
    R, K = x.shape[0], min(V, 9)
    lse, lp, H = plain(x, scale)
    tok = torch.tensor([0, 3, V - 1, V // 2], device="cuda").expand(R, 4).contiguous()
    logp, entropy, got_lse, top, idx = skl.logprobs_fwd(x, tok, scale, K)
    E = (16 * (1 + math.log(V)) + V / 64 + 128) * U
    size = torch.where(lse.isinf(), torch.zeros_like(lse), lse.abs())
    near(got_lse, lse, E + 2 * U * size, "lse")
    ref = torch.where(lp.gather(1, tok).float() == NEG, torch.full_like(lp[:, :4], NEG), lp.gather(1, tok))  # past fp32's range
    near(logp, ref, E + 4 * U * torch.where(ref == NEG, torch.zeros_like(ref), ref.abs()), "logp")
    near(entropy, H, (2 + H + math.log(V)) * E, "entropy")
    order = torch.sort(x.double(), dim=-1, descending=True, stable=True).indices[:, :K]
    assert torch.equal(idx, order)
    ref = torch.where(lp.gather(1, order).float() == NEG, torch.full_like(lp[:, :K], NEG), lp.gather(1, order))
    near(top, ref, E + 4 * U * torch.where(ref == NEG, torch.zeros_like(ref), ref.abs()), "top")


@pytest.mark.parametrize("scale", [1.0, 0.7, 3.0])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("V", [13, 5001, 131072])
def test_gradients_at_the_ends_of_the_range(V, dtype, scale):
    x = rows(V, dtype)
    R = x.shape[0]
    lse, lp, H = plain(x, scale)
    tok = torch.tensor([0, 3, V - 1], device="cuda").expand(R, 3).contiguous()
    gen = torch.Generator(device="cuda").manual_seed(1)
    g, gh = torch.randn(R, 3, generator=gen, device="cuda"), torch.randn(R, generator=gen, device="cuda")
    _, entropy, got_lse, _, _ = skl.logprobs_fwd(x, tok, scale)
    d = skl.logprobs_bwd(x, tok, got_lse, entropy, g, gh, scale)
    p = lp.exp()
    gd = torch.where((lse == NEG)[:, None], torch.zeros_like(g, dtype=torch.float64), g.double())
    l0 = torch.where(p > 0, lp, torch.zeros_like(lp))
    want = torch.zeros_like(p).scatter_add_(1, tok, gd) - p * gd.sum(-1, keepdim=True) - gh.double()[:, None] * p * (l0 + H[:, None])
    size = (torch.zeros_like(p).scatter_add_(1, tok, gd.abs()) + p * gd.abs().sum(-1, keepdim=True)
            + gh.double().abs()[:, None] * p * (l0.abs() + H[:, None]))
    want, size = want * scale, size * scale
    trusted = lse.abs() <= 256 * (1 + U)
    E = (16 * (1 + math.log(V)) + V / 64 + 128) * U + torch.where(trusted, 2 * U * lse.abs(), torch.zeros_like(lse))
    tol = want.abs() * HALF[dtype] + (1 + HALF[dtype]) * 4 * (2 + math.log(V)) * E[:, None] * size + LEAST[dtype] * (1 + scale)
    err = (d.double() - want).abs()
    assert bool((err <= tol).all()), f"{float((err / tol).max()):.2f} of the tolerance"


def test_gradient_onto_the_logits():
    """The C entry writes the entropy's gradient over the logits themselves; a row whose LSE is formed again is read whole
    before it is written.  The same bits as beside them."""
    for dtype, V in ((BF, 131072), (FP, 5001)):
        x = rows(V, dtype)[[0, 1, 4, 5, 6, 7]].contiguous()
        R = x.shape[0]
        _, H, lse, _, _ = skl.logprobs_fwd(x)
        gh = torch.ones(R, device="cuda")
        want = skl.logprobs_bwd(x, None, lse, H, None, gh)
        y = x.clone()
        status = _lib.lib().streamkl_logprobs_bwd(
            y.data_ptr(), _lib.DTYPES[dtype], R, V, V, None, 0, 1.0, lse.data_ptr(), H.data_ptr(), None, gh.data_ptr(),
            y.data_ptr(), V, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert status == _lib.OK and torch.equal(y, want)


def test_a_row_masked_whole_is_uniform_for_autograd():
    """What a training step sees where its mask of the lowest value leaves nothing: log V, and a gradient of g ([j = t] - 1 / V)."""
    V = 1000
    x = torch.full((2, V), torch.finfo(FP).min, device="cuda").requires_grad_()
    tok = torch.tensor([5, 999], device="cuda")
    logp, entropy, _, _ = skl.token_logprobs(x, tok)
    assert torch.allclose(logp, torch.full_like(logp, -math.log(V)), rtol=1e-6)
    assert torch.allclose(entropy, torch.full_like(entropy, math.log(V)), rtol=1e-5)
    logp.sum().backward()
    want = torch.full((2, V), -1.0 / V, device="cuda")
    want[0, 5] += 1
    want[1, 999] += 1
    assert torch.allclose(x.grad, want, rtol=1e-5, atol=1e-9)
