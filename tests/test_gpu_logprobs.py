"""Token log probabilities on the GPU against a plain implementation in 64 bits.

Tolerances, with u = 2^-24 (half a step of fp32), X = max |scale x| over a row's finite logits and n = V / 64 + 64, more
than the additions that any value passes through (a thread adds its columns one by one, 8 or 4 to a vector; then
lanes, warps and blocks):
  * an exponent y - m is off by at most u (|y| + |m| + ...) <= 4 X u log2(e) <= 6 X u, 2^d by a relative 2^-22 = 4 u (the
    bound of ex2.approx) plus that, a sum of them by n u more: LSE and log probabilities (one more rounding of |x| and of
    |LSE| <= X + log V each) within E = (16 X + n + 64) u;
  * the entropy is log s - t / s with |t / s| <= H + log V: within (2 + H + log V) E;
  * a gradient is a sum of terms, each off by a relative 4 E (p from a log probability, its product with sums of g):
    within 4 E times the sum of the terms' magnitudes, plus half a step of the result's type.
"""
import math

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import build

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NEG = float("-inf")
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def make(R, V, T, dtype, seed=0, by=3.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(R, V, generator=gen, device="cuda") * by).to(dtype)
    tok = torch.randint(0, V, (R, T), generator=gen, device="cuda")
    return x, tok, gen


def plain(x, tok, scale, top_k):
    """In 64 bits; rows of nothing but -inf as documented."""
    x = x.double()
    y = x * scale
    lse = torch.logsumexp(y, -1)
    none = lse == NEG
    lp = torch.where(none[:, None], torch.full_like(y, NEG), y - lse[:, None])
    H = -torch.where(lp > NEG, lp.exp() * lp, torch.zeros_like(lp)).sum(-1)
    logp = torch.where(tok >= 0, lp.gather(1, tok.clamp(min=0)), torch.zeros_like(tok, dtype=torch.float64))
    top, idx = torch.sort(x, dim=-1, descending=True, stable=True)
    return logp, H, lse, lp.gather(1, idx[:, :top_k]), idx[:, :top_k], lp


def bound(x, scale):
    V = x.shape[-1]
    X = torch.where(x.double() == NEG, torch.zeros_like(x, dtype=torch.float64), x.double() * scale).abs().amax(-1)
    return (16 * X + V / 64 + 128) * U


def near(got, ref, tol, what):
    got = got.double()
    assert torch.equal(got == NEG, ref == NEG), what
    fin = ref != NEG
    err = (got - ref).abs()[fin]
    tol = torch.broadcast_to(tol, ref.shape)[fin]
    assert bool((err <= tol).all()), f"{what}: {float((err / tol).max()):.2f} of the tolerance"


def check_fwd(x, tok, scale, top_k):
    logp, H, lse, top, idx = skl.logprobs_fwd(x, tok, scale, top_k)
    rlogp, rH, rlse, rtop, ridx, _ = plain(x, tok, scale, top_k)
    E = bound(x, scale)
    near(lse, rlse, E, "lse")
    near(logp, rlogp, E[:, None], "logp")
    near(H, rH, (2 + rH + math.log(x.shape[1])) * E, "entropy")
    assert torch.equal(idx, ridx)
    near(top, rtop, E[:, None], "top")


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("R,V,T,top_k", [(1, 1, 1, 1), (3, 2, 2, 2), (5, 7, 1, 3), (2, 31, 3, 31), (4, 33, 1, 32),
                                         (3, 257, 5, 32), (700, 1000, 1, 0), (2, 4097, 3, 20), (3, 5003, 1, 7),
                                         (1, 32768, 4, 32), (9, 50021, 1, 20), (160, 65536, 2, 5), (400, 8191, 40, 1)])
def test_forward(R, V, T, top_k, dtype):
    x, tok, gen = make(R, V, T, dtype, R + V)
    if T > 2:
        tok[:, 1] = -1
        tok[0, 2] = tok[0, 0]
    check_fwd(x, tok, 0.75, top_k)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("V", [40, 5001, 131072])
def test_rows_that_are_hard_to_rank(V, dtype):
    """All equal; falling and rising; few columns left; none left; zeros of both signs; the largest value twice."""
    K = 32
    x, tok, _ = make(8, V, 2, dtype, V)
    x[0] = 1.5
    x[1] = torch.linspace(4, -4, V).to(dtype)
    x[2] = torch.linspace(-4, 4, V).to(dtype)
    keep = torch.tensor([V - 1, V // 2, 3], device="cuda")
    kept = x[3, keep].clone()
    x[3] = NEG
    x[3, keep] = kept
    x[4] = NEG
    x[5] = 0.0
    x[5, ::2] = -0.0
    x[6, V - 1] = x[6, 1] = 30.0
    x[7, : V // 2] = NEG
    check_fwd(x, tok, 1.0, K)
    check_fwd(x, tok, 1.0, 1)


def test_long_rows_of_one_value():
    """2^21 equal logits: LSE = x + log V and H = log V, far past where a running fp32 sum in one thread would stop."""
    x = torch.full((2, 1 << 21), -3.0, device="cuda", dtype=BF)
    logp, H, lse, _, idx = skl.logprobs_fwd(x, torch.zeros(2, dtype=torch.int64, device="cuda"), 1.0, 4)
    n = 21 * math.log(2)
    assert abs(float(lse[0]) - (n - 3)) < 1e-4 and abs(float(H[1]) - n) < 1e-4 and abs(float(logp[0]) + n) < 1e-4
    assert idx.tolist() == [[0, 1, 2, 3]] * 2


def test_values_that_poison_a_row_stay_in_it():
    x, tok, _ = make(4, 3001, 1, BF)
    clean = skl.logprobs_fwd(x, tok, 1.0, 3)
    x[1, 77] = float("nan")
    x[2, 78] = float("inf")
    logp, H, lse, top, idx = skl.logprobs_fwd(x, tok, 1.0, 3)
    assert torch.isnan(H[1:3]).all() and torch.isnan(logp[1:3]).all()
    assert bool((idx >= 0).all()) and bool((idx < 3001).all())
    for a, b in zip((logp, H, lse, top, idx), clean):
        assert torch.equal(a[0], b[0]) and torch.equal(a[3], b[3])
    tok[0, 0] = 3001  # past the vocabulary
    logp, *_ = skl.logprobs_fwd(x, tok, 1.0, 0)
    assert torch.isnan(logp[0, 0]) and torch.equal(logp[3], clean[0][3])


def check_bwd(x, tok, scale, with_entropy, seed=1, out=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    R, V = x.shape
    g = torch.randn(tok.shape, generator=gen, device="cuda")
    gh = torch.randn(R, generator=gen, device="cuda") if with_entropy else None
    _, H, lse, _, _ = skl.logprobs_fwd(x, tok, scale)
    d = skl.logprobs_bwd(x, tok, lse, H, g, gh, scale)
    assert d.dtype == x.dtype and d.shape == x.shape
    rlogp, rH, rlse, _, _, lp = plain(x, tok, scale, 0)
    p = lp.exp()
    gd = torch.where(tok >= 0, g.double(), torch.zeros_like(g, dtype=torch.float64))
    empty = (rlse == NEG)[:, None]
    gd = torch.where(empty, torch.zeros_like(gd), gd)
    ref = torch.zeros_like(p).scatter_add_(1, tok.clamp(min=0), gd) - p * gd.sum(-1, keepdim=True)
    size = torch.zeros_like(p).scatter_add_(1, tok.clamp(min=0), gd.abs()) + p * gd.abs().sum(-1, keepdim=True)
    if with_entropy:
        pull = torch.where(p > 0, lp + rH[:, None], torch.zeros_like(p))
        ref -= gh.double()[:, None] * p * pull
        size += gh.double().abs()[:, None] * p * (torch.where(p > 0, lp.abs(), torch.zeros_like(p)) + rH[:, None])
    ref, size = ref * scale, size * scale
    E = bound(x, scale)[:, None] * (2 + math.log(V))
    half = {BF: 2.0 ** -8, HF: 2.0 ** -11, FP: U}[x.dtype]
    # below the type's normal range a step no longer shrinks; fp32 results below 2^-126 are flushed
    least = {BF: 2.0 ** -126, HF: 2.0 ** -25, FP: 2.0 ** -126}[x.dtype]
    tol = ref.abs() * half + (1 + half) * 4 * E * size + least * (1 + scale)
    err = (d.double() - ref).abs()
    assert bool((err <= tol).all()), f"{float((err / tol).max()):.2f} of the tolerance"
    return d


@pytest.mark.parametrize("with_entropy", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("R,V,T", [(1, 1, 1), (3, 2, 2), (5, 33, 3), (700, 1000, 1), (2, 4097, 600), (9, 50021, 16), (2, 131072, 1)])
def test_backward(R, V, T, dtype, with_entropy):
    x, tok, _ = make(R, V, T, dtype, R + V)
    if T > 2:
        tok[:, 1] = -1
        tok[0, 2] = tok[0, 0]  # one token twice
    check_bwd(x, tok, 0.75, with_entropy)


def test_backward_of_masked_rows():
    x, tok, _ = make(4, 5003, 3, BF)
    x[0, 100:] = NEG
    x[1] = NEG
    x[2, tok[2, 0]] = NEG  # a given token of probability 0
    d = check_bwd(x, tok, 1.0, True)
    assert bool((d[1] == 0).all())


def test_backward_skips_tokens_past_the_vocabulary():
    x, tok, _ = make(2, 1001, 2, FP)
    _, H, lse, _, _ = skl.logprobs_fwd(x, tok)
    g = torch.ones(2, 2, device="cuda")
    far = tok.clone()
    far[0, 1] = 1001
    none = tok.clone()
    none[0, 1] = -1
    assert torch.equal(skl.logprobs_bwd(x, far, lse, H, g), skl.logprobs_bwd(x, none, lse, H, g))


def test_views_shapes_and_types():
    """Strided rows, rows that start off a 16-byte boundary, leading dimensions, int32 tokens, one token a row."""
    x, tok, _ = make(12, 1007, 1, BF)
    base = skl.logprobs_fwd(x, tok, 1.0, 4)
    wide = torch.zeros(12, 1100, device="cuda", dtype=BF)
    wide[:, 13:1020] = x
    for view in (wide[:, 13:1020], x.t().contiguous().t()):
        for a, b in zip(skl.logprobs_fwd(view, tok, 1.0, 4), base):
            torch.testing.assert_close(a, b, rtol=1e-5, atol=1e-5)
        check_bwd(view, tok, 1.0, True)
    a = skl.logprobs_fwd(x.view(3, 4, 1007), tok.view(3, 4).int(), 1.0, 4)
    assert [t.shape for t in a] == [(3, 4), (3, 4), (3, 4), (3, 4, 4), (3, 4, 4)]
    for t, b in zip(a, base):
        assert torch.equal(t.reshape(-1), b.reshape(-1))
    shared = x[:1].expand(12, 1007)  # one row for all
    check_fwd(shared, tok, 1.0, 4)
    logp, H, lse, top, idx = skl.logprobs_fwd(x)  # no tokens, no alternatives
    assert logp.shape == (12, 0) and top.shape == (12, 0) and torch.equal(lse, base[2])
    assert skl.logprobs_fwd(x[:0], tok[:0], 1.0, 4)[0].shape == (0, 1)
    assert skl.logprobs_bwd(x[:0], tok[:0], base[2][:0], None, base[0][:0]).shape == (0, 1007)


def test_host_tensors_and_refusals():
    x, tok, _ = make(3, 500, 2, FP)
    dev = skl.logprobs_fwd(x, tok, 1.0, 2)
    host = skl.logprobs_fwd(x.cpu(), tok.cpu(), 1.0, 2)
    for a, b in zip(dev, host):
        assert b.device.type == "cpu" and torch.equal(a.cpu(), b)
    with pytest.raises(ValueError):
        skl.logprobs_fwd(x, tok, 1.0, 33)
    with pytest.raises(ValueError):
        skl.logprobs_fwd(x, tok.cpu())
    with pytest.raises(skl.StreamKLError):
        skl.logprobs_fwd(x, tok, 0.0)
    with pytest.raises(ValueError):
        skl.logprobs_bwd(x, tok, dev[2], None, dev[0], dev[1])  # a gradient of the entropy without the entropy
    with pytest.raises(ValueError):
        skl.logprobs_bwd(x, tok, dev[2], dev[1], dev[0].double())


def test_runs_are_bit_identical_alone_together_and_replayed():
    x, tok, _ = make(16, 131072, 3, BF)
    want = skl.logprobs_fwd(x, tok, 1.0, 32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = skl.logprobs_fwd(x, tok, 1.0, 32)
    again = skl.logprobs_fwd(x, tok, 1.0, 32)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        logp, H, lse, top, idx = skl.logprobs_fwd(x, tok, 1.0, 32)
        d = skl.logprobs_bwd(x, tok, lse, H, logp, H)
    y = torch.randn_like(x)
    x.copy_(y)
    g.replay()
    for a, b in zip(skl.logprobs_fwd(y, tok, 1.0, 32), (logp, H, lse, top, idx)):
        assert torch.equal(a, b)
    assert torch.equal(d, skl.logprobs_bwd(y, tok, lse, H, logp, H))
    for a, b, c in zip(want, other, again):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_autograd_against_64_bits_and_differences():
    x, tok, gen = make(5, 301, 4, FP)
    w, wh = torch.randn(5, 4, generator=gen, device="cuda"), torch.randn(5, generator=gen, device="cuda")
    leaf = x.clone().requires_grad_()
    logp, H, top, idx = skl.token_logprobs(leaf, tok, 0.5, 3)
    assert not top.requires_grad and not idx.requires_grad
    ((logp * w).sum() + (H * wh).sum()).backward()
    ref = x.double().requires_grad_()
    lp = torch.log_softmax(ref * 0.5, -1)
    loss = lambda l: (l.gather(1, tok) * w.double()).sum() - ((l.exp() * l).sum(-1) * wh.double()).sum()  # noqa: E731
    loss(lp).backward()
    scale = ref.grad.abs().max()
    assert float((leaf.grad.double() - ref.grad).abs().max() / scale) < 1e-5
    way = torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)
    h = 1e-4
    slope = (loss(torch.log_softmax((x.double() + h * way) * 0.5, -1)) - loss(torch.log_softmax((x.double() - h * way) * 0.5, -1))) / (2 * h)
    assert abs(float((leaf.grad.double() * way).sum() - slope)) < 1e-4 * max(1.0, abs(float(slope)))
    # one output alone, and neither
    leaf.grad = None
    skl.token_logprobs(leaf, tok, 0.5)[1].sum().backward()
    assert leaf.grad is not None
    assert not skl.token_logprobs(x, tok)[0].requires_grad
