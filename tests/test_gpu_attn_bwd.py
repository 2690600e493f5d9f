"""Attention backward on the GPU against the formulas in 64 bits (bounds: attn_util.py) and against differences."""
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


def lens(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


def modes(D):
    return {"separate": skl.BWD_SEPARATE, **({"fused": skl.BWD_FUSED} if D == 64 else {})}


def check(q, k, v, do, dlse=None, **kw):
    """Every path; returns the separate one's."""
    o, lse = skl.attn_fwd(q, k, v, **kw)
    want, bounds = A.backward(q, k, v, do, dlse, **kw)
    out = {}
    for mode, value in modes(q.shape[3]).items():
        out[mode] = skl.attn_bwd(q, k, v, o, lse, do, dlse, **kw, bwd_mode=value)
        for name, g, w, b in zip(("dq", "dk", "dv"), out[mode], want, bounds):
            A.within(g, w, b, f"{mode} {name}")
    return out["separate"]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,H,HK,NQ,NK", [
    (1, 1, 1, 1, 1), (1, 1, 1, 2, 2), (2, 2, 1, 1, 2), (1, 4, 2, 3, 127), (1, 3, 3, 128, 128), (1, 2, 2, 129, 129),
    (2, 6, 2, 255, 300), (1, 2, 1, 256, 256), (1, 2, 2, 257, 511), (1, 8, 1, 16, 1000), (1, 1, 1, 600, 640),
    (1, 1, 1, 300, 100), (1, 6, 3, 500, 70), (1, 2, 2, 1000, 1000),
    # long streams of few tiles, dealt out over several blocks
    (1, 2, 1, 100, 4200), (1, 8, 1, 1200, 90), (2, 1, 1, 2100, 2200), (1, 4, 1, 2100, 60)])
def test_backward(B, H, HK, NQ, NK, causal, D):
    q, k, v, do = A.tensors(B, H, HK, NQ, NK, D, B + NQ + NK)
    check(q, k, v, do, causal=causal)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("NQ,NK,G", [(1, 700, 4), (200, 333, 2), (400, 400, 1), (513, 300, 3)])
def test_padded_batch_whatever_lies_in_the_padding(NQ, NK, G, causal, D):
    ql = lens(NQ, NQ, max(NQ - 3, 1), 0, NQ + 9, NQ // 2 + 1)
    kl = lens(NK, 1, NK - 130, NK, -4, NK // 2)
    q, k, v, do = A.tensors(6, 2 * G, 2, NQ, NK, D, 3)
    dlse = torch.randn(6, 2 * G, NQ, device="cuda")
    for b in range(6):
        past_q, past_k = max(min(int(ql[b]), NQ), 0), max(min(int(kl[b]), NK), 0)
        q[b, :, past_q:] = do[b, :, past_q:] = float("nan")
        dlse[b, :, past_q:] = float("nan")
        k[b, :, past_k:] = float("nan")
        v[b, :, past_k:] = float("inf")
    clean = torch.where(dlse.isnan(), torch.zeros_like(dlse), dlse)
    o, lse = skl.attn_fwd(q, k, v, causal=causal, q_lens=ql, k_lens=kl)
    want, bounds = A.backward(q, k, v, do, clean, causal=causal, q_lens=ql, k_lens=kl)
    for mode, value in modes(D).items():
        got = skl.attn_bwd(q, k, v, o, lse, do, dlse, causal=causal, q_lens=ql, k_lens=kl, bwd_mode=value)
        for name, g, w, b in zip(("dq", "dk", "dv"), got, want, bounds):
            A.within(g, w, b, f"{mode} {name}")
        for b in range(6):
            past_q, past_k = max(min(int(ql[b]), NQ), 0), max(min(int(kl[b]), NK), 0)
            assert bool((got[0][b, :, past_q:] == 0).all())
            assert bool((got[1][b, :, past_k:] == 0).all()) and bool((got[2][b, :, past_k:] == 0).all())


def test_gradient_of_the_log_sum_exp():
    q, k, v, do = A.tensors(2, 4, 2, 200, 150, 128, 11)
    dlse = torch.randn(2, 4, 200, device="cuda") * 5
    check(q, k, v, do, dlse, causal=True)  # the first 50 rows see no key
    check(q, k, v, torch.zeros_like(do), dlse)


def test_scales_and_sharp_rows():
    q, k, v, do = A.tensors(1, 2, 1, 300, 400, 64, 12, by=3.0)
    check(q, k, v, do, scale=1.0)
    check(q, k, v, do * 1000, scale=0.02, causal=True)


def test_no_queries_or_no_keys():
    q, k, v, do = A.tensors(2, 4, 2, 30, 40, 64, 13)
    o, lse = skl.attn_fwd(q, k[:, :, :0], v[:, :, :0])
    dq, dk, dv = skl.attn_bwd(q, k[:, :, :0], v[:, :, :0], o, lse, do)
    assert bool((dq == 0).all()) and dk.shape == (2, 2, 0, 64)
    o, lse = skl.attn_fwd(q[:, :, :0], k, v)
    dq, dk, dv = skl.attn_bwd(q[:, :, :0], k, v, o, lse, do[:, :, :0])
    assert dq.shape == (2, 4, 0, 64) and bool((dk == 0).all()) and bool((dv == 0).all())


def test_views():
    """Any storage order for each tensor by itself; gradients keep the layout of their input."""
    q, k, v, do = A.tensors(2, 4, 2, 140, 260, 64, 14, rows_first=True)
    dq, dk, dv = check(q, k, v, do, causal=True)
    assert dq.stride() == q.stride() and dk.stride() == k.stride()
    check(q, k.contiguous(), v, do.contiguous())
    packed = torch.randn(2, 140, 8, 64, device="cuda").to(torch.bfloat16)
    qkv = [packed[:, :, a:b].transpose(1, 2) for a, b in ((0, 4), (4, 6), (6, 8))]
    check(*qkv, do, causal=True)
    one = torch.randn(2, 4, 1, 1, device="cuda").to(torch.bfloat16).expand(2, 4, 140, 64)  # a broadcast gradient
    check(q, k, v, one)
    check(q, k[:, :1].expand(2, 2, 260, 64), v, do)


def test_runs_are_bit_identical_alone_together_and_replayed():
    q, k, v, do = A.tensors(1, 8, 2, 700, 900, 128, 15)
    o, lse = skl.attn_fwd(q, k, v, causal=True)
    call = lambda: skl.attn_bwd(q, k, v, o, lse, do, causal=True, bwd_mode=skl.BWD_SEPARATE)  # noqa: E731
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call()
    again = call()
    torch.cuda.current_stream().wait_stream(side)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        first = call()
    with torch.cuda.graph(g2):
        second = call()
    g1.replay()
    g2.replay()
    g1.replay()
    for got in (other, again, first, second):
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_fused_runs_together_and_replayed():
    """The fused path on two streams at once and in two graphs, each with its own accumulator: dk and dv keep their bits,
    dq stays within its bound whatever the order of its additions."""
    q, k, v, do = A.tensors(1, 8, 2, 700, 900, 64, 18)
    o, lse = skl.attn_fwd(q, k, v, causal=True)
    call = lambda: skl.attn_bwd(q, k, v, o, lse, do, causal=True, bwd_mode=skl.BWD_FUSED)  # noqa: E731
    ref = call()
    want, bounds = A.backward(q, k, v, do, causal=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call()
    again = call()
    torch.cuda.current_stream().wait_stream(side)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        first = call()
    with torch.cuda.graph(g2):
        second = call()
    g1.replay()
    g2.replay()
    g1.replay()
    for got in (ref, other, again, first, second):
        A.within(got[0], want[0], bounds[0], "dq")
        assert torch.equal(got[1], ref[1]) and torch.equal(got[2], ref[2])


def test_autograd_against_differences():
    """The slope of a loss of O and LSE along a direction, from the gradients and from differences in 64 bits."""
    q, k, v, w = A.tensors(1, 4, 2, 70, 90, 64, 16)
    wl = torch.randn(1, 4, 70, device="cuda")
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    o, lse = skl.attention(*leaves, causal=True, return_lse=True)
    torch.autograd.backward([o, lse], [w, wl])

    def loss(*t):
        ro, rl, *_ = A.forward(*t, causal=True)
        return (ro * w.double()).sum() + (rl * wl.double()).sum()

    for i in range(3):
        way = torch.randn(leaves[i].shape, device="cuda", dtype=torch.float64)
        h = 1e-4
        at = lambda s: loss(*(t.double() + (s * h * way if j == i else 0) for j, t in enumerate((q, k, v))))  # noqa: E731
        slope = float(at(1) - at(-1)) / (2 * h)
        got = float((leaves[i].grad.double() * way).sum())
        # the bounds of the entries, met by a random sign each: their root of squares, five times
        bound = A.backward(q, k, v, w, wl, causal=True)[1][i]
        assert abs(got - slope) <= 5 * float((bound * way).norm()) + 1e-6 * abs(slope)


def test_autograd_outputs_alone():
    q, k, v, do = A.tensors(1, 2, 2, 40, 50, 64, 17)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    skl.attention(*leaves, bwd_mode=skl.BWD_SEPARATE).backward(do)
    for t, w in zip(leaves, check(q, k, v, do)):
        assert torch.equal(t.grad, w)
    for t in leaves:
        t.grad = None
    skl.attention(*leaves, return_lse=True)[1].sum().backward()
    want, bounds = A.backward(q, k, v, torch.zeros_like(do), torch.ones(1, 2, 40, device="cuda"))
    for t, w, b in zip(leaves, want, bounds):
        A.within(t.grad, w, b, "of the log-sum-exp")
    frozen = q.clone().requires_grad_()
    skl.attention(frozen, k, v).sum().backward()
    assert frozen.grad is not None


@pytest.mark.parametrize("D", [64, 128])
def test_two_streams_side_by_side(D):
    """Forward, merge, and both backward paths of two streams at once, kernels of every kind beside one another on the GPU:
    the bits of the calls made alone."""
    shapes = [(2, 16, 8, 141, 2123, False), (1, 8, 2, 1, 2694, False), (2, 4, 4, 600, 500, True), (1, 4, 1, 300, 1300, True)]
    inputs = [A.tensors(B, H, HK, NQ, NK, D, i) for i, (B, H, HK, NQ, NK, _) in enumerate(shapes)]

    def run(i):
        q, k, v, do = inputs[i]
        o, lse = skl.attn_fwd(q, k, v, causal=shapes[i][5])
        out = [o, lse, *skl.attn_bwd(q, k, v, o, lse, do, causal=shapes[i][5], bwd_mode=skl.BWD_SEPARATE)]
        if D == 64:  # dq's bits depend on the order of the reductions
            out += skl.attn_bwd(q, k, v, o, lse, do, causal=shapes[i][5], bwd_mode=skl.BWD_FUSED)[1:]
        return out

    want = [run(i) for i in range(len(shapes))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for round_ in range(60):
        i, j = round_ % len(shapes), (round_ * 3 + 1) % len(shapes)
        for _ in range(20):
            here = run(i)
            with torch.cuda.stream(side):
                there = run(j)
        torch.cuda.synchronize()
        for got, ref in ((here, want[i]), (there, want[j])):
            assert all(torch.equal(x, y) for x, y in zip(got, ref))
