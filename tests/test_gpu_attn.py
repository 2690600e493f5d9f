"""Attention forward on the GPU against a plain implementation in 64 bits (bounds: attn_util.py)."""
import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import build
from tests import attn_util as A

pytestmark = pytest.mark.gpu
NEG = float("-inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    yield
    assert skl.check_device_status() == 0


def lens(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


def check(q, k, v, **kw):
    o, lse = skl.attn_fwd(q, k, v, **kw)
    ro, rlse, bo, bl, _, _ = A.forward(q, k, v, **kw)
    A.within(lse, rlse, bl, "lse")
    A.within(o, ro, bo, "o")
    return o, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,H,HK,NQ,NK", [
    (1, 1, 1, 1, 1), (2, 2, 1, 1, 2), (1, 4, 2, 3, 127), (1, 3, 3, 128, 128), (1, 2, 2, 129, 129), (2, 6, 2, 255, 300),
    (1, 2, 1, 256, 256), (1, 2, 2, 257, 511), (1, 8, 1, 16, 1000), (1, 8, 1, 17, 1000), (1, 1, 1, 600, 640),
    (1, 1, 1, 300, 100), (3, 5, 5, 1, 640), (1, 16, 2, 2, 5000), (1, 2, 2, 100, 9000)])
def test_forward(B, H, HK, NQ, NK, causal, D):
    q, k, v, _ = A.tensors(B, H, HK, NQ, NK, D, B + NQ + NK)
    check(q, k, v, causal=causal)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("NQ,NK,G", [(1, 700, 4), (200, 333, 2), (400, 400, 1), (5, 3000, 8)])
def test_padded_batch_whatever_lies_in_the_padding(NQ, NK, G, causal, D):
    """Lengths of every kind (whole, none, one, past the extent, negative, inside a tile); NaN and inf past them."""
    ql = lens(NQ, NQ, max(NQ - 3, 1), 0, NQ + 9, NQ // 2 + 1)
    kl = lens(NK, 1, NK - 130, NK, -4, NK // 2)
    q, k, v, _ = A.tensors(6, 2 * G, 2, NQ, NK, D, 3)
    for b in range(6):
        q[b, :, max(min(int(ql[b]), NQ), 0):] = float("nan")
        k[b, :, max(min(int(kl[b]), NK), 0):] = float("nan")
        v[b, :, max(min(int(kl[b]), NK), 0):] = float("inf")
    o, lse = check(q, k, v, causal=causal, q_lens=ql, k_lens=kl)
    assert bool((o[3] == 0).all()) and bool((lse[3] == NEG).all()) and bool((o[4] == 0).all())
    check(q[:, :, :, :].contiguous(), k, v, causal=causal, q_lens=ql, k_lens=kl)


def test_rows_without_keys():
    q, k, v, _ = A.tensors(2, 2, 2, 300, 40, 64)
    o, lse = check(q, k, v, causal=True)  # the first 260 rows see nothing
    assert bool((o[:, :, :260] == 0).all()) and bool((lse[:, :, :260] == NEG).all())
    o, lse = skl.attn_fwd(q, k[:, :, :0], v[:, :, :0])
    assert bool((o == 0).all()) and bool((lse == NEG).all())
    o, lse = skl.attn_fwd(q[:, :, :0], k, v)
    assert o.shape == (2, 2, 0, 64) and lse.shape == (2, 2, 0)


def test_logits_that_outgrow_the_first_tile():
    """Later tiles bring far larger logits (the reference moves, O is rescaled), then far smaller ones; sharp rows."""
    q, k, v, _ = A.tensors(1, 2, 2, 300, 1024, 128, 5, by=4.0)
    k = k.float()
    k[:, :, :128] *= 0.01
    k[:, :, 300:310] *= 30
    k[:, :, 700:703] *= 60
    check(q, k.to(torch.bfloat16), v)
    check(q, k.to(torch.bfloat16), v, causal=True)
    # one row in a warp alone moves
    q2 = q.clone()
    q2[:, :, 1:] *= 0.01
    check(q2, k.to(torch.bfloat16), v)


def test_large_scale_and_equal_logits():
    q, k, v, _ = A.tensors(1, 2, 1, 130, 400, 64, 6)
    check(q, k, v, scale=3.0)
    check(torch.zeros_like(q), k, v, scale=1.0)  # the mean of the values
    check(q, k, v, scale=1e-6, causal=True)


@pytest.mark.parametrize("NQ", [1, 140])
def test_views(NQ):
    """Heads and rows in any storage order, slices of a packed tensor, an odd start; the output keeps q's layout."""
    q, k, v, _ = A.tensors(2, 4, 2, NQ, 260, 64, 7, rows_first=True)
    o, _ = check(q, k, v, causal=True)
    if NQ > 1:
        assert o.stride() == q.stride()
    packed = torch.randn(2, NQ, 8, 64, device="cuda").to(torch.bfloat16)
    qkv = [packed[:, :, a:b].transpose(1, 2) for a, b in ((0, 4), (4, 6), (6, 8))]
    check(*qkv, causal=True)
    odd = torch.randn(2 * 4 * NQ * 64 + 3, device="cuda").to(torch.bfloat16)[3:].view(2, 4, NQ, 64)  # not 16-byte aligned
    check(odd, k, v)
    check(q, k[:, :1].expand(2, 2, 260, 64), v[:, :, ::2].repeat_interleave(2, 2))
    half = torch.randn(2, 4, NQ, 128, device="cuda").to(torch.bfloat16)[..., ::2]  # D not contiguous
    check(half, k, v)


def test_other_streams_graphs_and_repeats_give_the_same_bits():
    q, k, v, _ = A.tensors(1, 8, 2, 2, 20000, 128, 8)  # split keys: a workspace and a merge
    assert skl.attn_fwd_plan(1, 8, 2, 2, 20000, 128, torch.cuda.get_device_properties(0).multi_processor_count)[1] > 1
    want = skl.attn_fwd(q, k, v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = skl.attn_fwd(q, k, v)
    again = skl.attn_fwd(q, k, v)  # both at once, each with its own workspace
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(skl.attn_fwd(q, k, v))
        graphs.append(g)
    for g in graphs * 2:
        g.replay()
    for got in (other, again, *outs):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    k.copy_(torch.randn_like(k, dtype=torch.float32).to(torch.bfloat16))
    graphs[0].replay()
    want = skl.attn_fwd(q, k, v)
    assert torch.equal(outs[0][0], want[0])


def test_lse_is_the_losses():
    """The attention's log-sum-exp of a model's Q and K is the one the attention-KL forward reports for them."""
    q1, k1, v, _ = A.tensors(1, 2, 2, 200, 260, 128, 9)
    q2, k2, _, _ = A.tensors(1, 2, 2, 200, 260, 128, 10)
    _, l1, l2 = skl.fwd(q1, k1, q2, k2, causal=True)
    for q, k, l in ((q1, k1, l1), (q2, k2, l2)):
        _, _, _, bl, _, _ = A.forward(q, k, v, causal=True)
        A.within(skl.attn_fwd(q, k, v, causal=True)[1], l.double(), 2 * bl, "lse")


def test_host_tensors_and_refusals():
    q, k, v, _ = A.tensors(1, 2, 2, 30, 40, 64)
    o, lse = skl.attn_fwd(q, k, v)
    ho, hl = skl.attn_fwd(q.cpu(), k.cpu(), v.cpu())
    assert ho.device.type == "cpu" and torch.equal(ho, o.cpu()) and torch.equal(hl, lse.cpu())
    with pytest.raises(ValueError):
        skl.attn_fwd(q, k, v, q_lens=lens(1, 2))
    with pytest.raises(ValueError):
        skl.attn_fwd(q, k, v, k_lens=lens(1).long())
    with pytest.raises(ValueError):
        skl.attn_fwd(q, k.cpu(), v)
    with pytest.raises(skl.StreamKLError):
        skl.attn_fwd(q[..., :32], k[..., :32], v[..., :32])


def test_offsets_past_32_bits():
    """A cache whose last head starts past 2^31 elements."""
    N = (1 << 31) // (128 * 2) + 4096
    k = torch.empty(1, 3, N, 128, dtype=torch.bfloat16, device="cuda").normal_()
    v = torch.empty(1, 3, N, 128, dtype=torch.bfloat16, device="cuda").normal_()
    q = torch.randn(1, 3, 1, 128, device="cuda").to(torch.bfloat16)
    o, lse = skl.attn_fwd(q, k, v)
    s = (k[0, 2].float() @ q[0, 2, 0].float()).double() / 128 ** 0.5
    p = torch.softmax(s, 0)
    assert abs(float(lse[0, 2, 0]) - float(torch.logsumexp(s, 0))) < 1e-3
    ref = (p[None].float() @ v[0, 2].float())[0].double()
    assert float((o[0, 2, 0].double() - ref).norm() / ref.norm()) < 2 ** -6
