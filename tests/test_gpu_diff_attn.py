"""Differential attention against its formulas in 64 bits.

Bounds, with those of attn_util (h half a step of bf16, W the relative error of a weight) for each map's own result O_t:
    the weights' rounding (h) and W move O_t by at most (h + W) (sum_j P_ij |v_j| + |O_t|), the second term where the forward
    divides by the rounded weights' sum; d = O_1 - lam O_2 is formed in fp32 and rounded once:
        |dd| <= e_1 + |lam| e_2 + 4 u (|O_1| + |lam O_2|) + h |d|
    Backward: attn_util's, for the gradients dO and -lam dO of the two maps, the second rounded by h:
        dP2 is off by h sum_d |dO_d v_jd| and delta2 by the same over O_2 (at most the weighted sum of the former),
        dV by h P2^T |lam dO|;
    dlam = -dO . O_2: sum_d |dO_d| e_2 + (D + 8) u + 2^-16 of sum_d |dO_d O_2d|.
"""
import math

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib as K
from tests import attn_util as A

pytestmark = pytest.mark.gpu
H, U = A.H, A.U
MORE = 1 + 2 ** -6


def inputs(B, Hd, HK, NQ, NK, D, seed=0, rows_first=False, by=1.0):
    q, k, v, do = A.tensors(B, 2 * Hd, HK, NQ, NK, D, seed, rows_first, by)
    gen = torch.Generator(device="cuda").manual_seed(seed + 100)
    lam = torch.rand(B, Hd, NQ, generator=gen, device="cuda") * 1.5 - 0.25
    return q, k, v, lam, do[:, :Hd]


def reference(q, k, v, lam, **kw):
    o, lse, _, b_lse, p, W = A.forward(q, k, v, **kw)
    kl = kw.get("k_lens")
    va = A._clean(v, kl).abs().repeat_interleave(q.shape[1] // k.shape[1], 1)
    e = (H + W[..., None]) * (p @ va + o.abs()) * MORE
    lam = torch.where(lse[:, 0::2] == A.NEG, torch.zeros_like(lam), lam).double()[..., None]
    d = o[:, 0::2] - lam * o[:, 1::2]
    b = e[:, 0::2] + lam.abs() * e[:, 1::2] + 4 * U * (o[:, 0::2].abs() + (lam * o[:, 1::2]).abs()) + H * d.abs() + 2.0 ** -126
    return d, lse, b, b_lse, o, e


def gradients(q, k, v, lam, do, dlse=None, **kw):
    B, H2, NQ, D = q.shape
    HK, NK = k.shape[1:3]
    ql, kl, scale = kw.get("q_lens"), kw.get("k_lens"), kw.get("scale") or 1 / math.sqrt(D)
    do = A._clean(do, ql)
    _, lse, _, _, o, e = reference(q, k, v, lam, **kw)
    lam = torch.where(lse[:, 0::2] == A.NEG, torch.zeros_like(lam), lam).double()[..., None]
    go = torch.stack((do, -lam * do), 2).flatten(1, 2)
    grads, bounds = A.backward(q, k, v, go, dlse, **kw)
    # the second map's rounding
    _, _, _, _, p, _ = A.forward(q, k, v, **kw)
    qa, ka, va = A._clean(q, ql).abs(), A._clean(k, kl).abs(), A._clean(v, kl).abs()
    ka, va = (t.repeat_interleave(H2 // HK, 1) for t in (ka, va))
    second = torch.zeros(1, H2, 1, 1, dtype=torch.float64, device="cuda")
    second[:, 1::2] = H * MORE
    ga = go.abs() * second
    a = ga @ va.transpose(2, 3)
    eds = p * (a + (p * a).sum(-1, keepdim=True))
    groups = lambda t: t.view(B, HK, H2 // HK, NK, D).sum(2)  # noqa: E731
    bounds = (bounds[0] + scale * eds @ ka, bounds[1] + groups(scale * eds.transpose(2, 3) @ qa),
              bounds[2] + groups(p.transpose(2, 3) @ ga))
    dlam = -(do * o[:, 1::2]).sum(-1)
    b = (do.abs() * (e[:, 1::2] + ((D + 8) * U + 2.0 ** -16) * o[:, 1::2].abs())).sum(-1) + 2.0 ** -126
    return (*grads, dlam), (*bounds, b)


def check(B, Hd, HK, NQ, NK, D, seed=0, rows_first=False, by=1.0, modes=(K.BWD_AUTO,), dlse=False, lam=None, **kw):
    q, k, v, l, do = inputs(B, Hd, HK, NQ, NK, D, seed, rows_first, by)
    l = l if lam is None else lam(l)
    wide = l.expand(B, Hd, NQ)
    d, lse = skl.diff_attn_fwd(q, k, v, l, **kw)
    rd, rz, bd, bz, o, e = reference(q, k, v, wide, **kw)
    A.within(d, rd, bd, "d")
    A.within(lse, rz, bz, "lse")
    d2, lse2, maps, rest = skl.diff_attn_fwd(q, k, v, l, return_maps=True, **kw)
    A.within(d2, rd, bd, "d with the maps")
    A.within(lse2, rz, bz, "lse with the maps")
    A.within(maps.double() + rest.double(), o, e + 2.0 ** -16 * o.abs() + 2.0 ** -126, "maps")
    z = None
    if dlse:
        z = torch.randn(B, 2 * Hd, NQ, device="cuda") * 0.1
    ref, bounds = gradients(q, k, v, wide, do, z, **kw)
    for mode in modes:
        got = skl.diff_attn_bwd(q, k, v, l, maps, lse, do, dlse=z, bwd_mode=mode, maps_rest=rest, **kw)
        for g, r, b, what in zip(got, ref, bounds, ("dq", "dk", "dv", "dlam")):
            A.within(g, r, b, f"{what}, mode {mode}")
        assert got[3].dtype == torch.float32 and got[0].stride() == q.stride()
    assert skl.check_device_status() == K.OK


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hd,HK,NQ,NK", [(1, 1, 1, 1, 1), (2, 3, 1, 1, 129), (1, 4, 2, 7, 40), (2, 2, 2, 16, 128), (1, 2, 1, 32, 33),
                                           (1, 3, 3, 33, 100), (3, 2, 1, 64, 64), (1, 1, 1, 65, 65), (2, 2, 1, 127, 300),
                                           (1, 2, 2, 128, 128), (1, 4, 2, 129, 257), (2, 1, 1, 300, 500), (1, 2, 1, 500, 100)])
def test_sizes(B, Hd, HK, NQ, NK, D, causal):
    modes = (K.BWD_SEPARATE, K.BWD_FUSED) if D == 64 else (K.BWD_SEPARATE,)
    check(B, Hd, HK, NQ, NK, D, NQ + NK, causal=causal, modes=modes, dlse=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hd,HK,NQ,NK", [(1, 4, 2, 1, 9000), (2, 4, 1, 3, 5001), (1, 2, 1, 200, 3001), (1, 8, 8, 1, 700)])
def test_split_keys(B, Hd, HK, NQ, NK, D):
    """Few query tiles over many keys: the splits' merge forms the difference."""
    assert skl.diff_attn_plan(B, Hd, HK, NQ, NK, D, 152)[1] > 1
    check(B, Hd, HK, NQ, NK, D, 5)


def test_many_packed_heads_without_splits():
    """So many key heads that packed tiles go without splits: the difference crosses rows of a tile."""
    assert skl.diff_attn_plan(24, 32, 16, 5, 300, 64, 152)[:2] == (True, 1)
    check(24, 32, 16, 5, 300, 64, 6)
    assert skl.diff_attn_plan(24, 16, 16, 3, 200, 128, 152)[:2] == (True, 1)
    check(24, 16, 16, 3, 200, 128, 7, causal=True, rows_first=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_padded_batches(D, causal):
    """Lengths from zero to all; NaN in everything past them, lam among it."""
    B, Hd, HK, NQ, NK = 6, 4, 2, 150, 200
    ql = torch.tensor([150, 0, 1, 77, 128, 150], dtype=torch.int32, device="cuda")
    kl = torch.tensor([200, 200, 0, 33, 129, 100], dtype=torch.int32, device="cuda")
    q, k, v, lam, do = inputs(B, Hd, HK, NQ, NK, D, 8)
    for b in range(B):
        q[b, :, ql[b]:], lam[b, :, ql[b]:], do[b, :, ql[b]:] = float("nan"), float("nan"), float("nan")
        k[b, :, kl[b]:], v[b, :, kl[b]:] = float("nan"), float("nan")
    kw = dict(causal=causal, q_lens=ql, k_lens=kl)
    d, lse, maps, rest = skl.diff_attn_fwd(q, k, v, lam, return_maps=True, **kw)
    plain = skl.diff_attn_fwd(q, k, v, lam, **kw)
    clean = torch.where(lam.isnan(), torch.zeros_like(lam), lam)
    rd, rz, bd, bz, o, e = reference(q, k, v, clean, **kw)
    A.within(d, rd, bd, "d")
    A.within(plain[0], rd, bd, "d alone")
    A.within(lse, rz, bz, "lse")
    A.within(maps.double() + rest.double(), o, e + 2.0 ** -16 * o.abs() + 2.0 ** -126, "maps")
    ref, bounds = gradients(q, k, v, clean, do, **kw)
    for mode in (K.BWD_SEPARATE, K.BWD_FUSED) if D == 64 else (K.BWD_SEPARATE,):
        got = skl.diff_attn_bwd(q, k, v, lam, maps, lse, do, bwd_mode=mode, maps_rest=rest, **kw)
        for g, r, b, what in zip(got, ref, bounds, ("dq", "dk", "dv", "dlam")):
            A.within(g, r, b, f"{what}, mode {mode}")


def test_padded_decode():
    """Single tokens over caches of their own lengths, some empty; packed heads."""
    kl = torch.tensor([4000, 0, 1, 129], dtype=torch.int32, device="cuda")
    q, k, v, lam, _ = inputs(4, 4, 2, 1, 4000, 128, 9)
    for b in range(4):
        k[b, :, kl[b]:], v[b, :, kl[b]:] = float("nan"), float("inf")
    d, lse = skl.diff_attn_fwd(q, k, v, lam, k_lens=kl)
    rd, rz, bd, bz, _, _ = reference(q, k, v, lam, k_lens=kl)
    A.within(d, rd, bd, "d")
    A.within(lse, rz, bz, "lse")
    assert not bool(d[1].any())


@pytest.mark.parametrize("shape", [(), (1,), (4, 1), (2, 1, 1), (1, 1, 100), (2, 4, 100)])
def test_weights_of_any_shape(shape):
    check(2, 4, 2, 100, 140, 64, 10, lam=lambda l: l[tuple(slice(0, n) for n in (1,) * (3 - len(shape)) + shape)].reshape(shape))


def test_special_weights():
    """lam 0 leaves the first map alone, bit for bit with attention's own where that sums the same way; 1 on equal maps leaves 0."""
    q, k, v, lam, _ = inputs(1, 2, 1, 200, 300, 128, 11)
    q[:, 1::2] = q[:, 0::2]
    d, _ = skl.diff_attn_fwd(q, k, v, torch.ones(1, device="cuda"))
    assert float(d.abs().max()) == 0.0
    o, _ = skl.attn_fwd(q[:, 0::2].contiguous(), k, v)
    d, _ = skl.diff_attn_fwd(q, k, v, torch.zeros(1, device="cuda"))
    assert float((d.float() - o.float()).abs().max()) <= 2 * H * float(o.abs().max())
    lam = torch.zeros(1, 2, 200, device="cuda")
    lam[0, 0, 7], lam[0, 1, 9] = float("nan"), float("inf")
    q, k, v, _, _ = inputs(1, 2, 1, 200, 300, 128, 12)
    d, _ = skl.diff_attn_fwd(q, k, v, lam)
    bad = ~d.isfinite()
    assert bool(bad[0, 0, 7].all()) and bool(bad[0, 1, 9].all()) and int(bad.sum()) == 2 * 128


def test_layouts():
    """Rows first, slices of a packed tensor, a scale of its own, host tensors."""
    check(2, 4, 2, 130, 200, 64, 13, rows_first=True, causal=True, scale=0.3)
    B, Hd, HK, N, D = 2, 2, 1, 90, 128
    packed = torch.randn(B, N, 2 * Hd + 2 * HK, D, device="cuda").to(torch.bfloat16)
    q, k, v = packed[:, :, :4].transpose(1, 2), packed[:, :, 4:5].transpose(1, 2), packed[:, :, 5:].transpose(1, 2)
    lam = torch.rand(B, Hd, N, device="cuda")
    d, lse, maps, rest = skl.diff_attn_fwd(q, k, v, lam, return_maps=True)
    qc, kc, vc = (t.contiguous() for t in (q, k, v))
    dc, lsec, mapsc, restc = skl.diff_attn_fwd(qc, kc, vc, lam, return_maps=True)
    assert torch.equal(d, dc) and torch.equal(lse, lsec) and torch.equal(maps, mapsc)
    do = torch.randn(B, N, Hd, D, device="cuda").to(torch.bfloat16).transpose(1, 2)
    a = skl.diff_attn_bwd(q, k, v, lam, maps, lse, do, maps_rest=rest)
    b = skl.diff_attn_bwd(qc, kc, vc, lam, mapsc, lsec, do.contiguous(), maps_rest=restc.transpose(1, 2).contiguous().transpose(1, 2))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    host = skl.diff_attn_fwd(*(t.cpu() for t in (q, k, v, lam)))
    assert torch.equal(host[0], skl.diff_attn_fwd(qc, kc, vc, lam)[0].cpu())


def test_nothing_to_see():
    q, k, v, lam, do = inputs(2, 2, 1, 10, 20, 64, 14)
    d, lse, maps, rest = skl.diff_attn_fwd(q, k[:, :, :0], v[:, :, :0], lam, return_maps=True)
    assert not bool(d.any()) and not bool(maps.any()) and not bool(rest.any()) and bool((lse == A.NEG).all())
    dq, dk, dv, dlam = skl.diff_attn_bwd(q, k[:, :, :0], v[:, :, :0], lam, maps, lse, do, maps_rest=rest)
    assert not bool(dq.any()) and not bool(dlam.any()) and dk.shape == (2, 1, 0, 64)
    d, lse = skl.diff_attn_fwd(q[:, :, :0], k, v, lam[:, :, :0])
    assert d.shape == (2, 2, 0, 64)
    m = torch.empty(2, 4, 0, 64, device="cuda", dtype=torch.bfloat16)
    dq, dk, dv, dlam = skl.diff_attn_bwd(q[:, :, :0], k, v, lam[:, :, :0], m, lse, d, maps_rest=m)
    assert not bool(dk.any()) and not bool(dv.any()) and dlam.shape == (2, 2, 0)


def test_large_logits_and_values():
    """Logits of hundreds and values of 2^60: references move, and nothing overflows."""
    check(1, 2, 1, 140, 300, 64, 15, by=40.0)
    q, k, v, lam, _ = inputs(1, 2, 1, 140, 300, 128, 16)
    d, _ = skl.diff_attn_fwd(q, k, v * 2.0 ** 60, lam)
    rd, _, bd, _, _, _ = reference(q, k, v, lam)
    A.within(d.double() * 2.0 ** -60, rd, bd, "d")


def test_the_same_bits_on_streams_and_in_graphs():
    cases = [inputs(2, 4, 2, 300, 300, 128, 17), inputs(1, 4, 1, 2, 9000, 64, 18)]

    def both(q, k, v, lam, do):
        d, lse, maps, rest = skl.diff_attn_fwd(q, k, v, lam, causal=True, return_maps=True)
        return (d, lse, *skl.diff_attn_bwd(q, k, v, lam, maps, lse, do, causal=True, bwd_mode=K.BWD_SEPARATE, maps_rest=rest))

    refs = [both(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(both(*c))
        torch.cuda.synchronize()
        for a, b in zip(got, refs):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    c = [t.clone() for t in cases[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(*c)
    for seed in (17, 19):
        for x, y in zip(c, inputs(2, 4, 2, 300, 300, 128, seed)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, both(*c)))
    assert skl.check_device_status() == K.OK


def test_autograd_and_differences():
    """Autograd's gradients are the formulas'; dlam against differences, in which d is linear: half of d(lam + e) - d(lam - e)
    over e, each rounded by h."""
    q, k, v, lam, do = inputs(1, 2, 1, 100, 180, 64, 20)
    lam = lam[:, :, :1].contiguous()
    leaves = [t.clone().requires_grad_() for t in (q, k, v, lam)]
    d, lse = skl.differential_attention(*leaves, causal=True, return_lse=True)
    z = torch.randn_like(lse) * 0.1
    torch.autograd.backward((d, lse), (do, z))
    ref, bounds = gradients(q, k, v, lam.expand(1, 2, 100), do, z, causal=True)
    for t, r, b, what in zip(leaves[:3], ref, bounds, ("q", "k", "v")):
        A.within(t.grad, r, b, what)
    n = 100
    total = ref[3].sum(-1, keepdim=True)
    assert leaves[3].grad.shape == lam.shape
    A.within(leaves[3].grad, total, bounds[3].sum(-1, keepdim=True) + n * U * ref[3].abs().sum(-1, keepdim=True), "lam")
    e = 0.5
    up, down = (skl.diff_attn_fwd(q, k, v, lam + s * e, causal=True)[0].double() for s in (1, -1))
    slope = ((up - down) / (2 * e) * do.double()).sum((2, 3))
    rd, _, bd, _, _, _ = reference(q, k, v, (lam + e).expand(1, 2, 100), causal=True)
    slack = 2 * ((bd + H * up.abs() + H * down.abs()) * do.double().abs()).sum((2, 3)) / (2 * e) * 1.5
    assert bool(((slope - total[..., 0]).abs() <= slack).all())
    only = skl.differential_attention(q, k, v, leaves[3].detach().requires_grad_())
    assert only.requires_grad
    with torch.no_grad():
        assert not skl.differential_attention(*leaves).requires_grad


def test_a_long_cache_past_32_bits():
    """Keys whose offsets pass 2^32 bytes."""
    B, Hd, HK, NK, D = 1, 2, 2, 1 << 18, 128
    k = torch.empty(B, NK, 70, D, device="cuda", dtype=torch.bfloat16)[:, :, 66:68].transpose(1, 2)
    v = torch.empty(B, NK, 70, D, device="cuda", dtype=torch.bfloat16)[:, :, 68:].transpose(1, 2)
    k.normal_(), v.normal_()
    q, _, _, lam, _ = inputs(B, Hd, HK, 1, 8, D, 21)
    d, lse = skl.diff_attn_fwd(q, k, v, lam)
    rd, rz, bd, bz, _, _ = reference(q, k, v, lam)
    A.within(d, rd, bd, "d")
    A.within(lse, rz, bz, "lse")
