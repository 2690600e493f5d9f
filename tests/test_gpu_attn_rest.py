"""Attention whose forward leaves what rounding O took, and whose backward reads it: gradients that do not carry O's rounding,
whatever part the values have in common and however sharp a row is.

Bounds, with attn_util's u, h, W.  The forward divides by the sum of its rounded weights, so their errors (h + W each) move O by
their share of v_j - O:  |O' - O| <= c (h + W) sum_j P_ij |v_j - O_i| + W sum_j P_ij |v_j|, where c is 1, and 2 where splits are
merged (each divides by its own sum: |v - O_split| <= |v - O| + |O_split - O|, and the second averages to no more than the
first).  o + o_rest holds O' within h^2 |O|.  So delta is off by
    e_i = c (h + W) sum_j P_ij |dP_ij - dO_i . O_i| + (W + h^2 + (D + 8) u) sum_d |dO_d| sum_j P_ij |v_jd|
instead of attn_util's, which has (2 h + W) before the last sum; the rest of the gradients' bounds is the same.
"""
import ctypes
import math

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib, build
from tests import attn_util as A

pytestmark = pytest.mark.gpu
NEG = float("-inf")
MORE = 1 + 2 ** -6


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    yield
    assert skl.check_device_status() == 0


def splits(q, k):
    n = torch.cuda.get_device_properties(0).multi_processor_count
    return skl.attn_fwd_plan(q.shape[0], q.shape[1], k.shape[1], q.shape[2], k.shape[2], q.shape[3], n)[1]


def make(B, H, HK, NQ, NK, D, common, by, seed=1, rows_first=False):
    q, k, v, do = A.tensors(B, H, HK, NQ, NK, D, seed, rows_first, by)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    way = torch.randn(B, HK, 1, D, generator=gen, device="cuda")
    shift = v.float() + common * way
    v = shift.transpose(1, 2).contiguous().to(v.dtype).transpose(1, 2) if rows_first else shift.to(v.dtype)
    return q, k, v, do


def bounds(q, k, v, do, dlse=None, **kw):
    """(O, bound of o + o_rest), ((dq, dk, dv), their bounds) in 64 bits."""
    B, H, NQ, D = q.shape
    HK, NK = k.shape[1:3]
    G, scale = H // HK, kw.get("scale") or 1 / math.sqrt(D)
    c = 2 if splits(q, k) > 1 else 1
    o, lse, _, _, p, W = A.forward(q, k, v, **kw)
    (dq, dk, dv), (_, _, bv) = A.backward(q, k, v, do, dlse, **kw)
    qd, kd, vd, dod = A._clean(q, kw.get("q_lens")), *(A._clean(t, kw.get("k_lens")) for t in (k, v)), A._clean(do, kw.get("q_lens"))
    kd, vd = (t.repeat_interleave(G, 1) for t in (kd, vd))
    W = W[..., None]
    # sum_j P_ij |v_jd - O_id|, a value column at a time
    away = torch.stack([(p * (vd[..., None, :, d] - o[..., :, None, d]).abs()).sum(-1) for d in range(D)], -1)
    bo = (c * (A.H + W) * away + W * (p @ vd.abs()) + A.H ** 2 * o.abs()) * MORE + 2.0 ** -126
    dp = dod @ vd.transpose(2, 3)
    pull = dp - (dod * o).sum(-1, keepdim=True)
    spread = (dod.abs() * (p @ vd.abs())).sum(-1, keepdim=True)
    extra = 0 if dlse is None else torch.where(lse == NEG, torch.zeros_like(lse), dlse.double())[..., None]
    e = (c * (A.H + W) * (p * pull.abs()).sum(-1, keepdim=True) + (W + A.H ** 2 + (D + 8) * A.U) * spread
         + (D + 8) * A.U * (extra.abs() if dlse is not None else 0))
    ds = p * (pull + extra)
    eds = (A.H + W) * ds.abs() + p * ((D + 4) * A.U * (dod.abs() @ vd.abs().transpose(2, 3)) + e)
    groups = lambda t: t.view(B, HK, G, NK, D).sum(2)  # noqa: E731
    bq = (scale * (eds + (NK + 64) * A.U * ds.abs()) @ kd.abs() + A.H * dq.abs()) * MORE + 2.0 ** -126
    bk = (groups(scale * (eds + (NQ * G + 64) * A.U * ds.abs()).transpose(2, 3) @ qd.abs()) + A.H * dk.abs()) * MORE + 2.0 ** -126
    return (o, bo), ((dq, dk, dv), (bq, bk, bv))


def modes(D):
    return (skl.BWD_SEPARATE, skl.BWD_FUSED) if D == 64 else (skl.BWD_SEPARATE,)


def check(q, k, v, do, dlse=None, **kw):
    o, lse, rest = skl.attn_fwd(q, k, v, return_rest=True, **kw)
    ro, rl, bo, bl, _, _ = A.forward(q, k, v, **kw)
    A.within(o, ro, bo, "o")
    A.within(lse, rl, bl, "lse")
    (ro, bo), (want, bound) = bounds(q, k, v, do, dlse, **kw)
    A.within(o.double() + rest.double(), ro, bo, "o + o_rest")
    for mode in modes(q.shape[3]):
        got = skl.attn_bwd(q, k, v, o, lse, do, dlse, bwd_mode=mode, o_rest=rest, **kw)
        for name, g, w, b in zip(("dq", "dk", "dv"), got, want, bound):
            A.within(g, w, b, name)
    return o, lse, rest


@pytest.mark.parametrize("common,by", [(0.0, 1.5), (10.0, 1.5), (10.0, 6.0)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,H,HK,NQ,NK", [(1, 4, 2, 512, 512), (2, 2, 1, 130, 700), (1, 8, 2, 3, 5000), (1, 8, 1, 16, 1000),
                                          (1, 2, 2, 257, 65), (1, 1, 1, 300, 100), (2, 96, 96, 200, 200),
                                          (3, 8, 2, 5, 90)])
def test_forward_and_backward(B, H, HK, NQ, NK, causal, D, common, by):
    check(*make(B, H, HK, NQ, NK, D, common, by), causal=causal)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("NQ,NK,G", [(1, 700, 4), (400, 400, 1)])
def test_padded_batch_whatever_lies_in_the_padding(NQ, NK, G, causal, D):
    lens = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")  # noqa: E731
    ql, kl = lens(NQ, NQ, max(NQ - 3, 1), 0, NQ // 2 + 1), lens(NK, 1, NK - 130, NK, NK // 2)
    q, k, v, do = make(5, 2 * G, 2, NQ, NK, D, 5.0, 1.5)
    dlse = torch.randn(5, 2 * G, NQ, device="cuda")
    for b in range(5):
        q[b, :, int(ql[b]):] = do[b, :, int(ql[b]):] = float("nan")
        dlse[b, :, int(ql[b]):] = float("nan")
        k[b, :, int(kl[b]):] = float("nan")
        v[b, :, int(kl[b]):] = float("inf")
    kw = dict(causal=causal, q_lens=ql, k_lens=kl)
    o, lse, rest = skl.attn_fwd(q, k, v, return_rest=True, **kw)
    assert bool((rest[lse == NEG] == 0).all()) and bool((o[lse == NEG] == 0).all())
    clean = dlse.nan_to_num(0.0)
    _, (want, bound) = bounds(q, k, v, do, clean, **kw)
    for mode in modes(D):
        got = skl.attn_bwd(q, k, v, o, lse, do, dlse, bwd_mode=mode, o_rest=rest, **kw)
        for name, g, w, b in zip(("dq", "dk", "dv"), got, want, bound):
            A.within(g, w, b, name)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("by", [1.5, 6.0])
def test_autograd_does_not_carry_the_rounding_of_o(by, D):
    """attention's gradients keep the tight bounds where values have a large common part (without the rest dq is off by several
    times the rounding of the result)."""
    q, k, v, do = make(1, 4, 2, 300, 512, D, 10.0, by)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    o, lse = skl.attention(*leaves, causal=True, return_lse=True, bwd_mode=skl.BWD_SEPARATE)
    dlse = torch.randn_like(lse)
    torch.autograd.backward([o, lse], [do, dlse])
    _, (want, bound) = bounds(q, k, v, do, dlse, causal=True)
    for t, w, b, name in zip(leaves, want, bound, ("dq", "dk", "dv")):
        A.within(t.grad, w, b, name)
    ro, rl, rest = skl.attn_fwd(q, k, v, causal=True, return_rest=True)
    for t, g in zip(leaves, skl.attn_bwd(q, k, v, ro, rl, do, dlse, causal=True, bwd_mode=skl.BWD_SEPARATE, o_rest=rest)):
        assert torch.equal(t.grad, g)
    assert torch.equal(o, ro) and torch.equal(lse, rl)


def test_without_gradients_nothing_more_is_computed():
    q, k, v, _ = make(1, 4, 2, 300, 512, 64, 1.0, 1.5)
    want = skl.attn_fwd(q, k, v)[0]
    assert torch.equal(skl.attention(q, k, v), want)
    leaf = q.clone().requires_grad_()
    with torch.no_grad():
        assert torch.equal(skl.attention(leaf, k, v), want)


@pytest.mark.parametrize("NK", [1, 33, 50, 64])
def test_up_to_64_keys_need_no_rest(NK):
    """The backward forms its row sums without o: the same bits with any o, and the exact bounds."""
    q, k, v, do = make(2, 4, 2, 40, NK, 64, 10.0, 1.5)
    o, lse = skl.attn_fwd(q, k, v)
    a = skl.attn_bwd(q, k, v, o, lse, do, bwd_mode=skl.BWD_SEPARATE)
    b = skl.attn_bwd(q, k, v, torch.zeros_like(o), lse, do, bwd_mode=skl.BWD_SEPARATE)
    _, (want, bound) = bounds(q, k, v, do)
    for x, y, w, n, name in zip(a, b, want, bound, ("dq", "dk", "dv")):
        assert torch.equal(x, y)
        A.within(x, w, n, name)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    for x, y in zip(a, torch.autograd.grad(skl.attention(*leaves, bwd_mode=skl.BWD_SEPARATE), leaves, do)):
        assert torch.equal(x, y)


def test_layouts_and_callers(monkeypatch):
    """Rows first, a rest and a gradient in other layouts than o, host tensors, and the step-by-step path: the same bits."""
    q, k, v, do = make(2, 4, 2, 140, 260, 64, 3.0, 1.5, rows_first=True)
    o, lse, rest = check(q, k, v, do, causal=True)
    assert rest.stride() == o.stride() == q.stride()
    call = lambda **kw: skl.attn_bwd(q, k, v, o, lse, do, causal=True, bwd_mode=skl.BWD_SEPARATE, **kw)  # noqa: E731
    want = call(o_rest=rest)
    for a, b in zip(want, call(o_rest=rest.contiguous())):
        assert torch.equal(a, b)
    for a, b in zip(want, skl.attn_bwd(*(t.cpu() for t in (q, k, v, o, lse, do)), causal=True, bwd_mode=skl.BWD_SEPARATE,
                                       o_rest=rest.cpu())):
        assert torch.equal(a.cpu(), b)

    class Nothing:
        def __getattr__(self, name):
            return lambda *a: None

    native = _lib.calls()
    monkeypatch.setattr(_lib, "_calls", Nothing())
    step = skl.attn_fwd(q, k, v, causal=True, return_rest=True)
    grads = call(o_rest=rest)
    monkeypatch.setattr(_lib, "_calls", native)
    assert all(torch.equal(a, b) and a.stride() == b.stride() for a, b in zip(step, (o, lse, rest)))
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    assert len(native.attn_fwd(q, k, v, None, True, None, None, True)) == 3
    o, lse, rest = skl.attn_fwd(q, k[:, :, :0], v[:, :, :0], return_rest=True)
    assert bool((rest == 0).all())
    for bad, error in ((rest.float(), TypeError), (rest[:, :, :2], ValueError)):
        with pytest.raises(error):
            call(o_rest=bad)


def test_streams_and_graphs():
    for args in ((1, 8, 2, 2, 20000, 128), (1, 8, 2, 300, 400, 64)):
        q, k, v, do = make(*args, 3.0, 1.5)
        want = skl.attn_fwd(q, k, v, return_rest=True)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = skl.attn_fwd(q, k, v, return_rest=True)
        again = skl.attn_fwd(q, k, v, return_rest=True)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        with torch.cuda.graph(g):
            got = skl.attn_fwd(q, k, v, return_rest=True)
            grads = skl.attn_bwd(q, k, v, *got[:2], do, bwd_mode=skl.BWD_SEPARATE, o_rest=got[2])
        g.replay()
        g.replay()
        for a, b, c, d in zip(want, other, again, got):
            assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)
        for a, b in zip(grads, torch.autograd.grad(skl.attention(*leaves, bwd_mode=skl.BWD_SEPARATE), leaves, do)):
            assert torch.equal(a, b)


def test_an_unaligned_rest_is_refused():
    q, k, v, do = make(1, 2, 2, 100, 100, 64, 0.0, 1.5)
    s = _lib.make_attn_shape(1, 2, 2, 100, 100, 64)
    s.o_rest = q.data_ptr() + 2
    n = ctypes.c_size_t()
    assert _lib.lib().streamkl_attn_fwd_workspace(s, ctypes.byref(n)) == _lib.ERR_INVALID
    assert _lib.lib().streamkl_attn_bwd_workspace(s, 0, ctypes.byref(n)) == _lib.ERR_INVALID
