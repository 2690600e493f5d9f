"""Cross entropy over a vocabulary against its formulas in 64 bits.

Bounds.  u = 2^-24, h = half a step of the inputs' type, X the largest scale sum_c |h_c| |w_vc| of a row.  A logit is a sum
of C products in fp32: within (C + 16) u X; the exponent 2^(c z - m) adds roundings of |z| and |m| <= X and 2^x's own 4 u:
    F = (C + 16) u (X + |LSE| + 1) + 4 u is the relative error of a term of the sum;
    LSE: 2 F + (V / 2048 + 96) u for the sums + 2 u |LSE|;   loss: that and the given logit's own F, and 4 u |loss|
d = scale (g (p - 1) + g' p):  p within P = 2 F + (LSE's bound) + 8 u, so |dd| <= h |d| + scale (|g| + |g'|) (p P + 4 u) + t, t
the least step of fp16 at the power of two on d: 2^-24 of 2^-13 of the largest scale (|g| + |g'|).
    dh: sum_v |dd| |w| + (V / 8 + 64) u sum_v |d| |w| + h |dh| (and fp16's least step);  dw: the same over the rows.
"""
import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib as K

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def inputs(R, C, V, dtype, seed=0, spread=2.5, none=0.2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn(R, C, generator=gen, device="cuda").to(TYPES[dtype])
    w = (torch.randn(V, C, generator=gen, device="cuda") * (spread / C ** 0.5)).to(TYPES[dtype])
    t = torch.randint(0, V, (R,), generator=gen, device="cuda")
    t[torch.rand(R, generator=gen, device="cuda") < none] = -1
    return h, w, t


def forward(h, w, t, scale):
    """(loss, lse, their bounds, z, F) in 64 bits."""
    C, V = h.shape[1], w.shape[0]
    z = scale * (h.double() @ w.double().T)
    X = (scale * (h.double().abs() @ w.double().abs().T)).amax(-1)
    lse = torch.logsumexp(z, -1)
    F = (C + 16) * U * (X + lse.abs() + 1) + 4 * U
    b_lse = 2 * F + (V / 2048 + 96) * U + 2 * U * lse.abs()
    there = (t >= 0) & (t < V)
    loss = torch.where(there, lse - z.gather(1, t.clamp(0, V - 1)[:, None])[:, 0], torch.zeros_like(lse))
    return loss, lse, b_lse + F + 4 * U * loss.abs(), b_lse, z, F


def backward(h, w, t, g, gl, scale):
    _, lse, _, b_lse, z, F = forward(h, w, t, scale)
    V, R = w.shape[0], h.shape[0]
    H = torch.finfo(h.dtype).eps / 2
    p = (z - lse[:, None]).exp()
    there = (t >= 0) & (t < V)
    gd = torch.where(there, g.double(), torch.zeros_like(lse))
    ld = torch.zeros_like(lse) if gl is None else gl.double()
    d = scale * (gd + ld)[:, None] * p
    d.scatter_add_(1, t.clamp(0, V - 1)[:, None], -scale * gd[:, None])
    size = scale * (gd.abs() + ld.abs())
    least = float((scale * (g.abs() + (0 if gl is None else gl.abs()))).max()) * 2.0 ** -37 if h.dtype == torch.float16 else 0.0
    dd = H * d.abs() + size[:, None] * (p * (2 * F + b_lse + 8 * U)[:, None] + 4 * U) + least
    ha, wa = h.double().abs(), w.double().abs()
    tiny = 2.0 ** -25 if h.dtype == torch.float16 else 2.0 ** -126
    dh, dw = d @ w.double(), d.T @ h.double()
    more = 1 + 2 ** -6
    bh = (dd @ wa + (V / 8 + 64) * U * (d.abs() @ wa) + H * dh.abs()) * more + tiny
    bw = (dd.T @ ha + (R / 8 + 64) * U * (d.abs().T @ ha) + H * dw.abs()) * more + tiny
    return dh, dw, bh, bw


def within(got, ref, bound, what):
    over = (got.double() - ref).abs() / bound
    assert bool((over <= 1).all()), f"{what}: {float(over.nan_to_num(1e9).max()):.2f} of its bound"


def check(h, w, t, scale=1.0, gl=False, seed=1):
    loss, lse = skl.vocab_xent_fwd(h, w, t, scale)
    rl, rz, bl, bz, _, _ = forward(h, w, t, scale)
    within(lse, rz, bz, "lse")
    within(loss, rl, bl, "loss")
    assert bool((loss[t < 0] == 0).all())
    gen = torch.Generator(device="cuda").manual_seed(seed)
    R = h.shape[0]
    g = torch.randn(R, generator=gen, device="cuda") / R
    gl = torch.randn(R, generator=gen, device="cuda") / R if gl else None
    dh, dw = skl.vocab_xent_bwd(h, w, t, lse, g, gl, scale)
    assert dh.dtype == h.dtype and dw.dtype == w.dtype
    rh, rw, bh, bw = backward(h, w, t, g, gl, scale)
    within(dh, rh, bh, "dhidden")
    within(dw, rw, bw, "dweight")
    assert skl.check_device_status() == K.OK
    return g, gl, lse, dh, dw


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R,C,V", [(1, 8, 1), (1, 8, 2), (2, 64, 33), (3, 72, 256), (31, 64, 257), (32, 200, 255), (33, 56, 64),
                                   (127, 128, 128), (128, 64, 129), (129, 264, 300), (255, 64, 512), (256, 256, 256),
                                   (257, 320, 513), (300, 1000, 1000), (513, 264, 2049)])
def test_small_and_ragged_sizes(R, C, V, dtype):
    check(*inputs(R, C, V, dtype, R + C + V), gl=True)


@pytest.mark.parametrize("R,C,V,dtype,scale", [(5, 64, 40001, "bf16", 0.5), (8, 520, 131072, "bf16", 1.0), (333, 1000, 50021, "fp16", 0.5),
                                               (1111, 2048, 9001, "bf16", 1.25), (2049, 128, 32000, "fp16", 1.0)])
def test_large_vocabularies(R, C, V, dtype, scale):
    check(*inputs(R, C, V, dtype, V), scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R,C,V", [(100, 512, 20000), (100, 1024, 28001), (300, 520, 12007), (64, 2000, 33000), (257, 1024, 12000)])
def test_narrower_tiles(R, C, V, dtype):
    """Vocabularies whose tiles of 256 columns would begin another wave; the last columns of a tile are 32 or 64."""
    check(*inputs(R, C, V, dtype, R + V), gl=True)


def test_every_width_of_a_tile_is_met():
    assert {skl.vocab_xent_fwd_plan(R, V, C, 152)[0] for R, C, V in
            [(300, 520, 12007), (100, 1024, 28001), (64, 2000, 33000), (8, 64, 300)]} == {160, 192, 224, 256}


def test_a_forward_workspace_a_byte_short():
    h, w, t = inputs(70, 64, 500, "bf16", 21)
    _, n = skl.vocab_xent_fwd_plan(70, 500, 64, torch.cuda.get_device_properties(0).multi_processor_count)
    out, ws = torch.empty(2, 70, device="cuda"), torch.empty(n, dtype=torch.uint8, device="cuda")
    args = (h.data_ptr(), w.data_ptr(), t.data_ptr(), K.make_xent_shape(70, 500, 64), out[0].data_ptr(), out[1].data_ptr(), ws.data_ptr())
    assert skl.lib().streamkl_vocab_xent_fwd(*args, n - 1, None) == K.ERR_WORKSPACE
    assert skl.lib().streamkl_vocab_xent_fwd(*args, n, None) == K.OK
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R,pieces", [(17000, 2), (33000, 3)])
def test_pieces_of_the_vocabulary(R, pieces, dtype):
    """So many rows that d is written in several pieces; the last is no whole tile."""
    C, V = 72, 17001
    assert skl.vocab_xent_plan(R, V, C, 152)[0] == pieces
    check(*inputs(R, C, V, dtype, 3))


def test_split_sums_with_a_short_last_piece():
    """Few tiles of dhidden over several pieces, each split over blocks."""
    R, C, V = 8200, 64, 2 * 40960 + 8
    pieces, splits, _ = skl.vocab_xent_plan(R, V, C, 152)
    assert pieces > 1 and splits > 1
    check(*inputs(R, C, V, "bf16", 4))


def test_tokens_that_are_none():
    h, w, t = inputs(70, 64, 300, "bf16", 5)
    t[:] = -1
    t[3], t[5] = -9223372036854775808, 299
    check(h, w, t, gl=True)
    loss, lse = skl.vocab_xent_fwd(h, w, t.clamp(min=-1))
    t[5] = -1
    dh, dw = skl.vocab_xent_bwd(h, w, t, lse, torch.ones(70, device="cuda"))
    assert not bool(dh.any()) and not bool(dw.any())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_column_may_be_the_given_one(dtype):
    """Each column of the vocabulary is some row's token, at every place of a tile, whole and narrower ones."""
    V = 771
    h, w, _ = inputs(V, 64, V, dtype, 21)
    check(h, w, torch.arange(V, device="cuda"), gl=True)
    check(h, w, torch.arange(V, device="cuda").flip(0))
    R, C, V = 100, 1024, 20000
    assert skl.vocab_xent_fwd_plan(R, V, C, 152)[0] < 256
    h, w, _ = inputs(R, C, V, dtype, 22)
    for first in (0, 100, 200, 300, 19900):
        check(h, w, torch.arange(first, first + R, device="cuda"))


def test_tokens_past_the_vocabulary():
    h, w, t = inputs(70, 64, 300, "bf16", 6, none=0.0)
    t[7], t[9] = 300, 2 ** 40
    loss, lse = skl.vocab_xent_fwd(h, w, t)
    bad = torch.zeros(70, dtype=torch.bool, device="cuda")
    bad[7] = bad[9] = True
    assert torch.equal(loss.isnan(), bad) and not bool(lse.isnan().any())
    g = torch.rand(70, device="cuda")
    got = skl.vocab_xent_bwd(h, w, t, lse, g)
    t[7] = t[9] = -1
    assert all(torch.equal(a, b) for a, b in zip(got, skl.vocab_xent_bwd(h, w, t, lse, g)))


def test_rows_that_are_not_finite():
    """NaN and infinities stay in their own rows; a hidden state of one channel masks columns of the vocabulary."""
    h, w, t = inputs(40, 64, 500, "bf16", 7, none=0.0)
    ref = skl.vocab_xent_fwd(h, w, t)
    h2 = h.clone()
    h2[3, 5], h2[8, 0] = float("nan"), float("inf")
    got = skl.vocab_xent_fwd(h2, w, t)
    for a, b in zip(got, ref):
        assert bool(a[[3, 8]].isnan().all())
        keep = [i for i in range(40) if i not in (3, 8)]
        assert torch.equal(a[keep], b[keep])
    # -inf logits: probability 0
    h[:, 0] = 1.0
    w[:, 0] = 0.0
    w[400:, 0] = float("-inf")
    t.clamp_(max=399)
    a, b = skl.vocab_xent_fwd(h, w, t), skl.vocab_xent_fwd(h, w[:400], t)
    assert bool(((a[1] - b[1]).abs() <= 2e-6 * (1 + b[1].abs())).all()) and bool(((a[0] - b[0]).abs() <= 4e-6 * (1 + b[1].abs())).all())
    w[:, 0] = float("-inf")
    loss, lse = skl.vocab_xent_fwd(h, w, t)
    assert bool((lse == float("-inf")).all())
    # the type's lowest value: finite, and no gradient past the rest
    w[:, 0] = 0.0
    w[400:, 0] = torch.finfo(torch.bfloat16).min
    check(h, w, t)


@pytest.mark.parametrize("R", [1, 40, 300])
@pytest.mark.parametrize("seen,V", [(200, 1024), (256, 700), (1, 20000)])
def test_whole_tiles_of_the_lowest_value(seen, V, R):
    """Columns behind `seen` are masked by a channel with the type's lowest value: some 128 columns hold nothing else."""
    h, w, t = inputs(R, 64, V, "bf16", 11, none=0.0)
    h[:, 0], w[:, 0] = 1.0, 0.0
    w[seen:, 0] = torch.finfo(torch.bfloat16).min
    t %= seen
    ref, got = skl.vocab_xent_fwd(h, w[:seen], t), skl.vocab_xent_fwd(h, w, t)
    F = forward(h, w[:seen], t, 1.0)
    within(got[0], F[0], F[2], "loss")
    within(got[1], F[1], F[3], "lse")
    g = torch.rand(R, device="cuda")
    (dh, dw), (rh, rw) = skl.vocab_xent_bwd(h, w, t, ref[1], g), skl.vocab_xent_bwd(h, w[:seen], t, ref[1], g)
    assert bool((dh[:, 1:].isfinite()).all()) and not bool(dw[seen:].any())
    _, _, bh, bw = backward(h, w[:seen], t, g, None, 1.0)
    within(dh, rh.double(), 2 * bh, "dhidden")
    within(dw[:seen], rw.double(), 2 * bw, "dweight")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R,V", [(40, 500), (300, 3000), (17000, 17000)])
def test_rows_without_a_gradient_may_hold_anything(R, V, dtype):
    """NaN and infinities in the hidden states of rows that have no token and no upstream gradient: nothing of them is seen."""
    h, w, t = inputs(R, 72, V, dtype, 18, none=0.3)
    gen = torch.Generator(device="cuda").manual_seed(19)
    g = torch.rand(R, generator=gen, device="cuda") / R
    g[5] = 0.0
    t[5], t[0] = 3, 1
    _, lse = skl.vocab_xent_fwd(h, w, t)
    off = (t < 0) | (g == 0)
    for what in (float("nan"), float("inf"), -float("inf")):
        bad = h.clone()
        bad[off, 7] = what
        bad[-1, 3] = h[-1, 3] if not bool(off[-1]) else what
        loss, z = skl.vocab_xent_fwd(bad, w, t)
        assert bool((loss[t < 0] == 0).all())
        got = skl.vocab_xent_bwd(bad, w, t, z, g)
        clean = torch.where(off[:, None], torch.zeros_like(h), h)
        rh, rw, bh, bw = backward(clean, w, torch.where(off, -1, t), g, None, 1.0)
        within(got[0], rh, bh, f"dhidden, {what}")
        within(got[1], rw, bw, f"dweight, {what}")
        assert not bool(got[0][off].any())
        strided = torch.full((R, 80), float("nan"), device="cuda", dtype=h.dtype)
        strided[:, :72] = bad
        assert all(torch.equal(a, b) for a, b in zip(got, skl.vocab_xent_bwd(strided[:, :72], w, t, z, g)))
    ref = skl.vocab_xent_bwd(h, w, t, lse, g)
    within(ref[1], rw, bw, "dweight, finite")


def test_logits_far_from_zero_keep_the_loss():
    """A vector that all rows of the weight share moves every logit by thousands, and the loss by nothing."""
    h, w, t = inputs(64, 64, 1000, "bf16", 8, none=0.0)
    h[:, 0], w[:, 0] = 64.0, 64.0
    check(h, w, t)


def test_strides_shapes_and_types_of_tokens():
    h, w, t = inputs(60, 64, 300, "bf16", 9)
    ref = skl.vocab_xent_fwd(h, w, t)
    g = torch.rand(60, device="cuda")
    gref = skl.vocab_xent_bwd(h, w, t, ref[1], g)
    wide = torch.full((60, 200), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide[:, 8:72] = h
    tall = torch.full((400, 72), float("nan"), device="cuda", dtype=torch.bfloat16)
    tall[:300, :64] = w
    odd = torch.empty(60 * 64 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(60, 64).copy_(h)
    for hh in (wide[:, 8:72], odd, h.t().contiguous().t()):
        for ww in (tall[:300, :64], w.t().contiguous().t()):
            got = skl.vocab_xent_fwd(hh, ww, t.int())
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
            assert all(torch.equal(a, b) for a, b in zip(skl.vocab_xent_bwd(hh, ww, t, ref[1], g), gref))
    loss, lse = skl.vocab_xent_fwd(h.view(3, 20, 64), w, t.view(3, 20))
    assert loss.shape == (3, 20) and torch.equal(loss.view(-1), ref[0])
    dh, dw = skl.vocab_xent_bwd(h.view(3, 20, 64), w, t.view(3, 20), lse, g.view(3, 20))
    assert dh.shape == (3, 20, 64) and torch.equal(dh.view(60, 64), gref[0])
    one = skl.vocab_xent_fwd(h[0], w, t[0])
    assert one[0].shape == () and torch.equal(one[1], ref[1][0])
    host = skl.vocab_xent_fwd(h.cpu(), w.cpu(), t.cpu())
    assert torch.equal(host[0], ref[0].cpu())
    none = skl.vocab_xent_bwd(h[:0], w, t[:0], lse.view(-1)[:0], g[:0])
    assert none[0].shape == (0, 64) and not bool(none[1].any())


def test_gradients_that_cancel():
    """g' = -g: the probabilities have no gradient, the given token has."""
    h, w, t = inputs(50, 64, 300, "bf16", 20, none=0.0)
    _, lse = skl.vocab_xent_fwd(h, w, t)
    g = torch.rand(50, device="cuda")
    dh, dw = skl.vocab_xent_bwd(h, w, t, lse, g, -g)
    rh, rw, bh, bw = backward(h, w, t, g, -g, 1.0)
    within(dh, rh, bh, "dhidden")
    within(dw, rw, bw, "dweight")


def test_one_gradient_alone():
    h, w, t = inputs(400, 264, 900, "fp16", 10)
    _, lse = skl.vocab_xent_fwd(h, w, t)
    g = torch.rand(400, device="cuda")
    dh, dw = skl.vocab_xent_bwd(h, w, t, lse, g)
    a, none = skl.vocab_xent_bwd(h, w, t, lse, g, want_dweight=False)
    assert none is None and torch.equal(a, dh)
    none, b = skl.vocab_xent_bwd(h, w, t, lse, g, want_dhidden=False)
    assert none is None and torch.equal(b, dw)


@pytest.mark.parametrize("size", [1e-6, 1.0, 1e6])
def test_fp16_gradients_of_any_size(size):
    """The power of two on d: upstream gradients far below and above fp16's range for p's small values."""
    h, w, t = inputs(200, 128, 3000, "fp16", 11)
    w = (w.float() * 2 ** -6).to(torch.float16)  # keeps large gradients within fp16
    _, lse = skl.vocab_xent_fwd(h, w, t)
    g = torch.rand(200, device="cuda") * size / 200
    dh, dw = skl.vocab_xent_bwd(h, w, t, lse, g)
    rh, rw, bh, bw = backward(h, w, t, g, None, 1.0)
    fits = rw.abs() < 6e4
    within(dh, rh, bh, "dhidden")
    within(dw[fits], rw[fits], bw[fits], "dweight")


def test_the_same_bits_on_streams_and_in_graphs():
    """Two streams side by side, and a graph that is replayed on new inputs in place."""
    cases = [inputs(500, 264, 5000, "bf16", 12), inputs(300, 128, 20000, "fp16", 13)]
    gs = [torch.rand(c[0].shape[0], device="cuda") for c in cases]

    def both(c, g):
        loss, lse = skl.vocab_xent_fwd(*c)
        return (loss, lse, *skl.vocab_xent_bwd(*c, lse, g))

    refs = [both(c, g) for c, g in zip(cases, gs)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for c, g, s in zip(cases, gs, streams):
            with torch.cuda.stream(s):
                got.append(both(c, g))
        torch.cuda.synchronize()
        for a, b in zip(got, refs):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    c, g = [x.clone() for x in cases[0]], gs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(c, g)
    for seed in (12, 14):
        for x, y in zip(c, inputs(500, 264, 5000, "bf16", seed)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, both(c, g)))
    assert skl.check_device_status() == K.OK


def test_offsets_past_32_bits():
    """A weight of more than 2^31 values and a piece of d past 2^31 bytes."""
    R, C, V = 12, 16384, 140000
    gen = torch.Generator(device="cuda").manual_seed(15)
    h = torch.randn(R, C, generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.empty(V, C, device="cuda", dtype=torch.bfloat16)
    for v in range(0, V, 10000):
        w[v:v + 10000] = (torch.randn(10000, C, generator=gen, device="cuda") / 64).to(torch.bfloat16)
    t = torch.randint(0, V, (R,), generator=gen, device="cuda")
    t[0], t[1], t[2] = V - 1, 131072, -1
    check_rows = torch.cat([torch.arange(0, 300), torch.arange(131000, 131300), torch.arange(V - 300, V)]).cuda()
    loss, lse = skl.vocab_xent_fwd(h, w, t)
    z = torch.cat([h.double() @ w[v:v + 10000].double().T for v in range(0, V, 10000)], 1)
    rz = torch.logsumexp(z, -1)
    X = float(h.abs().double().sum(-1).max()) * float(w[:10000].abs().max())
    bound = 3 * (C + 16) * U * (X + 20)
    assert float((lse - rz).abs().max()) <= bound
    g = torch.rand(R, device="cuda")
    _, dw = skl.vocab_xent_bwd(h, w, t, lse, g, want_dhidden=False)
    d = torch.where(t >= 0, g, torch.zeros_like(g)).double()[:, None] * (z - rz[:, None]).exp()
    d[torch.arange(R), t.clamp(min=0)] -= torch.where(t >= 0, g, torch.zeros_like(g)).double()
    ref = d[:, check_rows].T @ h.double()
    size = d[:, check_rows].abs().T @ h.double().abs()
    assert bool(((dw[check_rows].double() - ref).abs() <= (2.0 ** -8 + 4 * bound) * size + 2.0 ** -8 * ref.abs() + 1e-30).all())


def test_rows_of_d_past_32_bits():
    """d of one piece has more than 2^31 values."""
    R, C, V = 270000, 64, 8192
    h, w, t = inputs(R, C, V, "bf16", 16)
    loss, lse = skl.vocab_xent_fwd(h, w, t)
    g = torch.rand(R, device="cuda") / R
    dh, dw = skl.vocab_xent_bwd(h, w, t, lse, g)
    for rows in (slice(0, 300), slice(R - 300, R)):
        rl, rz, bl, bz, _, _ = forward(h[rows], w, t[rows], 1.0)
        within(lse[rows], rz, bz, "lse")
        within(loss[rows], rl, bl, "loss")
        rh, _, bh, _ = backward(h[rows], w, t[rows], g[rows], None, 1.0)
        within(dh[rows], rh, bh, "dhidden")


def test_autograd_and_differences():
    """The gradients against the loss's own central differences: a step e along a direction d of hidden states moves a row's
    logits by e x_v, x = scale w d, and the third derivative of log-sum-exp is at most (max x - min x)^3 / (6 sqrt 3)."""
    gen = torch.Generator(device="cuda").manual_seed(17)
    R, C, V = 32, 64, 400
    h = (torch.randint(-8, 9, (R, C), generator=gen, device="cuda") / 8).to(torch.bfloat16)
    w = (torch.randn(V, C, generator=gen, device="cuda") / 8).to(torch.bfloat16)
    t = torch.randint(0, V, (R,), generator=gen, device="cuda")
    t[4] = -1
    d = torch.randint(-1, 2, (R, C), generator=gen, device="cuda").to(torch.bfloat16)
    e = 1 / 64  # h +- e d is exact
    a, b = h.clone().requires_grad_(), w.clone().requires_grad_()
    loss, lse = skl.vocab_cross_entropy(a, b, t, return_lse=True)
    (loss.sum() + 0.5 * lse.sum()).backward()

    def value(x):
        loss, lse = skl.vocab_cross_entropy(x, w, t, return_lse=True)
        return loss.double() + 0.5 * lse.double()

    rows = (value(h + e * d) - value(h - e * d)) / (2 * e)
    x = d.double() @ w.double().T
    curved = 1.5 * (x.amax(-1) - x.amin(-1)) ** 3 / (6 * 3 ** 0.5) * e * e / 6
    _, _, bl, bz, _, _ = forward(h, w, t, 1.0)
    rh, rw, bh, bw = backward(h, w, t, torch.ones(R, device="cuda"), torch.full((R,), 0.5, device="cuda"), 1.0)
    slack = curved + (bl + bz) * 1.5 / e + (bh * d.double().abs()).sum(-1)
    assert bool(((rows - (a.grad.double() * d.double()).sum(-1)).abs() <= slack).all())
    within(a.grad, rh, bh, "hidden")
    within(b.grad, rw, bw, "weight")
    frozen = w.clone()
    a.grad = None
    skl.vocab_cross_entropy(a, frozen, t).sum().backward()
    assert a.grad is not None and frozen.grad is None
    only = skl.vocab_cross_entropy(a, b, t, return_lse=True)[1]
    b.grad = None
    only.sum().backward()
    within(b.grad, *backward(h, w, torch.full_like(t, -1), torch.ones(R, device="cuda"), torch.ones(R, device="cuda"), 1.0)[1::2], "lse alone")
