"""Rotary positions against complex numbers in 64 bits.

Bounds.  u = 2^-24.  The angle in the kernel is off by 2^-28 turns' rounding (within pi / 4 rounded to 24 bits: 2^-25) and
the constant's rounding (2^-25), sin and cos by that, the series' rest (2^-28) and their few roundings: within 6 u of a
value in [-1, 1]; times the amplitude (u), the products and their sum (2 u): |error| <= 10 u A (|x| + |y|), and half a
step of the type for the result.  (p turns' own error, |p| 2^-65 turns, is below 2^-40 here.)  The reference's angles are
those of the frequencies in 64 bits: |p| f 2^-52, added for positions far out.
"""
import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib as K

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def tensors(B, HQ, HK, N, D, dtype, seed=0, rows_first=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def one(h):
        if rows_first:
            return torch.randn(B, N, h, D, generator=gen, device="cuda").to(TYPES[dtype]).transpose(1, 2)
        return torch.randn(B, h, N, D, generator=gen, device="cuda").to(TYPES[dtype])

    return one(HQ) if HQ else None, one(HK) if HK else None


def reference(x, plan, positions, interleaved, inverse=False):
    """(the turned tensor, its bound) in 64 bits."""
    B, H, N, D = x.shape
    dim, half = plan.dim, plan.dim // 2
    positions = positions.expand(B, N).double()
    f = torch.tensor(plan.frequencies, dtype=torch.float64, device="cuda")
    angle = (positions[:, None, :, None] * f) * (-1 if inverse else 1)
    z = x.double()
    a, b = (z[..., 0:dim:2], z[..., 1:dim:2]) if interleaved else (z[..., :half], z[..., half:dim])
    turned = torch.complex(a, b) * torch.polar(torch.full_like(angle, plan.amplitude), angle)
    out, size = z.clone(), torch.zeros_like(z)
    mag = plan.amplitude * (a.abs() + b.abs())
    mag = mag * (10 * U + positions.abs()[:, None, :, None] * f * 2.0 ** -52)
    if interleaved:
        out[..., 0:dim:2], out[..., 1:dim:2], size[..., 0:dim:2], size[..., 1:dim:2] = turned.real, turned.imag, mag, mag
    else:
        out[..., :half], out[..., half:dim], size[..., :half], size[..., half:dim] = turned.real, turned.imag, mag, mag
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 2.0 ** -149
    step = torch.zeros_like(z)
    step[..., :dim] = torch.finfo(x.dtype).eps / 2 * (out.abs() + size)[..., :dim] + tiny
    return out, size + step


def within(got, x, plan, positions, interleaved, inverse=False, what=""):
    ref, bound = reference(x, plan, positions, interleaved, inverse)
    assert got.dtype == x.dtype and got.shape == x.shape
    over = (got.double() - ref).abs() - bound
    assert bool((over <= 0).all()), f"{what}: {float(over.max())} over"
    assert torch.equal(got[..., plan.dim:], x[..., plan.dim:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,HQ,HK,N,D,dim", [(1, 1, 1, 1, 2, 2), (2, 3, 1, 5, 64, 64), (1, 8, 2, 17, 128, 128), (3, 5, 5, 33, 80, 20),
                                             (1, 2, 0, 100, 64, 32), (2, 0, 3, 9, 96, 48), (1, 40, 1, 3, 256, 256), (64, 2, 1, 1, 64, 6),
                                             (1, 33, 7, 129, 66, 64), (1, 4, 4, 1000, 128, 96)])
def test_sizes_and_types(B, HQ, HK, N, D, dim, dtype, interleaved):
    plan = skl.rotary_plan(dim)
    q, k = tensors(B, HQ, HK, N, D, dtype, N + D)
    got = skl.rotary_fwd(q, k, plan, offset=37, interleaved=interleaved)
    back = skl.rotary_bwd(*got, plan, offset=37, interleaved=interleaved)
    at = 37 + torch.arange(N, device="cuda")
    for x, y, z in zip((q, k), got, back):
        assert (x is None) == (y is None) == (z is None)
        if x is not None:
            within(y, x, plan, at, interleaved, False, "forward")
            within(z, y, plan, at, interleaved, True, "inverse")


@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("positions", 4.0), ("base", 8.0), ("parts", 32.0)])
@pytest.mark.parametrize("wide", [True, False])
def test_positions_near_and_far(scaling, factor, wide):
    """Positions of each sequence's own: backwards, repeated, negative, millions and (64-bit) beyond 2^32."""
    plan = skl.rotary_plan(128, scaling=scaling, factor=factor, trained_length=4096)
    q, k = tensors(3, 2, 2, 40, 128, "fp32", 1)
    at = torch.randint(0, 1 << 20, (3, 40), device="cuda")
    at[0] = torch.arange(40, device="cuda").flip(0)
    at[1, :10] = 7
    at[1, 10:20] *= -1
    at[2, :5] = (1 << 31) - 1
    if wide:
        at[2, 5:10] = (1 << 33) + 5
    given = at if wide else at.int()
    got = skl.rotary_fwd(q, k, plan, given)
    back = skl.rotary_bwd(*got, plan, given)
    for x, y, z in zip((q, k), got, back):
        within(y, x, plan, at, False)
        within(z, y, plan, at, False, True)
    same = skl.rotary_fwd(q, k, plan, given[0])
    within(same[0], q, plan, at[0], False)
    strided = torch.stack((at, at + 1), -1)[..., 0]
    assert torch.equal(skl.rotary_fwd(q, k, plan, strided)[1], skl.rotary_fwd(q, k, plan, at)[1])
    assert torch.equal(skl.rotary_fwd(q, k, plan, at[:1].expand(3, 40))[0], same[0])


def test_positions_at_the_ends_of_64_bits():
    """p f mod a turn for |p| near 2^63, from the plan's own fractions in whole numbers."""
    plan = skl.rotary_plan(64)
    x = torch.zeros(1, 1, 4, 64, device="cuda")
    x[..., :32] = 1.0
    at = [2 ** 63 - 1, -(2 ** 63), 2 ** 62 + 12345, -1]
    y, _ = skl.rotary_fwd(x, None, plan, torch.tensor(at, device="cuda"))
    turns = [[(p * t % 2 ** 64) / 2 ** 64 for t in plan.turns.tolist()] for p in at]
    angle = torch.tensor(turns, dtype=torch.float64, device="cuda") * 2 * torch.pi
    assert float((y[0, 0, :, :32].double() - angle.cos()).abs().max()) <= 10 * U
    assert float((y[0, 0, :, 32:].double() - angle.sin()).abs().max()) <= 10 * U


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_layouts_and_outputs(dtype):
    """Rows first, slices of packed tensors, odd strides and starts, in place, into a cache's rows."""
    B, HQ, HK, N, D = 2, 6, 2, 24, 64
    plan = skl.rotary_plan(48)
    q, k = tensors(B, HQ, HK, N, D, dtype, 2)
    ref = skl.rotary_fwd(q, k, plan, offset=5)
    qr, kr = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k))
    got = skl.rotary_fwd(qr, kr, plan, offset=5)
    assert got[0].stride() == qr.stride() and all(torch.equal(a, b) for a, b in zip(got, ref))
    packed = torch.randn(B, N, HQ + 2 * HK, D, device="cuda").to(TYPES[dtype])
    packed[:, :, :HQ], packed[:, :, HQ:HQ + HK] = q.transpose(1, 2), k.transpose(1, 2)
    pq, pk = packed[:, :, :HQ].transpose(1, 2), packed[:, :, HQ:HQ + HK].transpose(1, 2)
    assert all(torch.equal(a, b) for a, b in zip(skl.rotary_fwd(pq, pk, plan, offset=5), ref))
    values = packed[:, :, HQ + HK:].clone()
    out = skl.rotary_fwd(pq, pk, plan, offset=5, out=(pq, pk))  # in place in the packed tensor
    assert out[0].data_ptr() == packed.data_ptr() and all(torch.equal(a, b) for a, b in zip(out, ref))
    assert torch.equal(packed[:, :, HQ + HK:], values)
    cache = torch.full((B, HK, 100, D), 7.0, device="cuda").to(TYPES[dtype])
    rows = cache[:, :, 30:30 + N]
    got = skl.rotary_fwd(q, k, plan, offset=5, out=(None, rows))
    assert torch.equal(rows, ref[1]) and torch.equal(got[0], ref[0])
    assert bool((cache[:, :, :30] == 7).all()) and bool((cache[:, :, 30 + N:] == 7).all())
    odd = torch.empty(B, HQ, N, D + 3, device="cuda").to(TYPES[dtype])[..., 1:D + 1].copy_(q)
    assert torch.equal(skl.rotary_fwd(odd, None, plan, offset=5)[0], ref[0])
    assert torch.equal(skl.rotary_fwd(odd, None, plan, offset=5, interleaved=True)[0], skl.rotary_fwd(q, None, plan, offset=5, interleaved=True)[0])
    turned = q.transpose(2, 3).contiguous().transpose(2, 3)
    assert torch.equal(skl.rotary_fwd(turned, k, plan, offset=5)[0], ref[0])
    wide = k[:, :1].expand(B, HQ, N, D)
    assert torch.equal(skl.rotary_fwd(wide, None, plan, offset=5)[0][:, 3], ref[1][:, 0])
    host = skl.rotary_fwd(q.cpu(), k.cpu(), plan, offset=5)
    assert all(torch.equal(a, b.cpu()) for a, b in zip(host, ref))
    assert skl.rotary_fwd(q[:, :, :0], k[:, :, :0], plan)[0].shape == (B, HQ, 0, D)


def test_refusals_on_the_device():
    q, k = tensors(1, 2, 2, 8, 64, "bf16", 3)
    plan = skl.rotary_plan(64)
    with pytest.raises(ValueError):
        skl.rotary_fwd(q, k, skl.rotary_plan(64, device="cpu"))
    with pytest.raises(ValueError):
        skl.rotary_fwd(q, k, plan, torch.arange(8, device="cuda"), offset=3)
    with pytest.raises(ValueError):
        skl.rotary_fwd(q, k, plan, torch.arange(7, device="cuda"))
    with pytest.raises(TypeError):
        skl.rotary_fwd(q, k, plan, torch.arange(8, device="cuda").float())
    with pytest.raises(ValueError):
        skl.rotary_fwd(q, k, plan, out=(q[:, :1], None))
    with pytest.raises(skl.StreamKLError):
        skl.rotary_fwd(q, k, plan, out=(torch.empty_like(q[:, :1]).expand_as(q), None))
    with pytest.raises(skl.StreamKLError):  # in place with other strides
        x = torch.empty(1, 8, 8, 64, device="cuda", dtype=torch.bfloat16)
        skl.rotary_fwd(x, None, plan, out=(x.transpose(1, 2), None))


def test_outputs_and_gradients():
    """An output that requires a gradient is refused; a backward that needs what stood in one says so."""
    q, k = tensors(1, 2, 2, 8, 64, "fp32", 5)
    plan = skl.rotary_plan(64)
    leaf = q.clone().requires_grad_()
    with pytest.raises(ValueError):
        skl.rotary_fwd(leaf, k, plan, out=(leaf, k))
    with torch.no_grad():
        skl.rotary_fwd(leaf, k, plan, out=(leaf, None))
    y = (leaf * k).sum()
    skl.rotary_fwd(q, k, plan, out=(None, k))
    with pytest.raises(RuntimeError):
        y.backward()
    ref = skl.rotary_fwd(q, k, plan)
    with torch.inference_mode():
        x = q.clone()
        skl.rotary_fwd(x, k, plan, out=(x, k))
        assert torch.equal(x, ref[0])
    assert torch.equal(k, ref[1])


def test_not_finite_values_stay_in_their_pairs():
    q, _ = tensors(1, 1, 0, 4, 64, "fp32", 4)
    plan = skl.rotary_plan(64)
    ref = skl.rotary_fwd(q, None, plan)[0]
    q[0, 0, 2, 5] = float("nan")
    got = skl.rotary_fwd(q, None, plan)[0]
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[0, 0, 2, 5] = bad[0, 0, 2, 37] = True
    assert torch.equal(got.isnan(), bad) and torch.equal(got[~bad], ref[~bad])


def test_large_offsets():
    """A q of more than 2^32 bytes, strided, in place."""
    big = torch.empty(2, 33, 40000, 2048, device="cuda", dtype=torch.bfloat16)[..., :128]
    x = torch.randn(1, 1, 4, 128, device="cuda").to(torch.bfloat16)
    big[1:, -1:, -4:] = x
    plan = skl.rotary_plan(128)
    skl.rotary_fwd(big, None, plan, offset=3, out=(big, None))
    within(big[1:, -1:, -4:], x, plan, 3 + 39996 + torch.arange(4, device="cuda"), False)


def test_streams_and_graphs():
    q, k = tensors(2, 4, 2, 200, 128, "bf16", 5)
    plan = skl.rotary_plan(128)
    at = torch.randint(0, 100000, (2, 200), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = skl.rotary_fwd(q, k, plan, at)
    for seed in (6, 7):
        nq, nk = tensors(2, 4, 2, 200, 128, "bf16", seed)
        q.copy_(nq), k.copy_(nk), at.random_(0, 100000)
        graph.replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            ref = skl.rotary_fwd(q, k, plan, at)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_autograd():
    """The gradient is the inverse with the same amplitude; and the products <Rx, y> = <x, R^T y> agree."""
    q, k = (t.requires_grad_() for t in tensors(2, 4, 2, 50, 64, "fp32", 8))
    plan = skl.rotary_plan(32, scaling="parts", factor=8.0, trained_length=2048)
    at = torch.randint(0, 9000, (2, 50), device="cuda")
    yq, yk = skl.rotary(q, k, plan, at, interleaved=True)
    gq, gk = torch.randn_like(yq), torch.randn_like(yk)
    torch.autograd.backward((yq, yk), (gq, gk))
    within(q.grad, gq, plan, at, True, True)
    within(k.grad, gk, plan, at, True, True)
    a, b = ((x.detach().double() * y.double()).sum() for x, y in ((yq, gq), (q, q.grad)))
    assert abs(float(a - b)) <= 24 * U * 1.3 * 2 * float((gq.double().abs() * yq.detach().double().abs().amax()).sum())
    q.grad = None
    skl.rotary(q, k.detach(), plan, at)[0].sum().backward()
    assert q.grad is not None
    k.grad = None
    skl.rotary(q.detach(), k, plan)[1].sum().backward()
    assert k.grad is not None
