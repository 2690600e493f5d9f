"""Attention on grids that a training step launches and small tests do not: more blocks than six for each SM (heads in order, not
longest tiles first), a fused backward whose last wave is dealt out, and every row and key by itself (bounds: attn_util.py)."""
import ctypes

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib, build
from tests import attn_util as A

pytestmark = pytest.mark.gpu
NEG = float("-inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    yield
    assert skl.check_device_status() == 0


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def lens(B, N, seed):
    """Lengths of a padded batch: whole, none, one, inside a tile."""
    some = [N, max(N - 131, 1), 1, 0, N // 2 + 1]
    return torch.tensor([some[(b + seed) % len(some)] for b in range(B)], dtype=torch.int32, device="cuda")


def tiles(n):
    return -(-n // 128)


def check_bwd(q, k, v, do, mode, dlse=None, **kw):
    o, lse = skl.attn_fwd(q, k, v, **kw)
    want, bounds = A.backward(q, k, v, do, dlse, **kw)
    got = skl.attn_bwd(q, k, v, o, lse, do, dlse, bwd_mode=mode, **kw)
    for name, g, w, b in zip(("dq", "dk", "dv"), got, want, bounds):
        A.within(g, w, b, name)
    return got


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal,padded", [(False, False), (True, False), (True, True)])
def test_forward_of_many_blocks(causal, padded, D):
    B, H, HK, NQ, NK = 5, 192, 48, 260, 300
    assert B * H * tiles(NQ) / 2 > 6 * sms() and skl.attn_fwd_plan(B, H, HK, NQ, NK, D, sms())[1] == 1
    q, k, v, _ = A.tensors(B, H, HK, NQ, NK, D, 1)
    kw = dict(causal=causal, **(dict(q_lens=lens(B, NQ, 0), k_lens=lens(B, NK, 1)) if padded else {}))
    o, lse = skl.attn_fwd(q, k, v, **kw)
    ro, rlse, bo, bl, _, _ = A.forward(q, k, v, **kw)
    A.within(lse, rlse, bl, "lse")
    A.within(o, ro, bo, "o")


@pytest.mark.parametrize("D,mode", [(64, skl.BWD_SEPARATE), (64, skl.BWD_FUSED), (128, skl.BWD_SEPARATE)])
@pytest.mark.parametrize("causal,padded", [(False, False), (True, False), (True, True)])
def test_backward_of_many_blocks(causal, padded, D, mode):
    B, H, HK, NQ, NK = 5, 130, 65, 140, 300
    assert B * HK * tiles(NK) > 6 * sms()  # the dK/dV blocks alone
    q, k, v, do = A.tensors(B, H, HK, NQ, NK, D, 2)
    kw = dict(causal=causal, **(dict(q_lens=lens(B, NQ, 2), k_lens=lens(B, NK, 0)) if padded else {}))
    dlse = torch.randn(B, H, NQ, device="cuda")
    check_bwd(q, k, v, do, mode, dlse, **kw)


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("G", [1, 3])
def test_fused_backward_with_a_last_wave_in_parts(G, padded):
    n, NK = sms(), 300
    HK = (n + n // 4) // tiles(NK) + 1  # a wave and a quarter of key tiles
    NQ = 1600 if G == 1 else 700
    path, parts, _, _ = skl.attn_bwd_plan(1, HK * G, HK, NQ, NK, 64, n)
    assert path == skl.BWD_FUSED and parts > 1 and HK * tiles(NK) > n
    q, k, v, do = A.tensors(1, HK * G, HK, NQ, NK, 64, 3)
    kw = dict(q_lens=lens(1, NQ, 1), k_lens=lens(1, NK, 1)) if padded else {}
    auto = check_bwd(q, k, v, do, skl.BWD_AUTO, **kw)
    fused = check_bwd(q, k, v, do, skl.BWD_FUSED, **kw)
    assert torch.equal(auto[1], fused[1]) and torch.equal(auto[2], fused[2])


@pytest.mark.parametrize("D,mode", [(64, skl.BWD_SEPARATE), (64, skl.BWD_FUSED), (128, skl.BWD_SEPARATE)])
@pytest.mark.parametrize("G", [1, 2])
def test_every_row_and_every_key_counts(G, D, mode):
    """Sequence b's loss reads one row of O alone (dk and dv are that row's share, dq is zero elsewhere), then one key alone has
    a value (dq and dv are that key's): a row or a key that a tile left out would be all of its gradient."""
    N = 1100
    at = [0, 1, 31, 32, 63, 127, 128, 200, 255, 256, 511, 512, 640, 767, 895, 896, 1023, 1024, 1098, 1099]
    B = len(at)
    q, k, v, do = A.tensors(B, G, 1, N, N, D, 4)
    one = torch.zeros_like(do)
    single = torch.zeros_like(v)
    for b, i in enumerate(at):
        one[b, :, i] = do[b, :, i]
        single[b, :, i] = v[b, :, i]
    for causal in (False, True):
        check_bwd(q, k, v, one, mode, causal=causal)
        dq, _, _ = check_bwd(q, k, single, do, mode, causal=causal)
        dq1, dk1, dv1 = check_bwd(q, k, single, one, mode, causal=causal)
        for b, i in enumerate(at):
            others = torch.arange(N, device="cuda") != i
            assert bool((dq1[b][:, others] == 0).all())
            if causal:
                assert bool((dq[b][:, :i] == 0).all()) and bool((dv1[b][:, i + 1:] == 0).all())


def exact_delta_bounds(q, k, v, do, **kw):
    """The bounds of attn_util.backward with delta computed as sum_j P_ij dP_ij in fp32, as it is for rows of at most 32 keys: P
    is within W, dP_ij within (D + 4) u a_ij and their sum within 64 u more, so the error of delta is
    e_i = sum_j P_ij ((W + 64 u) |dP_ij| + (D + 4) u a_ij), with no part that O's rounding leaves."""
    B, H, NQ, D = q.shape
    HK, NK = k.shape[1:3]
    G, scale = H // HK, D ** -0.5
    o, lse, _, _, p, W = A.forward(q, k, v, **kw)
    qd, kd, vd, dod = (t.double() for t in (q, k, v, do))
    kd, vd = (t.repeat_interleave(G, 1) for t in (kd, vd))
    dp = dod @ vd.transpose(2, 3)
    ds = p * (dp - (dod * o).sum(-1, keepdim=True))
    a = dod.abs() @ vd.abs().transpose(2, 3)
    W = W[..., None]
    e = (p * ((W + 64 * A.U) * dp.abs() + (D + 4) * A.U * a)).sum(-1, keepdim=True)
    eds = (A.H + W) * ds.abs() + p * ((D + 4) * A.U * a + e)
    groups = lambda t: t.view(B, HK, G, NK, D).sum(2)  # noqa: E731
    dq, dk = scale * ds @ kd, groups(scale * ds.transpose(2, 3) @ qd)
    more = 1 + 2 ** -6
    bq = (scale * (eds + (NK + 64) * A.U * ds.abs()) @ kd.abs() + A.H * dq.abs()) * more + 2.0 ** -126
    bk = (groups(scale * (eds + (NQ * G + 64) * A.U * ds.abs()).transpose(2, 3) @ qd.abs()) + A.H * dk.abs()) * more + 2.0 ** -126
    return (dq, bq), (dk, bk)


@pytest.mark.parametrize("D,mode", [(64, skl.BWD_SEPARATE), (64, skl.BWD_FUSED), (128, skl.BWD_SEPARATE)])
@pytest.mark.parametrize("NQ,NK", [(5, 1), (200, 2), (300, 31), (130, 32), (32, 32)])
def test_rows_of_few_keys_do_not_pass_on_the_rounding_of_o(NQ, NK, D, mode):
    """Values with a large common part: dO . O, with O rounded to bf16, would be off by more than these bounds."""
    for causal in (False, True):
        q, k, v, do = A.tensors(2, 4, 2, NQ, NK, D, NQ + NK)
        v = (v.float() + 10 * torch.randn(2, 2, 1, D, device="cuda", generator=torch.Generator("cuda").manual_seed(1))).to(v.dtype)
        got = check_bwd(q, k, v, do, mode, causal=causal)
        for g, (w, b), name in zip(got, exact_delta_bounds(q, k, v, do, causal=causal), ("dq", "dk")):
            A.within(g, w, b, name)


@pytest.mark.parametrize("B,H,HK,NQ,NK,D,mode,parts", [
    (2, 8, 2, 100, 100, 64, skl.BWD_SEPARATE, 1), (1, 4, 1, 2100, 60, 128, skl.BWD_SEPARATE, 2),
    (2, 8, 2, 100, 100, 64, skl.BWD_FUSED, 1), (1, 64, 64, 1600, 300, 64, skl.BWD_FUSED, 2)])
def test_a_workspace_that_is_a_byte_short_is_refused(B, H, HK, NQ, NK, D, mode, parts):
    """... before anything is launched, whatever part of the plan needs the byte."""
    need, kv, dq_parts = (skl.attn_bwd_plan(B, H, HK, NQ, NK, D, sms(), bwd_mode=mode)[i] for i in (3, 1, 2))
    assert (max(kv, dq_parts) > 1) == (parts > 1) and need > B * H * NQ * 32
    q, k, v, do = A.tensors(B, H, HK, NQ, NK, D, 5)
    o, lse = skl.attn_fwd(q, k, v)
    out = [torch.full_like(t, 7) for t in (q, k, v)]
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    s = _lib.make_attn_shape(B, H, HK, NQ, NK, D)
    call = lambda n: _lib.lib().streamkl_attn_bwd(  # noqa: E731
        *(ctypes.c_void_p(t.data_ptr()) for t in (q, k, v, o, lse, do)), None, s,
        *(ctypes.c_void_p(t.data_ptr()) for t in out), mode, ctypes.c_void_p(ws.data_ptr()), n,
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert call(need - 1) == _lib.ERR_WORKSPACE
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in out)
    assert call(need) == _lib.OK
    for a, b in zip(out, skl.attn_bwd(q, k, v, o, lse, do, bwd_mode=skl.BWD_SEPARATE)):
        assert float((a.double() - b.double()).norm() / b.double().norm()) < 1e-2


def test_a_forward_workspace_that_is_a_byte_short_is_refused():
    q, k, v, _ = A.tensors(1, 8, 2, 2, 20000, 128, 6)
    s = _lib.make_attn_shape(1, 8, 2, 2, 20000, 128)
    need = ctypes.c_size_t()
    assert _lib.lib().streamkl_attn_fwd_workspace(s, ctypes.byref(need)) == _lib.OK and need.value > 0
    o, lse = torch.full_like(q, 7), torch.full((1, 8, 2), 7.0, device="cuda")
    ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    status = _lib.lib().streamkl_attn_fwd(
        *(ctypes.c_void_p(t.data_ptr()) for t in (q, k, v)), s, *(ctypes.c_void_p(t.data_ptr()) for t in (o, lse, ws)),
        need.value - 1, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert status == _lib.ERR_WORKSPACE and bool((o == 7).all()) and bool((lse == 7).all())
