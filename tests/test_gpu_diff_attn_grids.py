"""Differential attention on grids that a training step launches and small tests do not: more blocks than six for each SM, a
backward whose tiles are dealt out over several blocks, many rows' blocks (bounds: test_gpu_diff_attn.py)."""
import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import build
from tests import attn_util as A
from tests.test_gpu_diff_attn import check, gradients, inputs, reference

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal,padded", [(False, False), (True, False), (True, True)])
def test_forward_of_many_blocks(causal, padded, D):
    B, H, HK, NQ, NK = 5, 96, 24, 260, 300
    assert B * H * -(-NQ // 128) > 6 * sms() and skl.diff_attn_plan(B, H, HK, NQ, NK, D, sms())[1] == 1
    q, k, v, lam, _ = inputs(B, H, HK, NQ, NK, D, 1)
    kw = dict(causal=causal, **(dict(q_lens=lens(B, NQ, 0), k_lens=lens(B, NK, 1)) if padded else {}))
    rd, rz, bd, bz, o, e = reference(q, k, v, lam, **kw)
    d, lse = skl.diff_attn_fwd(q, k, v, lam, **kw)
    A.within(d, rd, bd, "d")
    A.within(lse, rz, bz, "lse")
    d2, _, maps, rest = skl.diff_attn_fwd(q, k, v, lam, return_maps=True, **kw)
    A.within(d2, rd, bd, "d with the maps")
    A.within(maps.double() + rest.double(), o, e + 2.0 ** -16 * o.abs() + 2.0 ** -126, "maps")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("late", [0, 1])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5, 8, 13])
def test_one_map_is_done_before_the_other(tiles, late, D):
    """The late map's logits grow by 22 in the last key tile, so that its reference moves there, while the other map's tile is
    done; the last keys' values then lie in each place of the ring that a tile count leaves them in."""
    B, H, HK, NQ, NK = 2, 40, 20, 200, 128 * tiles
    assert skl.diff_attn_plan(B, H, HK, NQ, NK, D, sms())[:2] == (False, 1)
    q, k, v, lam, _ = inputs(B, H, HK, NQ, NK, D, 7)
    k[..., 0] = 0
    k[:, :, -128:, 0] = 16 * (D / 128) ** 0.25
    q[:, 1 - late::2, :, 0] = 0
    q[:, late::2, :, 0] = 16 * (D / 128) ** 0.25
    rd, rz, bd, bz, o, e = reference(q, k, v, lam)
    for _ in range(4):
        d, lse = skl.diff_attn_fwd(q, k, v, lam)
        A.within(d, rd, bd, "d")
        A.within(lse, rz, bz, "lse")
        d, _, maps, rest = skl.diff_attn_fwd(q, k, v, lam, return_maps=True)
        A.within(d, rd, bd, "d with the maps")
        A.within(maps.double() + rest.double(), o, e + 2.0 ** -16 * o.abs() + 2.0 ** -126, "maps")


@pytest.mark.parametrize("D", [64, 128])
def test_backward_of_many_blocks(D):
    """Every tile a block of its own, and for D 64 the path that visits each tile pair once."""
    B, H, HK, NQ, NK = 4, 24, 24, 300, 500
    path = skl.attn_bwd_plan(B, 2 * H, HK, NQ, NK, D, sms())
    assert path[1] == 1 and path[0] == (skl.BWD_FUSED if D == 64 else skl.BWD_SEPARATE)
    check(B, H, HK, NQ, NK, D, 2, causal=True, modes=(skl.BWD_AUTO, skl.BWD_SEPARATE), dlse=True)


@pytest.mark.parametrize("D", [64, 128])
def test_backward_in_parts(D):
    """Few key heads under many queries: a key tile's stream is dealt out over several blocks, its partial sums are added."""
    B, H, HK, NQ, NK = 1, 4, 1, 1100, 1000
    assert max(skl.attn_bwd_plan(B, 2 * H, HK, NQ, NK, D, sms(), bwd_mode=skl.BWD_SEPARATE)[1:3]) > 1
    q, k, v, lam, do = inputs(B, H, HK, NQ, NK, D, 3)
    _, lse, maps, rest = skl.diff_attn_fwd(q, k, v, lam, return_maps=True)
    ref, bounds = gradients(q, k, v, lam, do)
    first = None
    for _ in range(3):
        got = skl.diff_attn_bwd(q, k, v, lam, maps, lse, do, bwd_mode=skl.BWD_SEPARATE, maps_rest=rest)
        for g, r, b, what in zip(got, ref, bounds, ("dq", "dk", "dv", "dlam")):
            A.within(g, r, b, what)
        assert first is None or all(torch.equal(x, y) for x, y in zip(got, first))
        first = got


def test_weights_near_zero_and_large_with_gradients_of_the_log_sum_exps():
    """|lam| from 0 over 2^-30 to 2^10, signs mixed, beside gradients of both maps' log-sum-exps."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    sizes = torch.tensor([0.0, 2.0 ** -30, 2.0 ** -7, 2.0 ** -6, 2.0 ** -5, 1.0, 2.0 ** 10], device="cuda")

    def pick(l):
        at = torch.randint(0, 7, l.shape, generator=gen, device="cuda")
        return sizes[at] * (1 - 2 * torch.randint(0, 2, l.shape, generator=gen, device="cuda"))

    for D in (64, 128):
        check(1, 2, 1, 200, 150, D, 5, lam=pick, dlse=True, modes=(skl.BWD_SEPARATE,) + ((skl.BWD_FUSED,) if D == 64 else ()))
        check(1, 2, 1, 200, 150, D, 6, lam=pick, modes=(skl.BWD_SEPARATE,) + ((skl.BWD_FUSED,) if D == 64 else ()))
