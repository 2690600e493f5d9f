"""Rotary positions: the plan's frequencies, and what the entry points refuse, on the host before anything is launched."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib as K
from attention_kl_divergence_streamkl_gb300 import build as B

TWO_PI = Fraction("6.28318530717958647692528676655900576839433879875021")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return K.lib()


def ptr(off=0):
    return ctypes.c_void_p(0x10000000 + off)


SHAPE = dict(B=2, HQ=4, HK=2, N=8, D=64, dim=64, dtype=0, interleaved=0, amplitude=1.0, offset=0, positions=None, positions_bytes=0,
             positions_stride=0, qb=2048, qh=512, qn=64, kb=1024, kh=512, kn=64, qob=2048, qoh=512, qon=64, kob=1024, koh=512, kon=64)


def call(lib, q=ptr(), k=ptr(16), turns=ptr(32), q_out=ptr(64), k_out=ptr(128), **change):
    return lib.streamkl_rotary(q, k, K.RotaryShape(*{**SHAPE, **change}.values()), turns, q_out, k_out, 0, None)


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), K.ERR_INVALID), (dict(HQ=-1), K.ERR_INVALID), (dict(N=-1), K.ERR_INVALID), (dict(D=0), K.ERR_INVALID),
    (dict(dim=0), K.ERR_INVALID), (dict(dim=66), K.ERR_INVALID), (dict(dim=31), K.ERR_INVALID), (dict(dtype=3), K.ERR_INVALID),
    (dict(D=65), K.ERR_UNSUPPORTED), (dict(amplitude=float("nan")), K.ERR_INVALID), (dict(amplitude=float("inf")), K.ERR_INVALID),
    (dict(positions=ptr(), positions_bytes=2), K.ERR_INVALID), (dict(positions=ptr(4), positions_bytes=8), K.ERR_INVALID),
    (dict(positions=ptr(), positions_bytes=8, positions_stride=-1), K.ERR_INVALID), (dict(qh=-1), K.ERR_INVALID),
    (dict(HQ=65535), K.ERR_UNSUPPORTED), (dict(B=1 << 16, N=1 << 16), K.ERR_UNSUPPORTED),
    (dict(q=None), K.ERR_INVALID), (dict(k=None), K.ERR_INVALID), (dict(q=ptr(1)), K.ERR_INVALID), (dict(q_out=None), K.ERR_INVALID),
    (dict(k_out=None), K.ERR_INVALID), (dict(turns=None), K.ERR_INVALID), (dict(turns=ptr(4)), K.ERR_INVALID),
    (dict(dtype=2, q=ptr(2)), K.ERR_INVALID),
    (dict(qoh=0), K.ERR_INVALID), (dict(qon=32), K.ERR_INVALID), (dict(kob=512), K.ERR_INVALID),  # rows on one another
    (dict(q_out=ptr(), qoh=64, qon=256), K.ERR_INVALID),  # in place, rows on other rows
    (dict(k_out=ptr(64)), K.ERR_INVALID), (dict(q_out=ptr(16)), K.ERR_INVALID), (dict(k_out=ptr()), K.ERR_INVALID),  # on the other
])
def test_refuses(lib, change, code):
    assert call(lib, **change) == code


@pytest.mark.parametrize("change", [dict(B=0), dict(N=0), dict(HQ=0, HK=0)])
def test_nothing_to_turn(lib, change):
    assert call(lib, q=None, k=None, turns=None, q_out=None, k_out=None, **change) == K.OK


@pytest.mark.parametrize("dim,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (20, 1.5)])
def test_turns_are_the_frequencies(dim, base):
    """2^64 f / 2 pi to the nearest, for frequencies in 64 bits."""
    plan = skl.rotary_plan(dim, base, device="cpu")
    assert plan.dim == dim and plan.amplitude == 1.0 and plan.turns.dtype == torch.int64 and plan.turns.shape == (dim // 2,)
    for i, (f, t) in enumerate(zip(plan.frequencies, plan.turns.tolist())):
        assert abs(f - base ** (-2 * i / dim)) <= 1e-15 * f
        assert abs(Fraction(f) / TWO_PI * 2 ** 64 - t % 2 ** 64) <= Fraction(1, 2)


@pytest.mark.parametrize("factor", [1.0, 2.0, 32.0])
def test_scalings(factor):
    dim, plain = 128, skl.rotary_plan(128, device="cpu").frequencies
    between = skl.rotary_plan(dim, scaling="positions", factor=factor, device="cpu")
    assert between.frequencies == tuple(x / factor for x in plain) and between.amplitude == 1.0
    base = skl.rotary_plan(dim, scaling="base", factor=factor, device="cpu").frequencies
    assert base[0] == 1.0 and abs(base[-1] * factor / plain[-1] - 1) < 1e-12
    parts = skl.rotary_plan(dim, scaling="parts", factor=factor, trained_length=4096, device="cpu")
    assert abs(parts.amplitude - (0.1 * math.log(factor) + 1)) < 1e-15
    for x, y in zip(plain, parts.frequencies):
        turned = 4096 * x / (2 * math.pi)
        assert x / factor * (1 - 1e-12) <= y <= x * (1 + 1e-12)
        if turned >= 33:  # the ramp begins at a whole pair
            assert abs(y / x - 1) < 0.05 or turned < 40
        if turned < 0.8:
            assert abs(y * factor / x - 1) < 1e-12
    assert parts.frequencies[0] == 1.0


@pytest.mark.parametrize("args", [dict(dim=0), dict(dim=7), dict(dim=-2), dict(dim=64, base=1.0), dict(dim=64, base=float("inf")),
                                  dict(dim=64, scaling="other", factor=2.0), dict(dim=64, factor=2.0),
                                  dict(dim=64, scaling="base", factor=0.5), dict(dim=64, scaling="parts", factor=2.0),
                                  dict(dim=64, scaling="parts", factor=2.0, trained_length=4096, beta_fast=1.0)])
def test_plan_refuses(args):
    with pytest.raises(ValueError):
        skl.rotary_plan(**args, device="cpu")


@pytest.mark.parametrize("change,error", [
    (dict(q=torch.zeros(1, 2, 3, 8, dtype=torch.float64)), TypeError), (dict(q=torch.zeros(2, 3, 8)), ValueError),
    (dict(q=None, k=None), ValueError), (dict(q=torch.zeros(1, 2, 3, 9), k=None), ValueError),
    (dict(q=torch.zeros(1, 2, 3, 4), k=None), ValueError), (dict(k=torch.zeros(1, 2, 4, 8)), ValueError),
    (dict(k=torch.zeros(1, 2, 3, 8, dtype=torch.bfloat16)), ValueError),
])
def test_binding_refuses(change, error):
    """On the host alone: the sizes are looked at before the device."""
    args = dict(q=torch.zeros(1, 2, 3, 8), k=torch.zeros(1, 2, 3, 8))
    args.update(change)
    if not torch.cuda.is_available() and "k" in change and change["k"] is not None:
        pytest.skip("looked at beside the device's tensors")
    with pytest.raises(error):
        skl.rotary_fwd(args["q"], args["k"], skl.rotary_plan(8, device="cuda" if torch.cuda.is_available() else "cpu"))
