"""Rotary positions: how exact an angle is.

The product of a position and a frequency in 2^-64 of a turn is exact modulo a turn.  Sine and cosine are taken of its upper 32
bits, which the rest, below 2^-32 of a turn, is cut off from; they are each within 6 u = 6 2^-24 of themselves
(test_gpu_rotary.py).  So of a pair (1, 0) in fp32, the results are off by at most 2 pi 2^-32 + 6 u of their size.  The formula's
own angle, up to pi in 64 bits, has three roundings (pi, a division's, a product's): within 3 pi 2^-53 < 2^-49 of it.
"""
import math

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def whole(x):
    x %= 2 ** 64
    return x - 2 ** 64 if x >= 2 ** 63 else x


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_small_angles_and_those_next_to_quarter_turns(inverse, interleaved):
    turns = [2 ** 64 // 4 * i + s * x for i in range(4) for x in (0, 1, 12345, 2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 40 + 2 ** 31, 2 ** 50 + 1,
                                                                 2 ** 61 - 1, 2 ** 61, 2 ** 62 - 2 ** 33) for s in (-1, 1)]
    turns += [0x9E3779B97F4A7C15 * i for i in range(1, 41)]
    dim = 2 * len(turns)
    plan = skl.RotaryPlan(dim, torch.tensor([whole(t) for t in turns], device="cuda"), 1.0, tuple(t / 2 ** 64 * 2 * math.pi for t in turns))
    at = [1, 3, -1, 2 ** 20 + 1, 2 ** 33 + 5, -2 ** 63, 2 ** 63 - 1]
    x = torch.zeros(1, 1, len(at), dim, device="cuda")
    first, second = (slice(0, dim, 2), slice(1, dim, 2)) if interleaved else (slice(0, dim // 2), slice(dim // 2, dim))
    x[..., first] = 1.0
    f = skl.rotary_bwd if inverse else skl.rotary_fwd
    got, _ = f(x, None, plan, positions=torch.tensor(at, device="cuda"), interleaved=interleaved)
    for n, p in enumerate(at):
        angle = [whole(p * t) / 2 ** 64 * 2 * math.pi * (-1 if inverse else 1) for t in turns]
        for y, of in ((got[0, 0, n, first], math.cos), (got[0, 0, n, second], math.sin)):
            ref = torch.tensor([of(a) for a in angle], dtype=torch.float64, device="cuda")
            over = (y.double() - ref).abs() - (2 * math.pi * 2.0 ** -32 + 6 * U * ref.abs() + 2.0 ** -49)
            assert bool((over <= 0).all()), (p, float(over.max()))
