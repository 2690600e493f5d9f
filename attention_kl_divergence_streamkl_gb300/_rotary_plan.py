"""Rotary positions: the frequencies of a plan, unscaled or scaled for long contexts.

Frequencies are formed in 64-bit floating point and kept for the kernel as 64-bit
fractions of a turn, 2^64 f / 2 pi, so that position times frequency is exact
modulo a turn for any position.  The scalings:

* ``"positions"``: positions in between, f / factor (position interpolation, arXiv:2306.15595);
* ``"base"``: a larger base, base factor^(dim / (dim - 2)), which slows the slowest pair down by the factor and
  leaves the fastest;
* ``"parts"``: by parts (arXiv:2309.00071): pairs that turn beta_fast times or more within the trained length stay,
  those that turn beta_slow times or less slow down by the factor, a linear ramp over the pairs between; what is
  turned is multiplied by 0.1 ln(factor) + 1.
"""
from __future__ import annotations

import math
from decimal import Decimal, localcontext
from typing import NamedTuple

import torch

TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021")


class RotaryPlan(NamedTuple):
    """What rotary_fwd needs beside q and k; keep it for a model's life, and one for each device."""
    dim: int             # channels that turn
    turns: torch.Tensor  # int64 [dim / 2] on the device: 2^64 f / 2 pi, as bits
    amplitude: float     # factor on what is turned
    frequencies: tuple   # radians a position

    def to(self, device) -> "RotaryPlan":
        return self._replace(turns=self.turns.to(device))


def _parts(f, dim, base, factor, trained_length, beta_fast, beta_slow):
    def pair_that_turns(times):  # trained_length f = 2 pi times
        return dim * math.log(trained_length / (2 * math.pi * times)) / (2 * math.log(base))

    low = max(math.floor(pair_that_turns(beta_fast)), 0)
    high = min(math.ceil(pair_that_turns(beta_slow)), dim - 1)
    width = max(high - low, 1e-3)
    ramp = [min(max((i - low) / width, 0.0), 1.0) for i in range(dim // 2)]
    return [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)]


def rotary_plan(dim, base=10000.0, scaling=None, factor=1.0, trained_length=None, beta_fast=32.0, beta_slow=1.0,
                device=None) -> RotaryPlan:
    """The plan of rotary positions: pair i of `dim` channels turns by base^(-2 i / dim) radians a position.

    scaling: None, "positions", "base" or "parts" (see the module) by `factor` >= 1; "parts" needs the trained_length and
    takes beta_fast > beta_slow.  device: of the tensors that it will turn (default: the current CUDA device).
    """
    if dim != int(dim) or dim <= 0 or dim % 2:
        raise ValueError("dim must be a positive even number")
    if not (base > 1 and math.isfinite(base)):
        raise ValueError("base must be above 1")
    if not (factor >= 1 and math.isfinite(factor)):
        raise ValueError("factor must be at least 1")
    if scaling not in (None, "positions", "base", "parts"):
        raise ValueError("scaling must be None, 'positions', 'base' or 'parts'")
    if scaling is None and factor != 1:
        raise ValueError("a factor needs a scaling")
    dim, base, amplitude = int(dim), float(base), 1.0
    if scaling == "base" and dim > 2:
        base *= factor ** (dim / (dim - 2))
    f = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if scaling == "positions":
        f = [x / factor for x in f]
    if scaling == "parts":
        if trained_length is None or not trained_length > 0:
            raise ValueError("scaling by parts needs the trained_length")
        if not beta_fast > beta_slow > 0:
            raise ValueError("beta_fast must be above beta_slow, and both above 0")
        f = _parts(f, dim, base, factor, trained_length, beta_fast, beta_slow)
        amplitude = 0.1 * math.log(factor) + 1.0
    turns = []
    with localcontext() as ctx:
        ctx.prec = 60
        for x in f:
            t = int((Decimal(x) / TWO_PI * 2 ** 64).to_integral_value()) % 2 ** 64
            turns.append(t - 2 ** 64 if t >= 2 ** 63 else t)
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return RotaryPlan(dim, torch.tensor(turns, dtype=torch.int64, device=device), amplitude, tuple(f))
