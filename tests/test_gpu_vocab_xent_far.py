"""Cross entropy over a vocabulary: a loss keeps its digits however far from 0 its logits lie.

Hidden states and weights are small multiples of 1/4 and 1/8, and every sum of their products is exact in fp32, so that what
is left are the roundings behind the logits.  u = 2^-24, Y the largest |scale (z_v - z_t)| of a row.  The loss is the log of the
sum of 2^(c (z_v - z_t)), formed from differences to a maximum that is subtracted as it was rounded: c = scale log2(e) is off by 2 u,
each difference is rounded once, in units of log 2 and back (3 u), so an exponent by 6 u Y; 2^x by 4 u, the sum by
(V / 2048 + 96) u, the logarithm and the last sum by 2 u (|loss| + log V):
    |loss| off by (6 Y + V / 2048 + 100 + 4 (|loss| + log V)) u, whatever the logits themselves are;
    LSE, which is stored in fp32, by 4 u |LSE| more.
"""
import math

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from tests.test_gpu_vocab_xent import TYPES, U, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R,C,V", [(64, 64, 1000), (1, 64, 20000), (300, 1032, 3001)])
@pytest.mark.parametrize("far,scale", [(64.0, 1.0), (-64.0, 1.0), (64.0, 0.5), (60.0, 1.25), (0.0, 1.0)])
def test_a_loss_keeps_its_digits(far, scale, R, C, V, dtype):
    gen = torch.Generator(device="cuda").manual_seed(V + C)
    h = torch.randint(-8, 9, (R, C), generator=gen, device="cuda") / 4
    w = torch.randint(-4, 5, (V, C), generator=gen, device="cuda") / 8
    h[:, 0], w[:, 0] = 64.0, far  # every logit is moved by thousands
    h, w = h.to(TYPES[dtype]), w.to(TYPES[dtype])
    t = torch.randint(0, V, (R,), generator=gen, device="cuda")
    assert float((h.double().abs() @ w.double().abs().T).max()) * 32 < 2 ** 24  # multiples of 1/32: exact sums
    z = scale * (h.double() @ w.double().T)
    lse, given = torch.logsumexp(z, -1), z.gather(1, t[:, None])
    Y = (z - given).abs().amax(-1)
    ref = torch.logsumexp(z - given, -1)
    bound = (6 * Y + V / 2048 + 100 + 4 * (ref.abs() + math.log(V))) * U
    assert float(bound.max()) < 1e-4  # a rounding of the logits of 4096 is 2.4e-4 already
    loss, got = skl.vocab_xent_fwd(h, w, t, scale)
    within(loss, ref, bound, "loss")
    within(got, lse, bound + 4 * U * lse.abs(), "lse")
