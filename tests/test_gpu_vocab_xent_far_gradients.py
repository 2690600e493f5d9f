"""Cross entropy over a vocabulary: the gradients of rows whose logits lie far from 0.

As in test_gpu_vocab_xent_far.py all logits are exact in fp32.  p = 2^(c z - l') with l' = lse log2(e): with u = 2^-24 and
M = max(|z|, |lse|), c z is off by 2 u M (c), the stored lse by 2 u M (ln 2 and its own rounding) and 2 u M (c), l' by 2 u M: p is
within P = (8 M + 8 + V / 2048 + 100) u of itself, where 8 are the exponent's and 2^x's and the last the sum's.  d, with h half a
step of the type, within h |d| + scale (|g| + |g'|) (p P + 4 u) and fp16's least step; the products as in test_gpu_vocab_xent.py.
"""
import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from tests.test_gpu_vocab_xent import TYPES, U, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("far", [64.0, -64.0, 0.0])
@pytest.mark.parametrize("R,C,V,scale", [(64, 64, 1000, 1.0), (300, 72, 3001, 0.5), (5, 64, 20000, 1.25)])
def test_gradients_far_from_zero(R, C, V, scale, far, dtype):
    gen = torch.Generator(device="cuda").manual_seed(V + C + 1)
    h = torch.randint(-8, 9, (R, C), generator=gen, device="cuda") / 4
    w = torch.randint(-4, 5, (V, C), generator=gen, device="cuda") / 8
    h[:, 0], w[:, 0] = 64.0, far
    h, w = h.to(TYPES[dtype]), w.to(TYPES[dtype])
    t = torch.randint(0, V, (R,), generator=gen, device="cuda")
    g, gl = (torch.rand(R, generator=gen, device="cuda") + 0.5 for _ in range(2))
    z = scale * (h.double() @ w.double().T)
    lse = torch.logsumexp(z, -1)
    M = torch.maximum(z.abs().amax(-1), lse.abs())
    P = (8 * M + 8 + V / 2048 + 100) * U
    p = (z - lse[:, None]).exp()
    size = scale * (g + gl).double()
    d = size[:, None] * p
    d[torch.arange(R), t] -= scale * g.double()
    half = torch.finfo(h.dtype).eps / 2
    least = float(size.max()) * 2.0 ** -37 if dtype == "fp16" else 0.0
    dd = half * d.abs() + size[:, None] * (p * P[:, None] + 4 * U) + least
    tiny = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -126
    _, got = skl.vocab_xent_fwd(h, w, t, scale)
    within(got, lse, (4 * M + V / 2048 + 100) * U, "lse")
    dh, dw = skl.vocab_xent_bwd(h, w, t, got, g, gl, scale)
    for x, ref, size_of, off, n, what in ((dh, d @ w.double(), d.abs() @ w.double().abs(), dd @ w.double().abs(), V, "dhidden"),
                                          (dw, d.T @ h.double(), d.abs().T @ h.double().abs(), dd.T @ h.double().abs(), R, "dweight")):
        within(x, ref, (off + (n / 8 + 64) * U * size_of + half * ref.abs()) * (1 + 2 ** -6) + tiny, what)
