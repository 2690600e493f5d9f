"""Cross entropy over a vocabulary: a weight, its gradient and a piece of d of more than 2^31 values, against 64 bits.

The weight's case has hidden states of -1, 0 and 1 and a weight of multiples of 1/64 up to 1/16, so that all logits are exact in
fp32 and only the roundings behind them are left: with u = 2^-24 and Z = max |z| + |LSE| + 1 an exponent is off by 4 u Z, so
    LSE:  B = (8 Z + V / 2048 + 100) u,   the loss the same and 4 u of itself,   d: within h |d| + (g + |d|) 2 B
with h half a step of bf16.  Products and sums of both gradients as in test_gpu_vocab_xent.py.  These are about h of the sums of
magnitudes; an answer of zeros, or of another place's rows, is outside nearly everywhere, which the tests look at themselves.
"""
import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib as K
from tests import test_gpu_vocab_xent as X

pytestmark = pytest.mark.gpu
U, H = X.U, 2.0 ** -8
STEP = 10000  # rows of the weight at a time in 64 bits


def tells(ref, bound):
    """Zeros, or these rows in another order, would be seen in most places."""
    assert float((bound < ref.abs()).double().mean()) > 0.5
    assert float((bound < (ref - ref.roll(1, 0)).abs()).double().mean()) > 0.5


def test_a_weight_past_32_bits():
    R, C, V = 12, 16384, 140000  # 2^31 values end in row 131072
    gen = torch.Generator(device="cuda").manual_seed(51)
    h = torch.randint(-1, 2, (R, C), generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.empty(V, C, device="cuda", dtype=torch.bfloat16)
    for x in w.split(STEP):
        x.copy_(torch.randint(-4, 5, x.shape, generator=gen, device="cuda", dtype=torch.int8) / 64)
    t = torch.randint(0, V, (R,), generator=gen, device="cuda")
    t[0], t[1], t[2], t[3] = V - 1, 131072, -1, 131071
    g = torch.rand(R, generator=gen, device="cuda") + 0.5
    loss, lse = skl.vocab_xent_fwd(h, w, t)
    hd = h.double()
    z = torch.cat([hd @ x.double().T for x in w.split(STEP)], 1)
    rz = torch.logsumexp(z, -1)
    there = t >= 0
    rl = torch.where(there, rz - z.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    B = (8 * (z.abs().amax(-1) + rz.abs() + 1) + V / 2048 + 100) * U
    assert float(B.max()) < 1e-4
    X.within(lse, rz, B, "lse")
    X.within(loss, rl, B + 4 * U * rl.abs(), "loss")
    dh, dw = skl.vocab_xent_bwd(h, w, t, lse, g)
    g = torch.where(there, g, 0.0).double()
    d = g[:, None] * (z - rz[:, None]).exp()
    dd = d * 2 * B[:, None]
    d[torch.arange(R), t.clamp(min=0)] -= g
    dd += H * d.abs()
    dd[torch.arange(R), t.clamp(min=0)] += g * 4 * U
    ref, size = torch.zeros(R, C, dtype=torch.float64, device="cuda"), torch.zeros(R, C, dtype=torch.float64, device="cuda")
    off = torch.zeros(R, C, dtype=torch.float64, device="cuda")
    for v in range(0, V, STEP):
        here, cols = w[v:v + STEP].double(), slice(v, v + STEP)
        ref += d[:, cols] @ here
        off += dd[:, cols] @ here.abs()
        size += d[:, cols].abs() @ here.abs()
        rw = d[:, cols].T @ hd
        bw = (dd[:, cols].T @ hd.abs() + 66 * U * (d[:, cols].abs().T @ hd.abs()) + H * rw.abs()) * (1 + 2 ** -6) + 2.0 ** -126
        X.within(dw[cols], rw, bw, f"dweight from {v}")
        tells(rw, bw)
    bh = (off + (V / 8 + 64) * U * size + H * ref.abs()) * (1 + 2 ** -6) + 2.0 ** -126
    X.within(dh, ref, bh, "dhidden")
    tells(ref[there], bh[there])
    assert skl.check_device_status() == K.OK


@pytest.mark.parametrize("first", [0, 261900, 269500])
def test_rows_of_d_past_32_bits_in_both_gradients(first):
    """2^31 values of d end in row 262144; only 500 rows have a gradient."""
    R, C, V = 270000, 64, 8192
    assert skl.vocab_xent_plan(R, V, C, 152)[0] == 1
    h, w, t = X.inputs(R, C, V, "bf16", 52)
    rows = slice(first, first + 500)
    gen = torch.Generator(device="cuda").manual_seed(53)
    g, gl = torch.zeros(R, device="cuda"), torch.zeros(R, device="cuda")
    g[rows] = torch.rand(500, generator=gen, device="cuda")
    gl[rows] = torch.rand(500, generator=gen, device="cuda")
    _, lse = skl.vocab_xent_fwd(h, w, t)
    dh, dw = skl.vocab_xent_bwd(h, w, t, lse, g, gl)
    rh, rw, bh, bw = X.backward(h[rows], w, t[rows], g[rows], gl[rows], 1.0)
    X.within(dh[rows], rh, bh, "dhidden")
    X.within(dw, rw, bw, "dweight")
    tells(rh, bh)
    tells(rw, bw)
    dh[rows] = 0
    assert not bool(dh.any())
    assert skl.check_device_status() == K.OK
