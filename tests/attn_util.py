"""Attention's plain implementation in 64 bits, and the bounds its kernels' outputs are held to.

Bounds.  u = 2^-24 is half a step of fp32, h = 2^-8 half a step of bf16, X the largest scale sum_d |q_d| |k_d| over a
row's keys (so also above |S|).  A logit is a sum of D <= 128 products in fp32: off by at most (D + 4) u X, and its
exponent by that and a rounding of |x - m| <= 2 X + |LSE|: together within F = (D + 16) u (X + |LSE| + 1), of which 2^d
(ex2.approx: 2^-22 relative) adds 4 u.  So a weight p_ij / l_i is within a relative W = 2 F + (N_K / 32 + 80) u, the
second part for the sums (a row's thread adds its columns in chains; tiles and splits follow).
    O:    weights rounded to bf16 (h), summed with fp32 (W), O rounded (h):
          |dO| <= (h + W) sum_j P_ij |v_j| + h |O|
    LSE:  W + 2 u |LSE|
Gradients, with dP = dO V^T, delta = dO . O, dS = P (dP - delta + dlse):
    dP is a sum of D products: within (D + 4) u sum_d |dO_d| |v_jd| =: (D + 4) u a_ij;
    delta reads O as the forward rounded it: within e_i = (2 h + W) sum_d |dO_d| sum_j P_ij |v_jd| + (D + 8) u (same);
    dS, rounded to bf16 once (h) with P within W: |d dS| <= (h + W) |dS| + P_ij ((D + 4) u a_ij + e_i)
    dQ, dK: that through the product with |k|, |q| (fp32 sums add N u of the magnitudes), then h of the result;
    dV: P rounded to bf16: (h + W) sum_i P_ij |dO_i| + h |dV|.
Each bound is taken with a factor 1 + 2^-6 for products of errors.
"""
import math

import torch

H = 2.0 ** -8
U = 2.0 ** -24
NEG = float("-inf")


def tensors(B, H_, HK, NQ, NK, D, seed=0, rows_first=False, by=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def one(h, n, x=1.0):
        if rows_first:
            return (torch.randn(B, n, h, D, generator=gen, device="cuda") * x).to(torch.bfloat16).transpose(1, 2)
        return (torch.randn(B, h, n, D, generator=gen, device="cuda") * x).to(torch.bfloat16)

    return one(H_, NQ, by), one(HK, NK), one(HK, NK), one(H_, NQ)


def seen(B, NQ, NK, causal, q_lens, k_lens):
    """[B, 1, NQ, NK]: which keys a query sees."""
    i = torch.arange(NQ, device="cuda").view(1, 1, -1, 1)
    j = torch.arange(NK, device="cuda").view(1, 1, 1, -1)
    ql = torch.full((B,), NQ, device="cuda") if q_lens is None else q_lens.long().clamp(0, NQ)
    kl = torch.full((B,), NK, device="cuda") if k_lens is None else k_lens.long().clamp(0, NK)
    ql, kl = ql.view(-1, 1, 1, 1), kl.view(-1, 1, 1, 1)
    ok = (i < ql) & (j < kl)
    return ok & (j <= i + kl - ql) if causal else ok


def _clean(t, lens):
    """t in 64 bits with what lies past each sequence's length taken out."""
    t = t.double()
    if lens is None:
        return t
    past = torch.arange(t.shape[2], device="cuda").view(1, 1, -1, 1) >= lens.view(-1, 1, 1, 1)
    return torch.where(past, torch.zeros_like(t), t)


def forward(q, k, v, scale=None, causal=False, q_lens=None, k_lens=None):
    """(o, lse, bound of o, bound of lse) in 64 bits."""
    B, H_, NQ, D = q.shape
    HK, NK = k.shape[1:3]
    scale = scale or 1 / math.sqrt(D)
    q, k, v = _clean(q, q_lens), _clean(k, k_lens), _clean(v, k_lens)
    k, v = (t.repeat_interleave(H_ // HK, 1) for t in (k, v))
    ok = seen(B, NQ, NK, causal, q_lens, k_lens)
    s = torch.where(ok, scale * q @ k.transpose(2, 3), torch.full((), NEG, dtype=torch.float64, device="cuda"))
    lse = torch.logsumexp(s, -1) if NK else torch.full((B, H_, NQ), NEG, dtype=torch.float64, device="cuda")
    p = torch.where(ok, (s - torch.where(lse == NEG, torch.zeros_like(lse), lse)[..., None]).exp(), torch.zeros_like(s))
    o = p @ v
    if NK:
        X = torch.where(ok, scale * q.abs() @ k.abs().transpose(2, 3), torch.zeros_like(s)).amax(-1)
    else:
        X = torch.zeros_like(lse)
    size = torch.where(lse == NEG, torch.zeros_like(lse), lse.abs())
    W = 2 * (D + 16) * U * (X + size + 1) + (NK / 32 + 80) * U
    o_bound = ((H + W[..., None]) * (p @ v.abs()) + H * o.abs()) * (1 + 2 ** -6) + 2.0 ** -126
    return o, lse, o_bound, W + 2 * U * size, p, W


def backward(q, k, v, do, dlse=None, scale=None, causal=False, q_lens=None, k_lens=None):
    """((dq, dk, dv), their bounds) in 64 bits, from the formulas."""
    B, H_, NQ, D = q.shape
    HK, NK = k.shape[1:3]
    G = H_ // HK
    scale = scale or 1 / math.sqrt(D)
    o, lse, _, _, p, W = forward(q, k, v, scale, causal, q_lens, k_lens)
    q, k, v, do = _clean(q, q_lens), _clean(k, k_lens), _clean(v, k_lens), _clean(do, q_lens)
    k, v = (t.repeat_interleave(G, 1) for t in (k, v))
    dp = do @ v.transpose(2, 3)
    pull = dp - (do * o).sum(-1, keepdim=True)
    if dlse is not None:
        pull = pull + torch.where(lse == NEG, torch.zeros_like(lse), dlse.double())[..., None]
    ds = p * pull
    groups = lambda t: t.view(B, HK, G, NK, D).sum(2)  # noqa: E731
    dq, dk, dv = scale * ds @ k, groups(scale * ds.transpose(2, 3) @ q), groups(p.transpose(2, 3) @ do)
    a = do.abs() @ v.abs().transpose(2, 3)
    spread = (do.abs() * (p @ v.abs())).sum(-1, keepdim=True)
    W = W[..., None]
    e = (2 * H + W) * spread + (D + 8) * U * (spread + (0 if dlse is None else dlse.double().abs()[..., None]))
    eds = (H + W) * ds.abs() + p * ((D + 4) * U * a + e)
    more = 1 + 2 ** -6
    n = (NQ * G + 64) * U
    bq = (scale * (eds + (NK + 64) * U * ds.abs()) @ k.abs() + H * dq.abs()) * more + 2.0 ** -126
    bk = (groups(scale * (eds + n * ds.abs()).transpose(2, 3) @ q.abs()) + H * dk.abs()) * more + 2.0 ** -126
    bv = (groups(((H + W + n) * p).transpose(2, 3) @ do.abs()) + H * dv.abs()) * more + 2.0 ** -126
    return (dq, dk, dv), (bq, bk, bv)


def within(got, ref, bound, what):
    got = got.double()
    assert got.shape == ref.shape, what
    assert torch.equal(got == NEG, ref == NEG), what
    fin = ref != NEG
    over = ((got - ref).abs() / bound)[fin]
    assert over.numel() == 0 or bool((over <= 1).all()), f"{what}: {float(over.nan_to_num(1e9).max()):.2f} of its bound"
