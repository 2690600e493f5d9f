"""A student's step with the layer operators together: queries and keys turned by their positions, differential attention,
the KL of its first maps to the teacher's on the same turned Q and K, and the loss on the data's tokens from the hidden
states, with all gradients."""
import math

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import build

pytestmark = pytest.mark.gpu
B, H, N, D, V = 2, 4, 200, 64, 1003


def step(q, k, v, mix, head, tq, tk, at, data, ops):
    """q [B, 2 H, N, D], k and v [B, H, N, D], mix [H, 1] (the weights before their sigmoid), head [V, H D]; the teacher's tq,
    tk are turned already."""
    rotary, attention, kl, cross_entropy = ops
    q, k = rotary(q, k, at)
    o = attention(q, k, v, mix.sigmoid())
    hidden = o.transpose(1, 2).reshape(B, N, H * D)
    loss, lse = cross_entropy(hidden, head, data)
    return kl(tq, tk, q[:, 0::2], k) + loss.sum() / (data >= 0).sum() + 1e-3 * (lse * lse).mean()


def plain_ops(plan):
    f = torch.tensor(plan.frequencies, dtype=torch.float64, device="cuda")

    def rotary(q, k, at):
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), at.double()[:, None, :, None] * f) * plan.amplitude

        def one(x):
            half = plan.dim // 2
            z = torch.complex(x[..., :half], x[..., half:plan.dim]) * turn
            return torch.cat((z.real, z.imag, x[..., plan.dim:]), -1)

        return one(q), one(k)

    def log_map(q, k):
        s = q @ k.transpose(2, 3) / math.sqrt(D)
        see = torch.ones(N, N, dtype=torch.bool, device="cuda").tril()
        return torch.log_softmax(torch.where(see, s, torch.full_like(s, -1e300)), -1), see

    def attention(q, k, v, lam):
        return (log_map(q[:, 0::2], k)[0].exp() - lam.unsqueeze(-1) * log_map(q[:, 1::2], k)[0].exp()) @ v

    def kl(q1, k1, q2, k2):
        (a, see), (b, _) = log_map(q1, k1), log_map(q2, k2)
        return torch.where(see, a.exp() * (a - b), torch.zeros_like(a)).sum(-1).mean()

    def cross_entropy(hidden, head, data):
        x = hidden @ head.T
        lse = torch.logsumexp(x, -1)
        return torch.where(data >= 0, lse - x.gather(-1, data.clamp(min=0).unsqueeze(-1))[..., 0], torch.zeros_like(lse)), lse

    return rotary, attention, kl, cross_entropy


def own_ops(plan):
    return (lambda q, k, at: skl.rotary(q, k, plan, at),
            lambda q, k, v, lam: skl.differential_attention(q, k, v, lam, causal=True),
            lambda *t: skl.attention_kl(*t, causal=True),
            lambda hidden, head, data: skl.vocab_cross_entropy(hidden, head, data, return_lse=True))


def make(seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    student = [r(B, 2 * H, N, D), r(B, H, N, D), r(B, H, N, D), r(V, H * D) / 4]
    teacher = [(r(B, H, N, D) * 0.3 + student[0][:, 0::2]).to(torch.bfloat16), (r(B, H, N, D) * 0.3 + student[1]).to(torch.bfloat16)]
    student = [t.to(torch.bfloat16) for t in student]
    student.insert(3, r(H, 1))
    data = torch.randint(0, V, (B, N), generator=gen, device="cuda")
    data[torch.rand(B, N, generator=gen, device="cuda") < 0.2] = -1
    at = torch.randint(0, 5000, (B, 1), generator=gen, device="cuda") + torch.arange(N, device="cuda")
    return student, teacher, at, data


def test_step_and_its_gradients():
    """Against the same step in 64 bits.  With h = 2^-8: q, k, and O are rounded to bf16 where they pass between operators (twice
    each for q and k, as given and as turned); an attention logit s is off by at most h |s| for each of the two turned factors,
    h |s| / sqrt(3) each as a root of squares, a vocabulary's logit x by h |x| / sqrt(3) for O's rounding and by as much for the
    weights' and lam's path into O; a probability changes by its logit's error, and the gradients' terms each through their logit
    and through the sum: 2 * 2 h (S + X) / sqrt(3), with S^2 and X^2 the means of s^2 and x^2 under the probabilities.  Each
    gradient is held to that share of its norm plus 1e-2 for the at most four later roundings to bf16 (d, dO, P or dS, the
    result: 4 h / sqrt(3) < 1e-2)."""
    build.build()
    plan = skl.rotary_plan(48, scaling="parts", factor=4.0, trained_length=1024)
    student, teacher, at, data = make()
    leaves = [t.clone().requires_grad_() for t in student]
    turned = skl.rotary_fwd(*teacher, plan, at)
    loss = step(*leaves, *turned, at, data, own_ops(plan))
    loss.backward()
    ref = [t.double().requires_grad_() for t in student]
    ops = plain_ops(plan)
    rloss = step(*ref, *(t.double() for t in turned), at, data, ops)
    rloss.backward()
    with torch.no_grad():
        q, k = ops[0](ref[0], ref[1], at)
        s = torch.where(torch.ones(N, N, dtype=torch.bool, device="cuda").tril(), q @ k.repeat_interleave(2, 1).transpose(2, 3) / 8, 0.0)
        p = torch.softmax(torch.where(s == 0, -1e300, s), -1)
        S = float((p * s * s).sum(-1).mean().sqrt())
        x = ops[1](q, k, ref[2], ref[3].sigmoid()).transpose(1, 2).reshape(B, N, H * D) @ ref[4].T
        X = float((torch.softmax(x, -1) * x * x).sum(-1).mean().sqrt())
    tol = 1e-2 + 4 * 2.0 ** -8 * (S + X) / math.sqrt(3)
    assert tol < 0.1
    assert abs(float(loss.detach()) - float(rloss.detach())) < 2e-2
    for t, r, name in zip(leaves, ref, ("q", "k", "v", "mix", "head")):
        err = float((t.grad.double() - r.grad).norm() / r.grad.norm())
        assert err < tol, f"{name}: {err:.2e} of {tol:.2e}"
    assert skl.check_device_status() == 0


def test_step_captured_into_a_graph():
    """Forward and backward of the whole step, replayed on new values, give the eager step's gradients."""
    build.build()
    plan = skl.rotary_plan(64)
    ops = own_ops(plan)
    student, teacher, at, data = make(1)
    leaves = [t.clone().requires_grad_() for t in student]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(step(*leaves, *teacher, at, data, ops), leaves)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = torch.autograd.grad(step(*leaves, *teacher, at, data, ops), leaves)
    new, _, far, more = make(2)
    with torch.no_grad():
        for t, x in zip((*leaves, at, data), (*new, far, more)):
            t.copy_(x)
    graph.replay()
    eager = [t.clone().requires_grad_() for t in new]
    for g, e in zip(grads, torch.autograd.grad(step(*eager, *teacher, at, data, ops), eager)):
        err = float((g.double() - e.double()).norm() / e.double().norm())
        assert err < 1e-2
    assert skl.check_device_status() == 0


def test_decoding_a_token_at_a_time_gives_the_whole_sequence():
    """Keys turned straight into a cache, then one token's queries after another over what the cache holds, against the
    causal call over all of them: the same weights in another order of sums, each result rounded once: 2 h of the values' sizes."""
    build.build()
    plan = skl.rotary_plan(64)
    student, _, _, _ = make(3)
    q, k, v, mix, _ = student
    lam = mix.sigmoid()
    start = 1000
    whole_q, whole_k = skl.rotary_fwd(q, k, plan, offset=start)
    whole, _ = skl.diff_attn_fwd(whole_q, whole_k, v, lam, causal=True)
    cache_k, cache_v = (torch.full((B, H, 256, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    for n in range(0, N, 7):
        rows = slice(max(0, n - 6), n + 1)
        cache_v[:, :, rows] = v[:, :, rows]
        for m in range(rows.start, n + 1):
            skl.rotary_fwd(None, k[:, :, m:m + 1], plan, offset=start + m, out=(None, cache_k[:, :, m:m + 1]))
        one, _ = skl.rotary_fwd(q[:, :, n:n + 1], None, plan, offset=start + n)
        lens = torch.full((B,), n + 1, dtype=torch.int32, device="cuda")
        d, _ = skl.diff_attn_fwd(one, cache_k, cache_v, lam, k_lens=lens)
        assert torch.equal(cache_k[:, :, :n + 1], whole_k[:, :, :n + 1])
        size = v[:, :, :n + 1].float().abs().amax() * (1 + lam.amax())
        assert float((d[:, :, 0].float() - whole[:, :, n].float()).abs().max()) <= 4 * 2.0 ** -8 * float(size)
