"""The operators together, as a distillation step uses them: the student's attention, the KL of its attention to the
teacher's on the same Q and K, and the output layer's terms on the teacher's alternatives, with all gradients."""
import math

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import build

pytestmark = pytest.mark.gpu


def step(q, k, v, head, tq, tk, tv, thead, data, ops, alternatives=None):
    """Loss = KL of the attentions + cross entropy on the data's tokens + KL to the teacher on its four alternatives
    (or the given ones); also those and the student's logits."""
    attention, attention_kl, token_logprobs = ops
    flat = lambda o: o.transpose(1, 2).reshape(*data.shape, -1)  # noqa: E731
    with torch.no_grad():
        t_logits = flat(attention(tq, tk, tv)) @ thead
        if alternatives is None:
            _, _, t_logp, alternatives = token_logprobs(t_logits, data, 4)
        else:
            t_logp = token_logprobs(t_logits, alternatives, 1)[0]
    x = flat(attention(q, k, v)) @ head
    tokens = torch.cat([data.unsqueeze(-1), alternatives], -1)
    logp, entropy, _, _ = token_logprobs(x, tokens, 1)
    soft = (t_logp.exp() * (t_logp - logp[..., 1:])).sum(-1).mean()
    return attention_kl(tq, tk, q, k) - logp[..., 0].mean() + soft - 0.01 * entropy.mean(), alternatives, x.detach()


def plain_ops():
    def probs(q, k):
        k = k.repeat_interleave(q.shape[1] // k.shape[1], 1)
        s = q @ k.transpose(2, 3) / math.sqrt(q.shape[-1])
        n, m = s.shape[-2:]
        see = torch.ones(n, m, dtype=torch.bool, device=s.device).tril(m - n)
        return torch.log_softmax(torch.where(see, s, torch.full_like(s, -1e300)), -1), see

    def attention(q, k, v):
        return probs(q, k)[0].exp() @ v.repeat_interleave(q.shape[1] // v.shape[1], 1)

    def attention_kl(q1, k1, q2, k2):
        (a, see), (b, _) = probs(q1, k1), probs(q2, k2)
        return torch.where(see, a.exp() * (a - b), torch.zeros_like(a)).sum(-1).mean()

    def token_logprobs(x, tokens, top_k):
        lp = torch.log_softmax(x, -1)
        tokens = tokens if tokens.dim() == x.dim() else tokens.unsqueeze(-1)
        top = lp.topk(top_k, -1)
        return lp.gather(-1, tokens), -(lp.exp() * lp).sum(-1), top.values, top.indices

    return attention, attention_kl, token_logprobs


def own_ops():
    return (lambda q, k, v: skl.attention(q, k, v, causal=True),
            lambda *t: skl.attention_kl(*t, causal=True),
            lambda x, t, top_k: skl.token_logprobs(x, t, top_k=top_k))


def make(seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    B, H, N, D, V = 2, 4, 200, 64, 1003
    student = [r(B, H, N, D), r(B, H, N, D), r(B, H, N, D), r(H * D, V) / 4]
    teacher = [(x + 0.3 * r(*x.shape)) for x in student]
    student, teacher = ([t.to(torch.bfloat16) for t in x] for x in (student, teacher))
    return student, teacher, torch.randint(0, V, (B, N), generator=gen, device="cuda")


def test_step_and_its_gradients():
    """Against the same step in 64 bits on the same alternatives (which of two near-equal logits comes first is not a
    rounding error).  With h = 2^-8, a logit x that is rounded to bf16 is off by at most h |x|, h |x| / sqrt(3) as a root
    of squares, and the O it is made of by as much again; its probability changes by that factor, and so do the
    gradient's terms p_j, each through x_j and through the sum: 2 * 2 h X / sqrt(3) in all, with X^2 the mean of x^2 under
    the probabilities.  Each gradient is held to that share of its norm plus 1e-2, the tolerance of the KL gradients, for
    the at most four later roundings to bf16 (dlogits, dO, P or dS, the result: 4 h / sqrt(3) < 1e-2)."""
    build.build()
    student, teacher, data = make()
    leaves = [t.clone().requires_grad_() for t in student]
    loss, alternatives, _ = step(*leaves, *teacher, data, own_ops())
    loss.backward()
    ref = [t.double().requires_grad_() for t in student]
    rloss, _, x = step(*ref, *(t.double() for t in teacher), data, plain_ops(), alternatives)
    rloss.backward()
    X = float((torch.softmax(x, -1) * x * x).sum(-1).mean().sqrt())
    tol = 1e-2 + 4 * 2.0 ** -8 * X / math.sqrt(3)
    assert tol < 0.1
    assert abs(float(loss) - float(rloss)) < 2e-2
    for t, r, name in zip(leaves, ref, ("q", "k", "v", "head")):
        err = float((t.grad.double() - r.grad).norm() / r.grad.norm())
        assert err < tol, f"{name}: {err:.2e} of {tol:.2e}"


def test_step_captured_into_a_graph():
    """Forward and backward of the whole step, replayed on new values, give the eager step's gradients."""
    build.build()
    student, teacher, data = make(1)
    ops = own_ops()
    leaves = [t.clone().requires_grad_() for t in student]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(step(*leaves, *teacher, data, ops)[0], leaves)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = torch.autograd.grad(step(*leaves, *teacher, data, ops)[0], leaves)
    new, _, _ = make(2)
    with torch.no_grad():
        for t, x in zip(leaves, new):
            t.copy_(x)
    graph.replay()
    eager = [t.clone().requires_grad_() for t in new]
    for g, e in zip(grads, torch.autograd.grad(step(*eager, *teacher, data, ops)[0], eager)):
        err = float((g.double() - e.double()).norm() / e.double().norm())
        assert err < 1e-2
    assert skl.check_device_status() == 0
