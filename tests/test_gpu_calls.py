"""The native caller and the step-by-step path give the same tensors, bit for bit, and the same refusals."""
import threading

import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import _lib, build
from tests import attn_util as A

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    yield
    assert skl.check_device_status() == 0


class Nothing:
    """A native caller that takes nothing."""
    def __getattr__(self, name):
        return lambda *a: None


def both(monkeypatch, f):
    native, taken = _lib.calls(), []

    class Seen:
        def __getattr__(self, name):
            def call(*a):
                got = getattr(native, name)(*a)
                taken.append(got is not None)
                return got
            return call

    monkeypatch.setattr(_lib, "_calls", Seen())
    a = f()
    monkeypatch.setattr(_lib, "_calls", Nothing())
    b = f()
    monkeypatch.setattr(_lib, "_calls", native)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride() and x.device == y.device
        assert torch.equal(x.reshape(-1).view(torch.uint8), y.reshape(-1).view(torch.uint8))  # NaN too
    return taken


def lens(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rows_first", [False, True])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("H,HK,NQ,NK,D", [(1, 1, 1, 1, 64), (4, 2, 130, 200, 128), (8, 1, 3, 2000, 64)])
def test_attention(monkeypatch, H, HK, NQ, NK, D, given, rows_first):
    q, k, v, do = A.tensors(2, H, HK, NQ, NK, D, 1, rows_first)
    kw = dict(scale=0.3, causal=True, q_lens=lens(NQ, max(NQ - 1, 0)), k_lens=lens(NK // 2 + 1, NK)) if given else {}
    assert both(monkeypatch, lambda: skl.attn_fwd(q, k, v, **kw)) == [True]
    o, lse = skl.attn_fwd(q, k, v, **kw)
    dlse = torch.randn_like(lse) if given else None
    assert both(monkeypatch, lambda: skl.attn_bwd(q, k, v, o, lse, do, dlse, bwd_mode=skl.BWD_SEPARATE, **kw)) == [True]


@pytest.mark.parametrize("dtype", [BF, torch.float16, torch.float32])
@pytest.mark.parametrize("lead,T", [((5,), None), ((2, 3), 7), ((), 2), ((4,), 1)])
@pytest.mark.parametrize("top_k", [0, 5])
def test_logprobs(monkeypatch, lead, T, dtype, top_k):
    x = torch.randn(*lead, 1003, device="cuda").to(dtype)
    tok = torch.randint(-1, 1003, lead if T is None else (*lead, T), device="cuda")
    assert both(monkeypatch, lambda: skl.logprobs_fwd(x, tok, 0.7, top_k)) == [True]
    lp, ent, lse, _, _ = skl.logprobs_fwd(x, tok, 0.7, top_k)
    g, gh = torch.randn_like(lp), torch.randn_like(ent)
    assert both(monkeypatch, lambda: [skl.logprobs_bwd(x, tok, lse, ent, g, gh, 0.7)]) == [True]
    assert both(monkeypatch, lambda: [skl.logprobs_bwd(x, tok, lse, None, g, None, 0.7)]) == [True]


def test_what_the_library_does_not_read_in_place_is_copied(monkeypatch):
    q, k, v, do = A.tensors(1, 2, 2, 70, 90, 64, 2)
    odd = torch.empty(q.numel() + 1, dtype=BF, device="cuda")[1:].view(q.shape).copy_(q)  # starts off a 16-byte boundary
    for args in ((odd, k, v), (q, k.expand(1, 2, 90, 64).transpose(2, 3).contiguous().transpose(2, 3), v)):
        assert both(monkeypatch, lambda: skl.attn_fwd(*args)) == [False]
    x = torch.randn(3, 4, 200, device="cuda")[:, ::2]
    tok = torch.randint(0, 200, (3, 2), device="cuda")
    assert both(monkeypatch, lambda: skl.logprobs_fwd(x, tok)) == [False]
    assert both(monkeypatch, lambda: skl.logprobs_fwd(x[0], tok[0].int())) == [False]
    wide = torch.randn(6, 300, device="cuda")[:, :200]  # rows behind one another with a gap: read in place
    assert both(monkeypatch, lambda: skl.logprobs_fwd(wide, torch.zeros(6, dtype=torch.int64, device="cuda"))) == [True]


@pytest.mark.parametrize("call", [
    lambda q, x, t: skl.attn_fwd(q, q, q.float()), lambda q, x, t: skl.attn_fwd(q, q[..., :32], q),
    lambda q, x, t: skl.attn_fwd(q, q[:, :0], q[:, :0]), lambda q, x, t: skl.attn_fwd(q[..., :48], q[..., :48], q[..., :48]),
    lambda q, x, t: skl.attn_fwd(q, q, q, float("inf")), lambda q, x, t: skl.attn_fwd(q, q, q, float("nan")),
    lambda q, x, t: skl.attn_fwd(q, q, q, q_lens=t), lambda q, x, t: skl.attn_fwd(q, q, q, k_lens=t.int()[:0]),
    lambda q, x, t: skl.attn_bwd(q, q, q, q, x[:, 0], q),
    lambda q, x, t: skl.attn_bwd(q, q, q, q, q[..., 0].float().contiguous(), q, bwd_mode=99),
    lambda q, x, t: skl.logprobs_fwd(x.double(), t), lambda q, x, t: skl.logprobs_fwd(x, t[:2]),
    lambda q, x, t: skl.logprobs_fwd(x, t, 0.0), lambda q, x, t: skl.logprobs_fwd(x, t, 1.0, 33),
    lambda q, x, t: skl.logprobs_fwd(x, t, 1.0, -1), lambda q, x, t: skl.logprobs_fwd(x, t.float()),
    lambda q, x, t: skl.logprobs_bwd(x, t, x[:2, 0], None, x[:, 0]), lambda q, x, t: skl.logprobs_bwd(x, t, x[:, 0], None, None)])
def test_refusals_are_the_same(monkeypatch, call):
    q = torch.zeros(1, 2, 8, 64, dtype=BF, device="cuda")
    x, t = torch.zeros(3, 50, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    raised = []
    for c in (_lib.calls(), Nothing()):
        monkeypatch.setattr(_lib, "_calls", c)
        with pytest.raises((ValueError, TypeError, skl.StreamKLError)) as e:
            call(q, x, t)
        raised.append((e.type, str(e.value)))
    assert raised[0] == raised[1]


def test_threads_on_their_own_streams():
    """Two threads call at once, each on its stream; every result is the single call's."""
    q, k, v, do = A.tensors(2, 4, 2, 300, 400, 128, 5)
    x = torch.randn(40, 5000, device="cuda").to(BF)
    tok = torch.randint(0, 5000, (40, 3), device="cuda")

    def one():
        o, lse = skl.attn_fwd(q, k, v, causal=True)
        grads = skl.attn_bwd(q, k, v, o, lse, do, causal=True, bwd_mode=skl.BWD_SEPARATE)
        return (o, lse, *grads, *skl.logprobs_fwd(x, tok, top_k=4))

    want, wrong = one(), []
    torch.cuda.synchronize()

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = one()
                torch.cuda.current_stream().synchronize()
                wrong.extend(i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b))

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
