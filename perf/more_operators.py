"""Timed cases of rotary positions, differential attention and the cross entropy over a vocabulary.

Each case is one call that a distillation run makes around its attention: queries and keys turned by their positions
before it, the difference of two softmax maps in its place, and the loss on the data's tokens from the last hidden
states, with the gradients of all three.  `run` makes the call, either through the framework (`own`) or in its plain
form in torch.
"""
import math

import torch

own = False

NEG_INF = float("-inf")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TRAINED = 4096  # positions that the unscaled rotary frequencies were trained for


# ------------------------------------------------------------------------------ cases

def _rotary(op, name, B, H, HK, N, D, dim, dtype, interleaved=False, scaling="none", factor=1.0, start=0, ragged=False,
            rows_first=False):
    """q is [B, H, N, D] and k [B, HK, N, D]; the first `dim` of D turn.  Positions count from `start`, or with `ragged`
    every sequence has its own."""
    return {"name": name, "op": op, "B": B, "H": H, "HK": HK, "N": N, "D": D, "dim": dim, "dtype": dtype,
            "interleaved": interleaved, "scaling": scaling, "factor": factor, "start": start, "ragged": ragged,
            "rows_first": rows_first}


def _diff(op, name, B, H, HK, NQ, NK, D, causal=False, padded=False, rows_first=False, by_head=False):
    """H differences: q is [B, 2 H, NQ, D], k and v are [B, HK, NK, D]; `padded` gives every sequence its own lengths,
    `rows_first` stores the tensors as [B, N, heads, D], `by_head` has one weight for all rows of a head."""
    return {"name": name, "op": op, "B": B, "H": H, "HK": HK, "NQ": NQ, "NK": NK, "D": D, "causal": causal,
            "padded": padded, "rows_first": rows_first, "by_head": by_head}


def _xent(op, name, R, C, V, dtype, scale=1.0, lse_grad=False):
    """Hidden states [R, C], the vocabulary's matrix [V, C], a token for each row (or none)."""
    return {"name": name, "op": op, "R": R, "C": C, "V": V, "dtype": dtype, "scale": scale, "lse_grad": lse_grad}


def listed():
    return [
        # a training step's queries and keys at the 4K context, four query heads to a key head
        _rotary("rotary_fwd", "rotary_4k", 2, 32, 8, 4096, 128, 128, "bf16"),
        # one new token for each of eight sequences, far into contexts that the scaling reaches: latency
        _rotary("rotary_fwd", "rotary_token", 8, 32, 8, 1, 128, 128, "bf16", scaling="parts", factor=32.0, start=120011,
                ragged=True),
        # the gradient for a padded batch of odd length, interleaved pairs, half of the head, 32 bits
        _rotary("rotary_bwd", "rotary_grad_odd", 4, 12, 4, 1001, 64, 32, "fp32", interleaved=True, scaling="base", factor=4.0,
                ragged=True, rows_first=True),
        # the student's attention of a training step at the 4K context: 32 query heads in pairs
        _diff("diff_fwd", "diff_4k_causal", 2, 16, 8, 4096, 4096, 128, causal=True),
        # one new token for each of eight sequences over a long cache
        _diff("diff_fwd", "diff_token_64k", 8, 16, 8, 1, 65536, 128),
        # a padded batch of odd lengths, stored rows first; some rows see no key
        _diff("diff_fwd", "diff_padded", 4, 8, 4, 1001, 777, 64, causal=True, padded=True, rows_first=True),
        # the training step's backward at the 4K context
        _diff("diff_bwd", "diff_grad_4k_causal", 2, 16, 8, 4096, 4096, 128, causal=True),
        # the gradients of a padded batch of odd lengths, one weight to a head
        _diff("diff_bwd", "diff_grad_padded", 4, 8, 4, 1001, 777, 64, causal=True, padded=True, by_head=True),
        # the output layer of a training step: every position of a batch
        _xent("xent_fwd", "xent_8k_rows", 8192, 4096, 131072, "bf16"),
        # a few rows scored: the vocabulary's matrix is read for little work
        _xent("xent_fwd", "xent_8_rows", 8, 4096, 131072, "bf16"),
        # the training step's gradients of the hidden states and of the matrix
        _xent("xent_bwd", "xent_grad_4k_rows", 4096, 2048, 131072, "bf16"),
        # odd sizes in fp16, a temperature of 2, the loss also reads the log-sum-exp
        _xent("xent_bwd", "xent_grad_odd", 333, 1000, 50021, "fp16", scale=0.5, lse_grad=True),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary_fwd", "rotary_bwd", "diff_fwd", "diff_fwd", "diff_bwd", "diff_bwd", "xent_fwd", "xent_fwd",
                     "xent_bwd", "xent_bwd"])
    if op.startswith("rotary"):
        HK, G, B = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 3, 8, 64])
        D = rng.choice([64, 64, 80, 96, 128, 128, 256])
        dim = D if rng.random() < 0.6 else rng.choice([d for d in (16, 20, 32, 48, 64, 96) if d < D])
        N = 1 if rng.random() < 0.3 else _log_uniform(rng, 1, 16384)
        N = max(1, min(N, 2 ** 28 // (B * HK * (G + 1) * D)))
        scaling = rng.choice(["none", "none", "positions", "base", "parts"])
        return _rotary(op, "", B, HK * G, HK, N, D, dim, rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.random() < 0.4,
                       scaling, 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                       rng.choice([0, 0, _log_uniform(rng, 1, 1 << 20)]), rng.random() < 0.4, rng.random() < 0.4)
    if op.startswith("diff"):
        HK, G, B = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 3, 4]), rng.choice([1, 1, 2, 3, 8])
        H, D = HK * G, rng.choice([64, 128])
        if op == "diff_fwd" and rng.random() < 0.4:
            NQ, NK = rng.choice([1, 1, 2, 4, 7, 16]), _log_uniform(rng, 1, 131072)
            causal = NQ > 1 and NK >= NQ
        else:
            lo, hi = (1, 16384) if op == "diff_fwd" else (2, 8192)  # with one key the maps have no gradient
            NQ = _log_uniform(rng, lo, hi)
            NK = NQ if rng.random() < 0.6 else _log_uniform(rng, lo, hi)
            causal = rng.random() < 0.6
        while B * H * NQ * NK > 2 ** 29:  # no more work than the listed ones at the 4K context
            if NQ > 1024:
                NQ, NK = (NQ + 1) // 2, (NK + 1) // 2
            elif B > 1:
                B -= 1
            elif HK > 1:
                HK, H = HK // 2, HK // 2 * G
            else:
                NK = (NK + 1) // 2
        return _diff(op, "", B, H, HK, NQ, NK, D, causal, rng.random() < 0.4, rng.random() < 0.4, rng.random() < 0.3)
    C, V = 8 * _log_uniform(rng, 8, 1024), _log_uniform(rng, 32, 200003)
    R = max(1, min(_log_uniform(rng, 1, 8192), (2 ** 42 if op == "xent_fwd" else 2 ** 40) // (C * V)))
    return _xent(op, "", R, C, V, rng.choice(["bf16", "bf16", "fp16"]), rng.choice([1.0, 1.0, 0.5, 1.25]),
                 op == "xent_bwd" and rng.random() < 0.5)


def _lengths(c):
    """(query lengths, key lengths) of the batch's sequences: the first is whole, the others ever shorter."""
    if not c["padded"]:
        return [c["NQ"]] * c["B"], [c["NK"]] * c["B"]
    cut = [b / (2.0 * c["B"]) for b in range(c["B"])]
    return [max(1, c["NQ"] - int(x * c["NQ"])) for x in cut], [max(1, c["NK"] - int(0.9 * x * c["NK"])) for x in cut]


# ------------------------------------------------------------------------------ rotary frequencies

def _frequencies(c):
    """(radians a position for each pair, in 64 bits; the factor on what is turned)."""
    dim, s, base = c["dim"], c["factor"], 10000.0
    if c["scaling"] == "base" and dim > 2:  # a larger base: the slowest pair slows down by the factor
        base *= s ** (dim / (dim - 2.0))
    f = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if c["scaling"] == "positions":  # positions in between
        f = [x / s for x in f]
    if c["scaling"] != "parts":
        return f, 1.0

    # by parts: pairs that turn 32 times or more within the trained length stay, those below one turn slow down by the
    # factor, a ramp between
    def pair_of(turns):
        return dim * math.log(TRAINED / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

    low, high = max(0, math.floor(pair_of(32.0))), min(dim - 1, math.ceil(pair_of(1.0)))
    ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 1e-3))) for i in range(dim // 2)]
    return [x * (1.0 - r) + x / s * r for x, r in zip(f, ramp)], 0.1 * math.log(s) + 1.0


# ------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*size, by=1.0, dtype=torch.float32):
        return torch.randn(*size, generator=gen, device="cuda", dtype=torch.float32).mul_(by).to(dtype)

    s = {"case": dict(case)}
    if case["op"].startswith("xent"):
        R, C, V, dtype = case["R"], case["C"], case["V"], TYPES[case["dtype"]]
        s["hidden"] = normal(R, C, dtype=dtype)
        s["weight"] = normal(V, C, by=2.5 / math.sqrt(C), dtype=dtype)
        s["tokens"] = torch.randint(0, V, (R,), generator=gen, device="cuda")
        if R > 1:
            s["tokens"][1:][torch.rand(R - 1, generator=gen, device="cuda") < 0.1] = -1  # no loss here
        if case["op"] == "xent_bwd":
            _, s["lse"] = _plain_xent_fwd(s)  # from the forward pass
            by = (1024.0 if case["dtype"] == "fp16" else 1.0) / R  # as half-precision training scales its loss
            s["g_loss"] = normal(R, by=0.2).add_(1.0).mul_(by)
            s["g_lse"] = s["lse"].mul(2e-2 * by) if case["lse_grad"] else None
        return s

    def heads(h, n, by=1.0, dtype=torch.bfloat16):
        D = case["D"]
        if case["rows_first"]:
            return normal(case["B"], n, h, D, by=by, dtype=dtype).transpose(1, 2)
        return normal(case["B"], h, n, D, by=by, dtype=dtype)

    if case["op"].startswith("rotary"):
        B, N = case["B"], case["N"]
        by, dtype = (0.02 if case["op"] == "rotary_bwd" else 1.5), TYPES[case["dtype"]]
        s["q"], s["k"] = heads(case["H"], N, by, dtype), heads(case["HK"], N, by, dtype)
        s["positions"] = None
        if case["ragged"]:  # every sequence counts from its own start
            first = torch.randint(0, max(1, case["start"] // 2) + 7, (B, 1), generator=gen, device="cuda")
            s["positions"] = case["start"] + first + torch.arange(N, device="cuda")
        if own:
            import attention_kl_divergence_streamkl_gb300 as skl
            s["plan"] = skl.rotary_plan(case["dim"], scaling=None if case["scaling"] == "none" else case["scaling"],
                                        factor=case["factor"], trained_length=TRAINED, device="cuda")
        else:
            f, s["amplitude"] = _frequencies(case)
            s["frequencies"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        return s

    B, H, HK, NQ, NK = (case[x] for x in ("B", "H", "HK", "NQ", "NK"))
    s["q"], s["k"], s["v"] = heads(2 * H, NQ, 1.5), heads(HK, NK), heads(HK, NK)
    if case["by_head"]:
        s["lam"] = normal(1, H, 1).sigmoid_().expand(B, H, NQ)
    else:
        s["lam"] = normal(B, H, NQ).sigmoid_()
    s["q_lens"] = s["k_lens"] = None
    if case["padded"]:
        s["q_lens"], s["k_lens"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in _lengths(case))
    if case["op"] == "diff_bwd":
        s["do"] = heads(H, NQ, 0.02)
        # from the forward pass: each map's own result in two parts, and the log-sum-exps
        o, s["lse"] = _plain_maps(s)
        s["maps"] = o.to(torch.bfloat16)
        s["rest"] = (o - s["maps"].float()).to(torch.bfloat16)
        if case["rows_first"]:
            s["maps"], s["rest"] = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (s["maps"], s["rest"]))
    return s


# ------------------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        import attention_kl_divergence_streamkl_gb300 as skl
        if c["op"].startswith("rotary"):
            f = skl.rotary_fwd if c["op"] == "rotary_fwd" else skl.rotary_bwd
            return f(s["q"], s["k"], s["plan"], positions=s["positions"], offset=0 if c["ragged"] else c["start"],
                     interleaved=c["interleaved"])
        if c["op"] == "diff_fwd":
            return skl.diff_attn_fwd(s["q"], s["k"], s["v"], s["lam"], causal=c["causal"], q_lens=s["q_lens"],
                                     k_lens=s["k_lens"])
        if c["op"] == "diff_bwd":
            return skl.diff_attn_bwd(s["q"], s["k"], s["v"], s["lam"], s["maps"], s["lse"], s["do"], causal=c["causal"],
                                     q_lens=s["q_lens"], k_lens=s["k_lens"], maps_rest=s["rest"])
        if c["op"] == "xent_fwd":
            return skl.vocab_xent_fwd(s["hidden"], s["weight"], s["tokens"], scale=c["scale"])
        return skl.vocab_xent_bwd(s["hidden"], s["weight"], s["tokens"], s["lse"], s["g_loss"], s["g_lse"],
                                  scale=c["scale"])
    if c["op"].startswith("rotary"):
        return _plain_rotary(s)
    if c["op"] == "diff_fwd":
        o, lse = _plain_maps(s)
        return (o[:, 0::2] - s["lam"].unsqueeze(-1) * o[:, 1::2]).to(torch.bfloat16), lse
    if c["op"] == "diff_bwd":
        return _plain_diff_bwd(s)
    return _plain_xent_fwd(s) if c["op"] == "xent_fwd" else _plain_xent_bwd(s)


def _pairs_of(x, dim, interleaved):
    """The two parts of the pairs that turn, as views of x."""
    return (x[..., 0:dim:2], x[..., 1:dim:2]) if interleaved else (x[..., :dim // 2], x[..., dim // 2:dim])


def _plain_rotary(s):
    c = s["case"]
    at = s["positions"] if c["ragged"] else c["start"] + torch.arange(c["N"], device="cuda")
    angle = at.double().unsqueeze(-1) * s["frequencies"]  # far positions: 64 bits
    shape = (-1, 1, c["N"], c["dim"] // 2)
    cos, sin = angle.cos().float().view(shape) * s["amplitude"], angle.sin().float().view(shape) * s["amplitude"]
    if c["op"] == "rotary_bwd":
        sin = -sin
    out = []
    for x in (s["q"], s["k"]):
        y = x.float()
        a, b = _pairs_of(y, c["dim"], c["interleaved"])
        turned = y.clone()
        ta, tb = _pairs_of(turned, c["dim"], c["interleaved"])
        ta.copy_(a * cos - b * sin)
        tb.copy_(b * cos + a * sin)
        out.append(turned.to(x.dtype))
    return tuple(out)


def _hidden(s):
    """True where a query may not see a key, [B, 1, NQ, NK] (B = 1 where every sequence has the same lengths);
    None where every query sees every key."""
    c = s["case"]
    if not c["causal"] and not c["padded"]:
        return None
    i = torch.arange(c["NQ"], device="cuda").view(1, 1, -1, 1)
    j = torch.arange(c["NK"], device="cuda").view(1, 1, 1, -1)
    if not c["padded"]:
        return j > i + (c["NK"] - c["NQ"])
    ql, kl = s["q_lens"].view(-1, 1, 1, 1), s["k_lens"].view(-1, 1, 1, 1)
    out = (i >= ql) | (j >= kl)
    return out | (j > i + (kl - ql)) if c["causal"] else out


def _grouped(x, hk):
    """[B, heads, N, D] in 32 bits as [B, HK, heads / HK * N, D]: the query heads of a key head, one after the other."""
    b, h, n, d = x.shape
    return x.float().reshape(b, hk, h // hk * n, d)


def _logits(s):
    """(the scaled and masked logits of all maps as [B, 2 H, NQ, NK], the grouped queries and the keys in 32 bits)."""
    c = s["case"]
    q, k = _grouped(s["q"], c["HK"]), s["k"].float()
    x = torch.matmul(q, k.transpose(2, 3)).view(c["B"], 2 * c["H"], c["NQ"], c["NK"]).mul_(1.0 / math.sqrt(c["D"]))
    hidden = _hidden(s)
    if hidden is not None:
        x.masked_fill_(hidden, NEG_INF)
    return x, q, k


def _plain_maps(s):
    """Each map's own result and log-sum-exp, in 32 bits."""
    c = s["case"]
    x, _, _ = _logits(s)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == NEG_INF, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log()).squeeze(-1)  # -inf where a row sees no key
    pv = torch.matmul(p.view(c["B"], c["HK"], -1, c["NK"]), s["v"].float()).view(c["B"], 2 * c["H"], c["NQ"], c["D"])
    return pv / torch.where(l == 0, torch.ones_like(l), l), lse


def _plain_diff_bwd(s):
    c = s["case"]
    shape = (c["B"], c["HK"], -1, c["NK"])
    x, q, k = _logits(s)
    lse = torch.where(s["lse"] == NEG_INF, torch.zeros_like(s["lse"]), s["lse"]).unsqueeze(-1)
    p = x.sub_(lse).exp_()
    do, v = s["do"].float(), s["v"].float()
    # what reaches each map: do, and -lam do
    each = torch.stack((do, -s["lam"].unsqueeze(-1) * do), 2).view(c["B"], c["HK"], -1, c["D"])
    dv = torch.matmul(p.view(shape).transpose(2, 3), each)
    dp = torch.matmul(each, v.transpose(2, 3)).view(p.shape)
    delta = (p * dp).sum(-1, keepdim=True)
    ds = dp.sub_(delta).mul_(p).mul_(1.0 / math.sqrt(c["D"])).view(shape)
    dq = torch.matmul(ds, k).view(c["B"], 2 * c["H"], c["NQ"], c["D"])
    dk = torch.matmul(ds.transpose(2, 3), q)
    second = torch.matmul(p.view(shape), v).view(c["B"], c["H"], 2, c["NQ"], c["D"])[:, :, 1]
    return dq.to(torch.bfloat16), dk.to(torch.bfloat16), dv.to(torch.bfloat16), -(do * second).sum(-1)


def _plain_xent_fwd(s):
    x = torch.matmul(s["hidden"].float(), s["weight"].float().T).mul_(s["case"]["scale"])
    m = x.amax(-1, keepdim=True)
    given = x.gather(1, s["tokens"].clamp(min=0).unsqueeze(1))
    log_sum = x.sub_(m).exp_().sum(-1, keepdim=True).log()
    loss = (m - given + log_sum).squeeze(1)
    return torch.where(s["tokens"] >= 0, loss, torch.zeros_like(loss)), (m + log_sum).squeeze(1)


def _plain_xent_bwd(s):
    c = s["case"]
    hidden, weight = s["hidden"].float(), s["weight"].float()
    d = torch.matmul(hidden, weight.T).mul_(c["scale"]).sub_(s["lse"].unsqueeze(1)).exp_()
    g = torch.where(s["tokens"] >= 0, s["g_loss"], torch.zeros_like(s["g_loss"]))
    d.mul_((g if s["g_lse"] is None else g + s["g_lse"]).unsqueeze(1))
    d.scatter_add_(1, s["tokens"].clamp(min=0).unsqueeze(1), -g.unsqueeze(1))
    d.mul_(c["scale"])
    dtype = s["hidden"].dtype
    return torch.matmul(d, weight).to(dtype), torch.matmul(d.T, hidden).to(dtype)


# ------------------------------------------------------------------------------ what a pass cannot do without

def _seen_pairs(c):
    """Query-key pairs that some mask leaves, over the batch, for one head."""
    total = 0
    for ql, kl in zip(*_lengths(c)):
        if not c["causal"]:
            total += ql * kl
        else:
            off = kl - ql  # row i keeps keys 0 .. i + off
            first = max(0, -off)
            n = ql - first
            total += n * (first + off + 1) + n * (n - 1) // 2
    return total


def work(case):
    if case["op"].startswith("rotary"):
        B, N, values = case["B"], case["N"], case["B"] * case["N"] * (case["H"] + case["HK"])
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 2 * size * values * case["D"] + (8 * B * N if case["ragged"] else 0) + 4 * case["dim"],
                "flops": 3 * values * case["dim"]}
    if case["op"].startswith("xent"):
        R, C, V = case["R"], case["C"], case["V"]
        if case["op"] == "xent_fwd":
            return {"bytes": 2 * C * (R + V) + 16 * R, "flops": 2 * R * C * V}
        return {"bytes": 4 * C * (R + V) + (20 if case["lse_grad"] else 16) * R, "flops": 6 * R * C * V}
    qn, kn = (sum(x) for x in _lengths(case))
    H, D = case["H"], case["D"]
    o, k = 2 * H * D * qn, 2 * case["HK"] * D * kn  # q is twice o
    lam, pairs = (4 * H if case["by_head"] else 4 * H * qn), 2 * H * _seen_pairs(case)
    if case["op"] == "diff_fwd":
        return {"bytes": 3 * o + 2 * k + lam + 8 * H * qn, "flops": 4 * D * pairs}
    # dP is the same product for both maps; q, dq, the second map's result in two parts, do
    return {"bytes": 7 * o + 4 * k + lam + 12 * H * qn, "flops": 9 * D * pairs}


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rotary"):
        return _exact_rotary(case, s)
    return _exact_xent(case, s) if case["op"].startswith("xent") else _exact_diff(case, s)


def _exact_rotary(c, s):
    """Pairs as complex numbers, turned by exp(i position frequency)."""
    f, amplitude = _frequencies(c)
    at = s["positions"] if c["ragged"] else torch.arange(c["start"], c["start"] + c["N"], device="cuda").expand(c["B"], -1)
    angle = at.double()[:, None, :, None] * torch.tensor(f, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, amplitude), -angle if c["op"] == "rotary_bwd" else angle)
    out = []
    for x in (s["q"], s["k"]):
        z, half = x.double(), c["dim"] // 2
        part = z[..., :c["dim"]]
        pairs = part.unflatten(-1, (half, 2)) if c["interleaved"] else part.unflatten(-1, (2, half)).transpose(-1, -2)
        pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        turned = (pairs if c["interleaved"] else pairs.transpose(-1, -2)).flatten(-2)
        out.append(torch.cat((turned, z[..., c["dim"]:]), -1))
    return tuple(out)


def _exact_diff(c, s):
    """Sequence by sequence and key head by key head, over the rows and keys that a sequence has."""
    if 2 * c["B"] * c["H"] * c["NQ"] * c["NK"] * c["D"] * (4 if c["op"] == "diff_fwd" else 10) > 6e12:
        return None
    G, D, NQ, NK = c["H"] // c["HK"], c["D"], c["NQ"], c["NK"]
    f64 = dict(dtype=torch.float64, device="cuda")
    o, dq = torch.zeros(c["B"], c["H"], NQ, D, **f64), torch.zeros(c["B"], 2 * c["H"], NQ, D, **f64)
    dk, dv = (torch.zeros(c["B"], c["HK"], NK, D, **f64) for _ in range(2))
    lse, dlam = torch.full((c["B"], 2 * c["H"], NQ), NEG_INF, **f64), torch.zeros(c["B"], c["H"], NQ, **f64)
    for b, (ql, kl) in enumerate(zip(*_lengths(c))):
        first = max(0, ql - kl) if c["causal"] else 0  # the rows before see no key
        if first >= ql:
            continue
        seen = torch.ones(ql - first, kl, dtype=torch.bool, device="cuda").tril(first + kl - ql) if c["causal"] else None
        for h in range(c["HK"]):
            group, maps = slice(h * G, (h + 1) * G), slice(2 * h * G, 2 * (h + 1) * G)
            q, k, v = s["q"][b, maps, first:ql].double(), s["k"][b, h, :kl].double(), s["v"][b, h, :kl].double()
            x = (q @ k.T) / math.sqrt(D)
            if seen is not None:
                x = torch.where(seen, x, torch.full((), NEG_INF, **f64))
            lse[b, maps, first:ql] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1)
            del x
            lam = s["lam"][b, group, first:ql, None].double()
            if c["op"] == "diff_fwd":
                o[b, group, first:ql] = (p[0::2] - lam * p[1::2]) @ v
                continue
            do = s["do"][b, group, first:ql].double()
            pull = do @ v.T  # the gradient of the difference of the maps
            dv[b, h, :kl] = torch.einsum("gij,gid->jd", p[0::2] - lam * p[1::2], do)
            dlam[b, group, first:ql] = -(p[1::2] * pull).sum(-1)
            for t in range(2):
                weight = p[t::2] if t == 0 else -lam * p[t::2]
                ds = weight * (pull - (p[t::2] * pull).sum(-1, keepdim=True))
                dq[b, 2 * h * G + t:2 * (h + 1) * G:2, first:ql] = (ds @ k) / math.sqrt(D)
                dk[b, h, :kl] += torch.einsum("gij,gid->jd", ds, q[t::2]) / math.sqrt(D)
    return (o, lse) if c["op"] == "diff_fwd" else (dq, dk, dv, dlam)


def _exact_xent(c, s):
    """A block of rows at a time."""
    if c["R"] * c["C"] * c["V"] * (2 if c["op"] == "xent_fwd" else 6) > 1.2e13:
        return None
    weight = s["weight"].double()
    loss, lse, dhidden, dweight = [], [], [], torch.zeros_like(weight) if c["op"] == "xent_bwd" else None
    step = max(1, 2 ** 28 // c["V"])
    for r in range(0, c["R"], step):
        hidden, tokens = s["hidden"][r:r + step].double(), s["tokens"][r:r + step]
        x = c["scale"] * (hidden @ weight.T)
        z = torch.logsumexp(x, -1)
        there = tokens >= 0
        picked = torch.nn.functional.one_hot(tokens.clamp(min=0), c["V"]) * there[:, None] if c["op"] == "xent_bwd" else None
        if picked is None:
            lse.append(z)
            loss.append(torch.where(there, z - x.gather(1, tokens.clamp(min=0)[:, None])[:, 0], torch.zeros_like(z)))
            continue
        p = torch.softmax(x, -1)
        d = s["g_loss"][r:r + step].double()[:, None] * (p * there[:, None] - picked)
        if s["g_lse"] is not None:
            d += s["g_lse"][r:r + step].double()[:, None] * p
        d *= c["scale"]
        dhidden.append(d @ weight)
        dweight += d.T @ hidden
    if c["op"] == "xent_fwd":
        return torch.cat(loss), torch.cat(lse)
    return torch.cat(dhidden), dweight
