"""Timed cases of the attention and token-log-probability operators.

Each case is one call that a distillation run makes next to the attention-KL
loss: the student's attention forward and backward, the attention of single
tokens over a long cache, and the log probabilities of given tokens with their
entropy, their top alternatives and their gradient.  `run` makes the call,
either through the framework (`own`) or in its plain form in torch.
"""
import math

import torch

own = False

NEG_INF = float("-inf")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------ cases

def _attn(op, name, B, H, HK, NQ, NK, D, causal=False, padded=False, rows_first=False, lse_grad=False):
    """q is [B, H, NQ, D], k and v are [B, HK, NK, D]; `padded` gives every sequence its own lengths and
    `rows_first` stores the tensors as [B, N, heads, D]."""
    return {"name": name, "op": op, "B": B, "H": H, "HK": HK, "NQ": NQ, "NK": NK, "D": D, "causal": causal,
            "padded": padded, "rows_first": rows_first, "lse_grad": lse_grad}


def _logp(op, name, R, V, dtype, T=1, top_k=0, scale=1.0, entropy_grad=False, hidden=0):
    """Logits [R, V], T given tokens for each row; the last `hidden` columns are -inf (a padded vocabulary)."""
    return {"name": name, "op": op, "R": R, "V": V, "dtype": dtype, "T": T, "top_k": top_k, "scale": scale,
            "entropy_grad": entropy_grad, "hidden": hidden}


def listed():
    return [
        # a long training sequence, four query heads to a key head
        _attn("attn_fwd", "fwd_16k_causal", 1, 32, 8, 16384, 16384, 128, causal=True),
        # one new token for each of eight sequences over a long cache
        _attn("attn_fwd", "fwd_token_128k", 8, 32, 8, 1, 131072, 128),
        # the smallest call: one token of one short sequence, where only latency counts
        _attn("attn_fwd", "fwd_token_short", 1, 8, 2, 1, 129, 64),
        # a padded batch of odd length, stored rows first
        _attn("attn_fwd", "fwd_padded", 4, 16, 4, 1001, 1001, 64, causal=True, padded=True, rows_first=True),
        # the training step's backward at the 4K context
        _attn("attn_bwd", "bwd_4k_causal", 2, 32, 8, 4096, 4096, 128, causal=True),
        # every query sees every key, a head for each key head
        _attn("attn_bwd", "bwd_8k_full", 1, 8, 8, 8192, 8192, 64),
        # a padded batch of odd lengths; some rows see no key; the loss also reads the log-sum-exp
        _attn("attn_bwd", "bwd_padded", 4, 12, 4, 1001, 777, 128, causal=True, padded=True, lse_grad=True),
        # the output layer of a training step: every position of a batch
        _logp("logp_fwd", "logp_8k_rows", 8192, 131072, "bf16", top_k=8),
        # a decode step: a few rows, so that one row has to fill the GPU
        _logp("logp_fwd", "logp_8_rows", 8, 131072, "bf16", top_k=20),
        # the teacher's alternatives scored by the student, an odd vocabulary in 32 bits, a temperature of 2
        _logp("logp_fwd", "logp_alternatives", 333, 50021, "fp32", T=16, top_k=16, scale=0.5, hidden=21),
        # the gradient of the mean negative log probability
        _logp("logp_bwd", "logp_grad_4k_rows", 4096, 131072, "bf16"),
        # the gradient of a loss on alternatives and on the entropy, an odd vocabulary in fp16
        _logp("logp_bwd", "logp_grad_alternatives", 333, 50021, "fp16", T=16, scale=0.5, entropy_grad=True,
              hidden=21),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "logp_fwd", "logp_bwd"])
    if op.startswith("attn"):
        HK, G, B = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 3, 8])
        H, D = HK * G, rng.choice([64, 128])
        if op == "attn_fwd" and rng.random() < 0.4:
            NQ, NK = rng.choice([1, 1, 2, 4, 7, 16]), _log_uniform(rng, 1, 131072)
            causal = NQ > 1 and NK >= NQ
        else:
            # backward: two keys at least, since with one every gradient of q and k is zero
            lo, hi = (1, 16384) if op == "attn_fwd" else (2, 8192)
            NQ = _log_uniform(rng, lo, hi)
            NK = NQ if rng.random() < 0.6 else _log_uniform(rng, lo, hi)
            causal = rng.random() < 0.6
        pairs = 2 ** 31 if op == "attn_fwd" else 2 ** 29  # no more work than the largest listed cases
        while B * H * NQ * NK > pairs:
            if NQ > 1024:
                NQ, NK = (NQ + 1) // 2, (NK + 1) // 2
            elif B > 1:
                B -= 1
            elif HK > 1:
                HK, H = HK // 2, HK // 2 * G
            else:
                NK = (NK + 1) // 2
        return _attn(op, "", B, H, HK, NQ, NK, D, causal, rng.random() < 0.4, rng.random() < 0.4,
                     op == "attn_bwd" and rng.random() < 0.4)
    V = _log_uniform(rng, 32, 200003)
    R = min(_log_uniform(rng, 1, 8192), (2 ** 30 if op == "logp_fwd" else 2 ** 29) // V)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if dtype == "fp32":
        R = (R + 1) // 2
    hidden = rng.choice([0, 0, 1, V // 7])
    return _logp(op, "", R, V, dtype, rng.choice([1, 1, 3, 16, 32]), 0 if op == "logp_bwd" else rng.choice([0, 1, 5, 20, 32]),
                 rng.choice([1.0, 1.0, 0.5, 1.25]), op == "logp_bwd" and rng.random() < 0.5, hidden)


def _lengths(c):
    """(query lengths, key lengths) of the batch's sequences: the first is whole, the others ever shorter."""
    if not c["padded"]:
        return [c["NQ"]] * c["B"], [c["NK"]] * c["B"]
    cut = [b / (2.0 * c["B"]) for b in range(c["B"])]
    return [max(1, c["NQ"] - int(x * c["NQ"])) for x in cut], [max(1, c["NK"] - int(0.9 * x * c["NK"])) for x in cut]


# ------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*size, by=1.0, dtype=torch.float32):
        return torch.randn(*size, generator=gen, device="cuda", dtype=torch.float32).mul_(by).to(dtype)

    s = {"case": dict(case)}
    if case["op"].startswith("attn"):
        B, H, HK, NQ, NK, D = (case[x] for x in ("B", "H", "HK", "NQ", "NK", "D"))

        def heads(h, n, by=1.0):
            if case["rows_first"]:
                return normal(B, n, h, D, by=by, dtype=torch.bfloat16).transpose(1, 2)
            return normal(B, h, n, D, by=by, dtype=torch.bfloat16)

        s["q"], s["k"], s["v"] = heads(H, NQ, 1.5), heads(HK, NK), heads(HK, NK)
        s["q_lens"] = s["k_lens"] = None
        if case["padded"]:
            s["q_lens"], s["k_lens"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in _lengths(case))
        if case["op"] == "attn_bwd":
            s["do"] = heads(H, NQ, 0.02)
            s["dlse"] = normal(B, H, NQ, by=0.01) if case["lse_grad"] else None
            s["o"], s["lse"] = _plain_attn_fwd(s)  # a training step has these from its forward pass
    else:
        R, V, T = case["R"], case["V"], case["T"]
        logits = normal(R, V, by=2.5)
        if case["hidden"]:
            logits[:, V - case["hidden"]:] = NEG_INF
        s["logits"] = logits.to(TYPES[case["dtype"]])
        s["tokens"] = torch.randint(0, V - case["hidden"], (R, T), generator=gen, device="cuda")
        if T > 1:
            s["tokens"][:, 1][torch.rand(R, generator=gen, device="cuda") < 0.25] = -1  # no token here
        if case["op"] == "logp_bwd":
            _, s["entropy"], s["lse"], _, _ = _plain_logp_fwd(s)  # from the forward pass
            loss_scale = 1024.0 if case["dtype"] == "fp16" else 1.0  # as half-precision training scales its loss
            s["g_logp"] = normal(R, T, by=0.2).sub_(1.0).mul_(loss_scale / R)
            s["g_entropy"] = normal(R, by=0.05).mul_(loss_scale / R) if case["entropy_grad"] else None
    return s


# ------------------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        import attention_kl_divergence_streamkl_gb300 as skl
        if c["op"] == "attn_fwd":
            return skl.attn_fwd(s["q"], s["k"], s["v"], causal=c["causal"], q_lens=s["q_lens"], k_lens=s["k_lens"])
        if c["op"] == "attn_bwd":
            return skl.attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], dlse=s["dlse"], causal=c["causal"],
                                q_lens=s["q_lens"], k_lens=s["k_lens"])
        if c["op"] == "logp_fwd":
            return skl.logprobs_fwd(s["logits"], s["tokens"], scale=c["scale"], top_k=c["top_k"])
        return skl.logprobs_bwd(s["logits"], s["tokens"], s["lse"], s["entropy"], s["g_logp"], s["g_entropy"],
                                scale=c["scale"])
    if c["op"] == "attn_fwd":
        return _plain_attn_fwd(s)
    if c["op"] == "attn_bwd":
        return _plain_attn_bwd(s)
    return _plain_logp_fwd(s) if c["op"] == "logp_fwd" else _plain_logp_bwd(s)


def _grouped(x, hk):
    """[B, H, N, D] in 32 bits as [B, HK, G * N, D]: the query heads of a key head, one after the other."""
    b, h, n, d = x.shape
    return x.float().reshape(b, hk, h // hk * n, d)


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


def _logits(s):
    """(the scaled and masked logits as [B, H, NQ, NK], the mask, the grouped queries and keys in 32 bits)."""
    c = s["case"]
    q, k = _grouped(s["q"], c["HK"]), s["k"].float()
    x = torch.matmul(q, k.transpose(2, 3)).view(c["B"], c["H"], c["NQ"], c["NK"]).mul_(1.0 / math.sqrt(c["D"]))
    hidden = _hidden(s)
    if hidden is not None:
        x.masked_fill_(hidden, NEG_INF)
    return x, hidden, q, k


def _plain_attn_fwd(s):
    c = s["case"]
    x, _, _, _ = _logits(s)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == NEG_INF, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log()).squeeze(-1)  # -inf where a row sees no key
    pv = torch.matmul(p.view(c["B"], c["HK"], -1, c["NK"]), s["v"].float()).view(c["B"], c["H"], c["NQ"], c["D"])
    return (pv / torch.where(l == 0, torch.ones_like(l), l)).to(torch.bfloat16), lse


def _plain_attn_bwd(s):
    c = s["case"]
    shape = (c["B"], c["HK"], -1, c["NK"])
    x, hidden, q, k = _logits(s)
    lse = torch.where(s["lse"] == NEG_INF, torch.zeros_like(s["lse"]), s["lse"]).unsqueeze(-1)
    p = x.sub_(lse).exp_()
    do, v = _grouped(s["do"], c["HK"]), s["v"].float()
    dv = torch.matmul(p.view(shape).transpose(2, 3), do)
    dp = torch.matmul(do, v.transpose(2, 3)).view(p.shape)
    delta = (p * dp).sum(-1, keepdim=True)
    if s["dlse"] is not None:
        delta = delta - s["dlse"].unsqueeze(-1)
    ds = dp.sub_(delta).mul_(p).mul_(1.0 / math.sqrt(c["D"])).view(shape)
    dq = torch.matmul(ds, k).view(c["B"], c["H"], c["NQ"], c["D"])
    dk = torch.matmul(ds.transpose(2, 3), q)
    return dq.to(torch.bfloat16), dk.to(torch.bfloat16), dv.to(torch.bfloat16)


def _plain_logp_fwd(s):
    c = s["case"]
    V, tokens = c["V"], s["tokens"]
    raw = s["logits"].float()
    x = raw * c["scale"]
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1)
    weighted = torch.where(e > 0, (x - m) * e, torch.zeros_like(e)).sum(-1)
    entropy = total.log().squeeze(-1) - weighted / total.squeeze(-1)
    there = tokens >= 0
    logp = torch.where(there, x.gather(1, tokens.clamp(min=0)) - lse.unsqueeze(-1), torch.zeros_like(lse).unsqueeze(-1))
    # the largest logits; equal ones go to the lowest index: the value's order above, the column's below
    bits = (raw + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()
    keys = (order << 32) | (V - 1 - torch.arange(V, device="cuda"))
    index = V - 1 - (keys.topk(c["top_k"], dim=-1).values & 0xFFFFFFFF)
    return logp, entropy, lse, x.gather(1, index) - lse.unsqueeze(-1), index


def _plain_logp_bwd(s):
    c = s["case"]
    tokens = s["tokens"]
    logp = s["logits"].float() * c["scale"] - s["lse"].unsqueeze(-1)
    p = logp.exp()
    g = torch.where(tokens >= 0, s["g_logp"], torch.zeros_like(s["g_logp"]))
    d = p * -g.sum(-1, keepdim=True)
    if s["g_entropy"] is not None:
        pull = torch.where(p > 0, logp + s["entropy"].unsqueeze(-1), torch.zeros_like(p))
        d -= s["g_entropy"].unsqueeze(-1) * p * pull
    d.scatter_add_(1, tokens.clamp(min=0), g)
    return (d * c["scale"]).to(s["logits"].dtype)


# ------------------------------------------------------------------------------ what a pass cannot do without

def _pairs(c):
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
    if case["op"].startswith("attn"):
        qn, kn = (sum(x) for x in _lengths(case))
        q, k, rows = 2 * case["H"] * case["D"] * qn, 2 * case["HK"] * case["D"] * kn, 4 * case["H"] * qn
        pairs = case["H"] * _pairs(case)
        if case["op"] == "attn_fwd":
            return {"bytes": 2 * q + 2 * k + rows, "flops": 4 * case["D"] * pairs}
        return {"bytes": 4 * q + 4 * k + rows * (2 if case["lse_grad"] else 1), "flops": 10 * case["D"] * pairs}
    R, V, T, K = case["R"], case["V"], case["T"], case["top_k"]
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "logp_fwd":
        return {"bytes": R * (V * size + 12 * T + 8 + 12 * K), "flops": 6 * R * V}
    return {"bytes": R * (2 * V * size + 12 * T + 12), "flops": 6 * R * V}


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attn(case, s) if case["op"].startswith("attn") else _exact_logp(case, s)


def _exact_attn(c, s):
    """Sequence by sequence and key head by key head, over the rows and keys that a sequence has."""
    if c["B"] * c["H"] * c["NQ"] * c["NK"] * c["D"] * (4 if c["op"] == "attn_fwd" else 10) > 6e12:
        return None
    G = c["H"] // c["HK"]
    f64 = dict(dtype=torch.float64, device="cuda")
    o, dq = (torch.zeros(c["B"], c["H"], c["NQ"], c["D"], **f64) for _ in range(2))
    dk, dv = (torch.zeros(c["B"], c["HK"], c["NK"], c["D"], **f64) for _ in range(2))
    lse = torch.full((c["B"], c["H"], c["NQ"]), NEG_INF, **f64)
    for b, (ql, kl) in enumerate(zip(*_lengths(c))):
        first = max(0, ql - kl) if c["causal"] else 0  # the rows before see no key
        seen = torch.ones(ql - first, kl, dtype=torch.bool, device="cuda").tril(first + kl - ql) if c["causal"] else None
        for h in range(c["HK"]):
            group = slice(h * G, (h + 1) * G)
            q, k, v = s["q"][b, group, first:ql].double(), s["k"][b, h, :kl].double(), s["v"][b, h, :kl].double()
            x = (q @ k.T) / math.sqrt(c["D"])
            if seen is not None:
                x = torch.where(seen, x, torch.full((), NEG_INF, **f64))
            z = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1)
            del x
            o[b, group, first:ql], lse[b, group, first:ql] = p @ v, z
            if c["op"] == "attn_bwd":
                do = s["do"][b, group, first:ql].double()
                # dp centred on its mean under p, which is do . o
                pull = do @ v.T - (do * o[b, group, first:ql]).sum(-1, keepdim=True)
                if s["dlse"] is not None:
                    pull += s["dlse"][b, group, first:ql].double().unsqueeze(-1)
                pull *= p
                dv[b, h, :kl] = torch.einsum("gij,gid->jd", p, do)
                dq[b, group, first:ql] = (pull @ k) / math.sqrt(c["D"])
                dk[b, h, :kl] = torch.einsum("gij,gid->jd", pull, q) / math.sqrt(c["D"])
    return (o, lse) if c["op"] == "attn_fwd" else (dq, dk, dv)


def _exact_logp(c, s):
    x = s["logits"].double() * c["scale"]
    lse = torch.logsumexp(x, -1)
    logq = x - lse[:, None]
    q = logq.exp()
    tokens = s["tokens"]
    here = (tokens >= 0).double()
    if c["op"] == "logp_fwd":
        logp = torch.gather(logq, 1, tokens.clamp(min=0)).mul(here)
        entropy = -torch.xlogy(q, q).sum(-1)
        top, index = torch.sort(s["logits"].double(), dim=-1, descending=True, stable=True)
        return logp, entropy, lse, top[:, :c["top_k"]] * c["scale"] - lse[:, None], index[:, :c["top_k"]]
    g = s["g_logp"].double() * here
    d = torch.zeros_like(q).scatter_add_(1, tokens.clamp(min=0), g) - q * g.sum(-1, keepdim=True)
    if s["g_entropy"] is not None:
        d -= s["g_entropy"].double()[:, None] * (torch.xlogy(q, q) - q * torch.xlogy(q, q).sum(-1, keepdim=True))
    return d * c["scale"]
