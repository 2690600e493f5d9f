"""Autograd entry point: the attention KL divergence as a differentiable loss.

``attention_kl(q1, k1, q2, k2)`` returns KL(P1 || P2) per query row (or its mean
or sum) with P_t = softmax(scale Q_t K_t^T).  The forward is streamkl_fwd; the
backward calls the recompute backward of the StreamKL technical summary
(gist.science/ja/paper/2606.20005, section 手法 2) in whichever settings the
inputs need: setting 1 (P1 held fixed) for gradients of Q2/K2, setting 2 (P2
held fixed) for gradients of Q1/K1, both when both sides require grad (in one
call, which rebuilds each logit tile pair once for both settings where that is
faster).  Only
the reduction of the per-row values to a scalar happens in PyTorch.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _lib


class _AttentionKL(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q1, k1, q2, k2, scale, causal, reduction, bwd_mode):
        kl, lse1, lse2 = _lib.fwd(q1, k1, q2, k2, scale, causal)
        ctx.save_for_backward(q1, k1, q2, k2, kl, lse1, lse2)
        ctx.scale, ctx.causal, ctx.reduction, ctx.bwd_mode = scale, causal, reduction, bwd_mode
        if reduction == "none":
            return kl
        return kl.sum() if reduction == "sum" else kl.mean()

    @staticmethod
    def backward(ctx, grad_out):
        q1, k1, q2, k2, kl, lse1, lse2 = ctx.saved_tensors
        if ctx.reduction == "none":
            g = grad_out.contiguous().float()
        else:
            w = 1.0 if ctx.reduction == "sum" else 1.0 / kl.numel()
            g = (grad_out.float() * w).expand_as(kl).contiguous()
        need1 = ctx.needs_input_grad[0] or ctx.needs_input_grad[1]
        need2 = ctx.needs_input_grad[2] or ctx.needs_input_grad[3]
        dq1 = dk1 = dq2 = dk2 = None
        if need1 and need2 and ctx.bwd_mode in (_lib.BWD_AUTO, _lib.BWD_FUSED, _lib.BWD_SEPARATE):
            # the mutual case in one call (the library picks one recompute for both settings, or a pass each)
            return (*_lib.bwd_mutual(q1, k1, q2, k2, lse1, lse2, kl, g, ctx.scale, ctx.causal, ctx.bwd_mode),
                    None, None, None, None)
        if need2:
            dq2, dk2 = _lib.bwd_s1(q1, k1, q2, k2, lse1, lse2, g, ctx.scale, ctx.causal, ctx.bwd_mode)
        if need1:
            dq1, dk1 = _lib.bwd_s2(q1, k1, q2, k2, lse1, lse2, kl, g, ctx.scale, ctx.causal, ctx.bwd_mode)
        return dq1, dk1, dq2, dk2, None, None, None, None


def attention_kl(q1, k1, q2, k2, scale=None, causal=False, reduction="mean", bwd_mode=_lib.BWD_AUTO):
    """KL(softmax(scale Q1 K1^T) || softmax(scale Q2 K2^T)) per row, reduced by `reduction`.

    q_t: [B, H, N_Q, D] and k_t: [B, H, N_K, D] bf16 CUDA tensors; reduction is
    "mean" (over all B*H*N_Q rows), "sum" or "none" (fp32 [B, H, N_Q]).
    """
    if reduction not in ("mean", "sum", "none"):
        raise ValueError("reduction must be 'mean', 'sum' or 'none'")
    return _AttentionKL.apply(q1, k1, q2, k2, scale, causal, reduction, bwd_mode)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, scale, causal, q_lens, k_lens, bwd_mode, train):
        # up to 64 keys the backward forms its row sums without o
        o, lse, *rest = _lib.attn_fwd(q, k, v, scale, causal, q_lens, k_lens, train and k.shape[2] > _lib.ATTN_EXACT_KEYS)
        ctx.save_for_backward(q, k, v, o, lse, q_lens, k_lens, *rest)
        ctx.scale, ctx.causal, ctx.bwd_mode = scale, causal, bwd_mode
        ctx.set_materialize_grads(False)
        return o, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, do, dlse):
        q, k, v, o, lse, q_lens, k_lens, *rest = ctx.saved_tensors
        if do is None and dlse is None:
            return (None,) * 9
        if do is None:
            do = torch.zeros_like(o)
        return (*_lib.attn_bwd(q, k, v, o, lse, do, dlse, ctx.scale, ctx.causal, q_lens, k_lens, ctx.bwd_mode, *rest),
                None, None, None, None, None, None)


def attention(q, k, v, scale=None, causal=False, q_lens=None, k_lens=None, return_lse=False, bwd_mode=_lib.BWD_AUTO):
    """softmax(scale Q K^T) V, differentiable: bf16 [B, H, N_Q, D], and with return_lse the rows' log-sum-exp
    (fp32 [B, H, N_Q], differentiable too).

    The attention of a model that is distilled with attention_kl, which takes the same q and k.  k and v may have
    fewer heads than q; q_lens, k_lens (int32 [B]) are the lengths of a padded batch's sequences.  See attn_fwd,
    and attn_bwd for bwd_mode.  Where a gradient will be asked for, what rounding o left (a tensor like o) is kept for
    the backward beside q, k, v, o and lse.
    """
    train = torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad)
    o, lse = _Attention.apply(q, k, v, scale, causal, q_lens, k_lens, bwd_mode, train)
    return (o, lse) if return_lse else o


class _DifferentialAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, lam, scale, causal, q_lens, k_lens, bwd_mode, train):
        d, lse, *maps = _lib.diff_attn_fwd(q, k, v, lam, scale, causal, q_lens, k_lens, train)
        ctx.save_for_backward(q, k, v, lam, lse, q_lens, k_lens, *maps)
        ctx.scale, ctx.causal, ctx.bwd_mode = scale, causal, bwd_mode
        ctx.set_materialize_grads(False)
        return d, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dd, dlse):
        q, k, v, lam, lse, q_lens, k_lens, maps, rest = ctx.saved_tensors
        if dd is None and dlse is None:
            return (None,) * 10
        if dd is None:
            dd = q.new_zeros(q.shape[0], q.shape[1] // 2, *q.shape[2:])
        *grads, dlam = _lib.diff_attn_bwd(q, k, v, lam, maps, lse, dd, dlse, ctx.scale, ctx.causal, q_lens, k_lens,
                                          ctx.bwd_mode, rest)
        return (*grads, dlam.sum_to_size(lam.shape), None, None, None, None, None, None)


def differential_attention(q, k, v, lam, scale=None, causal=False, q_lens=None, k_lens=None, return_lse=False,
                           bwd_mode=_lib.BWD_AUTO):
    """softmax(scale Q1 K^T) V - lam softmax(scale Q2 K^T) V, differentiable in q, k, v and lam: bf16 [B, H, N_Q, D], and with
    return_lse both maps' log-sum-exps (fp32 [B, 2 H, N_Q], differentiable too).

    The attention of a model whose heads are differences of two maps: q [B, 2 H, N_Q, D] has heads 2 i and 2 i + 1 for
    difference i, k and v [B, HK, N_K, D] may have fewer heads; lam fp32 broadcasts to [B, H, N_Q].  Either map is distilled
    with attention_kl on its heads of q.  See diff_attn_fwd and diff_attn_bwd; where a gradient will be asked for, each map's
    own result is kept for the backward in two parts like q.
    """
    train = torch.is_grad_enabled() and any(t.requires_grad for t in (q, k, v, lam))
    d, lse = _DifferentialAttention.apply(q, k, v, lam, scale, causal, q_lens, k_lens, bwd_mode, train)
    return (d, lse) if return_lse else d


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, scale, top_k):
        logp, entropy, lse, top_logp, top_index = _lib.logprobs_fwd(logits, tokens, scale, top_k)
        ctx.save_for_backward(logits, tokens, lse, entropy)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(top_logp, top_index)
        return logp, entropy, top_logp, top_index

    @staticmethod
    @once_differentiable
    def backward(ctx, g_logp, g_entropy, _top_logp, _top_index):
        logits, tokens, lse, entropy = ctx.saved_tensors
        if g_logp is None and g_entropy is None:
            return None, None, None, None
        given = tokens if g_logp is not None else None
        return _lib.logprobs_bwd(logits, given, lse, entropy, g_logp, g_entropy, ctx.scale), None, None, None


def token_logprobs(logits, tokens=None, scale=1.0, top_k=0):
    """(logp, entropy, top_logp, top_index) of each row of logits, differentiable in logp and entropy.

    The output-layer terms of a distillation loss: the log probabilities of the data's tokens (tokens [...]) or of
    a teacher's alternatives (tokens [..., T], for example the teacher's top_index) under
    softmax(scale * logits), the rows' entropy, and their own top_k alternatives, which have no gradient (give
    them as tokens to train on them).  See logprobs_fwd for shapes, types and masked values.
    """
    return _TokenLogprobs.apply(logits, tokens, scale, top_k)


class _VocabCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, tokens, scale):
        loss, lse = _lib.vocab_xent_fwd(hidden, weight, tokens, scale)
        ctx.save_for_backward(hidden, weight, tokens, lse)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return loss, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, g_loss, g_lse):
        hidden, weight, tokens, lse = ctx.saved_tensors
        if g_loss is None and g_lse is None:
            return None, None, None, None
        if g_loss is None:
            g_loss = torch.zeros_like(lse)
        return (*_lib.vocab_xent_bwd(hidden, weight, tokens, lse, g_loss, g_lse, ctx.scale, ctx.needs_input_grad[0],
                                     ctx.needs_input_grad[1]), None, None)


def vocab_cross_entropy(hidden, weight, tokens, scale=1.0, return_lse=False):
    """-log softmax(scale hidden weight^T)[token] of each row, differentiable in hidden and weight: fp32 like tokens, and
    with return_lse the rows' log-sum-exp, differentiable too (for a penalty on it).

    The loss on the data's tokens beside attention_kl, where the logits themselves are not wanted: they are never in memory
    (token_logprobs takes logits that are).  hidden [..., C] and weight [V, C] are bf16 or fp16; a negative token is none:
    its loss is 0.  See vocab_xent_fwd and vocab_xent_bwd.
    """
    loss, lse = _VocabCrossEntropy.apply(hidden, weight, tokens, scale)
    return (loss, lse) if return_lse else loss


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, plan, positions, offset, interleaved):
        ctx.save_for_backward(positions)
        ctx.plan, ctx.offset, ctx.interleaved = plan, offset, interleaved
        ctx.set_materialize_grads(False)
        return _lib.rotary_fwd(q, k, plan, positions, offset, interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        if dq is None and dk is None:
            return (None,) * 6
        positions, = ctx.saved_tensors
        return (*_lib.rotary_bwd(dq, dk, ctx.plan, positions, ctx.offset, ctx.interleaved), None, None, None, None)


def rotary(q, k, plan, positions=None, offset=0, interleaved=False):
    """(q, k) turned by their positions, differentiable: what attention, differential_attention and attention_kl take.

    q: [B, HQ, N, D], k: [B, HK, N, D]; plan: rotary_plan's; positions int64 or int32 [N] or [B, N], or rows from offset on.
    See rotary_fwd.
    """
    return _Rotary.apply(q, k, plan, positions, offset, interleaved)
