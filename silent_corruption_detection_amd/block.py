"""The two recomputed halves of a transformer block, differentiable, with what they
recompute audited: softmax attention and the gated feed-forward block.

Activation checkpointing computes most of a block a second time; the scores of
attention and the projections of the feed-forward block are not even kept between the
passes that use them.  A recomputation must reproduce the original bit for bit (AEGIS
review page, "Safeguarding LLM Training at Scale", section "core method", item 4), but
what is nowhere in memory no scan can cover.  Both passes therefore take the
fingerprint row of the scores (projections) while they are in registers, and the
backward pass compares the two on the device.

`attention` and `gated_ffn` are what `RecomputeAudit.attention` and
`RecomputeAudit.gated_ffn` call; without an audit they are the operators alone.  Their
outputs and gradients are bit-reproducible, as the ring replay's comparison of gradient
fingerprints needs (AWS Machine Learning Blog, "Detecting and recovering from silent data
corruption on Amazon SageMaker HyperPod", section "Check 2").

Captured into a HIP graph, forward and backward pass belong into the same capture, with no
output of the same leaves from before it still alive (autograd would wait for that one's
stream inside the capture).
"""
import torch
from torch.autograd.function import once_differentiable

from . import sdc_attention, sdc_attention_grad, sdc_gated_ffn, sdc_gated_ffn_grad


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, seq_q, seq_k, how, row, checked):
        out, lse = sdc_attention(q, k, v, seq_q=seq_q, seq_k=seq_k, row=row, **how)
        ctx.save_for_backward(q, k, v, seq_q, seq_k, out, lse)
        ctx.how, ctx.checked = how, checked
        ctx.mark_non_differentiable(lse)
        ctx.set_materialize_grads(False)  # no zeros for lse
        return out, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, grad, _):
        q, k, v, seq_q, seq_k, out, lse = ctx.saved_tensors
        kw = {} if ctx.checked is None else ctx.checked()
        needs = ctx.needs_input_grad
        dq, dk, dv = sdc_attention_grad(q, k, v, out, lse, grad, seq_q=seq_q, seq_k=seq_k, need_dq=needs[0],
                                        need_dkv=needs[1] or needs[2], **ctx.how, **kw)
        return dq, dk if needs[1] else None, dv if needs[2] else None, None, None, None, None, None


def attention(q, k, v, causal=False, window=0, scale=None, seq_q=None, seq_k=None, row=None, checked=None):
    """softmax(scale q k^T) v, differentiable in q, k and v; see sdc_attention for the
    arguments.  Rows of no packed sequence are zero, in the output and in the gradients.

    row: an int64 [1, 4] device tensor that receives the scores' fingerprint row.
    checked: called when the backward pass starts; returns sdc_attention_grad's
    arguments of the comparison (row, ref, mismatch, col_mask)."""
    how = dict(causal=causal, window=window, scale=scale)
    return _Attention.apply(q, k, v, seq_q, seq_k, how, row, checked)[0]


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, act, row, checked):
        ctx.save_for_backward(x, w_gate, w_up)
        ctx.act, ctx.checked = act, checked
        return sdc_gated_ffn(x, w_gate, w_up, act=act, row=row)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, w_gate, w_up = ctx.saved_tensors
        kw = {} if ctx.checked is None else ctx.checked()
        needs = ctx.needs_input_grad
        dx, dw_gate, dw_up = sdc_gated_ffn_grad(x, w_gate, w_up, grad, act=ctx.act, need_dx=needs[0],
                                                need_dw=needs[1] or needs[2], **kw)
        return dx, dw_gate if needs[1] else None, dw_up if needs[2] else None, None, None, None


def gated_ffn(x, w_gate, w_up, act="silu", row=None, checked=None):
    """act(x w_gate^T) * (x w_up^T), differentiable in all three; x: [..., d].  The
    projections are computed again in the backward pass; the matrix that takes the
    block's output back to d is an ordinary linear layer behind it.

    row: an int64 [1, 4] device tensor that receives the projections' fingerprint row.
    checked: called when the backward pass starts; returns sdc_gated_ffn_grad's
    arguments of the comparison (row, ref, mismatch, col_mask)."""
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    h = _GatedFfn.apply(x.reshape(-1, x.shape[-1]), w_gate, w_up, act, row, checked)
    return h.reshape(*x.shape[:-1], w_gate.shape[0])
