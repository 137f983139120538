"""The cross entropy of a linear head, differentiable, with its logits audited.

The logits of a large vocabulary are never kept: the backward pass computes them
again.  That is a recomputation in the sense of the AEGIS review page
("Safeguarding LLM Training at Scale"), section "core method", item 4 -- it must
reproduce the original bit for bit -- whose original is nowhere in memory, so a
scan of saved tensors cannot cover it.  Both passes therefore take the logits'
fingerprint row while the logits are in registers, and the backward pass compares
the two on the device.

`linear_cross_entropy` is what `RecomputeAudit.cross_entropy` calls; without an
audit it is the loss alone.  The loss it returns and the gradients are
bit-reproducible, as the ring replay's comparison of loss bits and gradient
fingerprints needs (AWS Machine Learning Blog, "Detecting and recovering from
silent data corruption on Amazon SageMaker HyperPod", section "Check 2").
"""
import torch
from torch.autograd.function import once_differentiable

from . import sdc_cross_entropy, sdc_cross_entropy_grad


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, target, mean, row, checked):
        count = torch.empty(1, dtype=torch.int64, device=x.device)
        _, lse, total = sdc_cross_entropy(x, w, target, count=count, row=row)
        ctx.save_for_backward(x, w, target, lse, count)
        ctx.mean, ctx.checked = mean, checked
        total = total[0]
        return total / count[0] if mean else total

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, w, target, lse, count = ctx.saved_tensors
        # no row with a target: the loss is 0 / 0, the gradient zero
        g = (grad / count.clamp(min=1) if ctx.mean else grad).float().reshape(1)
        kw = {} if ctx.checked is None else ctx.checked()
        dx, dw = sdc_cross_entropy_grad(x, w, target, lse, g, need_dx=ctx.needs_input_grad[0],
                                        need_dw=ctx.needs_input_grad[1], **kw)
        return dx, dw, None, None, None, None


def linear_cross_entropy(x, w, target, reduction="mean", row=None, checked=None):
    """Cross entropy of the logits x w^T as a scalar fp32 tensor.

    x: [..., d], w: [vocab, d], bfloat16 or float16 on one GPU; target: int64
    [...], an index outside [0, vocab) (for example -100) for a position without
    a target.  reduction: "mean" over the positions with a target (NaN when there
    is none) or "sum".

    row: an int64 [1, 4] device tensor that receives the logits' fingerprint row.
    checked: called when the backward pass starts; returns sdc_cross_entropy_grad's
    arguments of the comparison (row, ref, mismatch, col_mask).

    Captured into a HIP graph, forward and backward pass belong into the same
    capture, with no loss of the same leaves from before it still alive (autograd
    would wait for that one's stream inside the capture)."""
    if reduction not in ("mean", "sum"):
        raise ValueError(f"reduction must be 'mean' or 'sum', not {reduction!r}")
    if x.dim() < 1 or target.shape != x.shape[:-1]:
        raise ValueError(f"target must have the shape {tuple(x.shape[:-1])}, is {tuple(target.shape)}")
    return _LinearCrossEntropy.apply(x.reshape(-1, x.shape[-1]), w, target.reshape(-1).contiguous(),
                                     reduction == "mean", row, checked)
