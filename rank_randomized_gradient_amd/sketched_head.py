"""The vocabulary head of a model trained through sketches: a linear layer and
its softmax cross entropy in one, so that neither the logits nor their gradient
exist as a whole.

Where SketchedLinear turns D = dL/dY into its sketch, this layer's D is the
largest tensor of a step (tokens x vocabulary). It is formed a piece of the
vocabulary at a time from the logits of that piece, used for dX = D W and
C += D^T (X P), and dropped. X is kept for that besides X P.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import rgc
from .sketched_linear import SketchedLinear


class SketchedCrossEntropyFunction(torch.autograd.Function):
    """Per-token losses; saves X, X P and each token's log sum of exponentials.

    `anchor` is a scalar that requires a gradient and gets none: it brings the
    backward here, where the sketch is added to, whether or not x requires one
    (the weight does not)."""

    @staticmethod
    def forward(ctx, x, weight, targets, proj, sketch, anchor=None):
        x2 = x.reshape(-1, x.shape[-1])
        if not x2.is_contiguous():
            x2 = x2.contiguous()
        t = targets.reshape(-1).contiguous()
        loss, lse, xp = rgc.rgc_linear_cross_entropy_forward(x2, weight, t, proj)
        ctx.save_for_backward(x2, weight, t, lse, xp)
        ctx.sketch = sketch
        ctx.in_shape = x.shape
        return loss.reshape(targets.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        x2, weight, t, lse, xp = ctx.saved_tensors
        g = dloss.reshape(-1).to(torch.float32).contiguous()
        dx = rgc.rgc_linear_cross_entropy_backward(x2, weight, t, lse, g, xp, ctx.sketch,
                                                   input_grad=ctx.needs_input_grad[0])
        return None if dx is None else dx.reshape(ctx.in_shape), None, None, None, None, None


class SketchedCrossEntropy(SketchedLinear):
    """vocabulary x in bf16 head; forward(x, targets) gives each token's loss (float32).

    x: (..., in_features) bf16; targets: (...) int64, a token whose target lies
    outside 0 .. vocabulary - 1 (-100, say) is ignored: loss 0, no gradient.
    Weigh and sum the losses as the objective asks (a mean over the tokens that
    count, advantages). begin_update, apply_update and the carried norm are
    SketchedLinear's: the losses' backward adds the head's D^T (X P) to `sketch`,
    also for an x that requires no gradient.
    The vocabulary is a multiple of 8, as every sketched layer's width.
    """

    def forward(self, x: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        if self.proj_seed is None:
            raise rgc.RgcError("begin_update(seed) must draw the projection before the first forward")
        if targets.dtype != torch.int64 or targets.shape != x.shape[:-1]:
            raise rgc.RgcError("targets must be int64, one for each row of x")
        anchor = torch.zeros((), device="cpu", requires_grad=True)
        return SketchedCrossEntropyFunction.apply(x, self.weight, targets, self.proj, self.sketch, anchor)
