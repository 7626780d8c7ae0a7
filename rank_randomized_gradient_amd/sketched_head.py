"""The vocabulary head of a model trained through sketches: a linear layer and
its softmax cross entropy in one, so that neither the logits nor their gradient
exist as a whole.

Where SketchedLinear turns D = dL/dY into its sketch, this layer's D is the
largest tensor of a step (tokens x vocabulary). It is formed a piece of the
vocabulary at a time from the logits of that piece, used for dX = D W and
C += D^T (X P), and dropped. X is kept for that besides X P.

The same head gives a policy's log probabilities and entropies (log_prob), with
their gradient, and the most likely alternatives of each token (alternatives).
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
        return loss.resize_(targets.shape)  # (a tensor of its own and no view, which autograd lets nobody change in place)

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        x2, weight, t, lse, xp = ctx.saved_tensors
        g = dloss.reshape(-1).to(torch.float32).contiguous()
        dx = rgc.rgc_linear_cross_entropy_backward(x2, weight, t, lse, g, xp, ctx.sketch,
                                                   input_grad=ctx.needs_input_grad[0])
        return None if dx is None else dx.reshape(ctx.in_shape), None, None, None, None, None


class SketchedLogProbFunction(torch.autograd.Function):
    """Per-token log probabilities and entropies; saves X, X P, each token's log sum of exponentials
    and its entropy. `anchor` as for the losses."""

    @staticmethod
    def forward(ctx, x, weight, tokens, proj, sketch, anchor=None):
        ctx.set_materialize_grads(False)
        x2 = x.reshape(-1, x.shape[-1])
        if not x2.is_contiguous():
            x2 = x2.contiguous()
        t = tokens.reshape(-1).contiguous()
        logp, entropy, lse, xp = rgc.rgc_linear_log_prob_forward(x2, weight, t, proj)
        # (tensors of their own and no views, which autograd lets nobody change in place)
        logp.resize_(tokens.shape), entropy.resize_(tokens.shape)
        ctx.save_for_backward(x2, weight, t, lse, entropy, xp)
        ctx.sketch = sketch
        ctx.in_shape = x.shape
        return logp, entropy

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp, dentropy):
        x2, weight, t, lse, entropy, xp = ctx.saved_tensors
        if dlogp is None and dentropy is None:
            return None, None, None, None, None, None
        flat = lambda g: None if g is None else g.reshape(-1).to(torch.float32).contiguous()  # noqa: E731
        dx = rgc.rgc_linear_log_prob_backward(x2, weight, t, lse, flat(entropy), flat(dlogp), flat(dentropy), xp, ctx.sketch,
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

    log_prob(x, tokens) gives (log probabilities, entropies) instead, for a policy's
    loss: its backward takes the gradients of both and adds to `sketch` likewise.
    Losses and log probabilities need no projection under torch.no_grad(): begin_update may come later, or never.
    alternatives(x, top) gives each row's `top` most likely entries.
    """

    def _projection(self) -> torch.Tensor | None:
        """What X is projected with for the backward; none where no gradient is recorded."""
        if not torch.is_grad_enabled():
            return None
        if self.proj_seed is None:
            raise rgc.RgcError("begin_update(seed) must draw the projection before the first forward")
        return self.proj

    def forward(self, x: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        proj = self._projection()
        if targets.dtype != torch.int64 or targets.shape != x.shape[:-1]:
            raise rgc.RgcError("targets must be int64, one for each row of x")
        anchor = torch.zeros((), device="cpu", requires_grad=True)
        return SketchedCrossEntropyFunction.apply(x, self.weight, targets, proj, self.sketch, anchor)

    def log_prob(self, x: torch.Tensor, tokens: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
        """(log probability of each token, entropy of its distribution), float32; both 0 for a token outside
        0 .. vocabulary - 1."""
        proj = self._projection()
        if tokens.dtype != torch.int64 or tokens.shape != x.shape[:-1]:
            raise rgc.RgcError("tokens must be int64, one for each row of x")
        anchor = torch.zeros((), device="cpu", requires_grad=True)
        return SketchedLogProbFunction.apply(x, self.weight, tokens, proj, self.sketch, anchor)

    @torch.no_grad()
    def alternatives(self, x: torch.Tensor, top: int) -> tuple[torch.Tensor, torch.Tensor]:
        """(log probabilities, indices) of each row's `top` most likely entries, in descending order, (..., top)
        each. The logits are formed in bf16 (as a plain head's are), up to 256 MB of them at a time, so that a log
        probability may be off from log_prob's by half a bf16 step of its logit (1/16 at 16 to 32); of equal ones the
        lowest index comes first."""
        if not 1 <= top <= 64:
            raise rgc.RgcError("top must lie in 1 .. 64")
        x2 = x.reshape(-1, x.shape[-1])
        if not x2.is_contiguous():
            x2 = x2.contiguous()
        rows, vocabulary = x2.shape[0], self.weight.shape[0]
        logp = torch.empty((rows, top), dtype=torch.float32, device=x.device)
        ids = torch.empty((rows, top), dtype=torch.int64, device=x.device)
        piece = max(1, min(65536, (1 << 27) // vocabulary))
        with rgc._on(rgc._need_gpu(x2, self.weight)):
            for i in range(0, rows, piece):
                logits, _ = rgc.rgc_linear_forward(x2[i:i + piece], self.weight)
                _, _, _, logp[i:i + piece], ids[i:i + piece] = rgc.rgc_log_prob_forward(logits, top=top)
        return logp.reshape(*x.shape[:-1], top), ids.reshape(*x.shape[:-1], top)
