"""Log probabilities and entropies of logits at hand: those of a head that is not
sketched, of a reference model, or changed on their way (scaled, capped, masked)."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import rgc
from .layer_norm import _row_major


class LogProbFunction(torch.autograd.Function):
    """Saves the logits, and each row's log sum of exponentials and entropy."""

    @staticmethod
    def forward(ctx, logits, tokens):
        ctx.set_materialize_grads(False)
        z = _row_major(logits)
        t = tokens.reshape(-1).contiguous()
        logp, entropy, lse, _, _ = rgc.rgc_log_prob_forward(z, t)
        # (tensors of their own and no views, which autograd lets nobody change in place)
        logp.resize_(tokens.shape), entropy.resize_(tokens.shape)
        ctx.save_for_backward(z, t, lse, entropy)
        ctx.shape = logits.shape
        return logp, entropy

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp, dentropy):
        z, t, lse, entropy = ctx.saved_tensors
        if dlogp is None and dentropy is None:
            return None, None
        flat = lambda g: None if g is None else g.reshape(-1).to(torch.float32).contiguous()  # noqa: E731
        dz = rgc.rgc_log_prob_backward(z, t, lse, flat(entropy), flat(dlogp), flat(dentropy))
        return dz.reshape(ctx.shape), None


def log_prob(logits: torch.Tensor, tokens: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """(log probability of each token, entropy of its row), float32, of logits (..., vocabulary) in bf16 or
    float32; both 0 for a token outside 0 .. vocabulary - 1. Entries of -inf are forbidden ones. Both have a
    gradient."""
    if tokens.dtype != torch.int64 or tokens.shape != logits.shape[:-1]:
        raise rgc.RgcError("tokens must be int64, one for each row of logits")
    return LogProbFunction.apply(logits, tokens)
