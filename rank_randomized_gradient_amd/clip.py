"""Clipping of all dense gradients by their global norm."""
from __future__ import annotations

import torch

from . import rgc


@torch.no_grad()
def clip_grad_norm(params, max_norm: float) -> torch.Tensor:
    """Multiplies the parameters' gradients (all on one device), in place, by min(1, max_norm / norm) and
    returns their norm (a scalar on the device; nothing waits for it; zero where there are none). A norm that is not
    finite (in 64 bits) leaves the gradients as they are. Where AdamW takes the gradients
    next, its step(max_norm=...) clips them as it reads them instead."""
    params = [params] if torch.is_tensor(params) else list(params)
    grads, seen = [], set()
    for p in params:
        if p.grad is not None and id(p) not in seen:
            seen.add(id(p))
            grads.append(p.grad)
    if not grads:
        return torch.zeros((), dtype=torch.float32, device=params[0].device if params else None)
    norm, scale = rgc.rgc_grad_norm_batch(grads, max_norm)
    rgc.rgc_scale_batch(grads, scale)
    return norm[0]
