"""Layer norms and root-mean-square norms between the sketched layers. Their
gains and biases are small and keep a dense gradient (AdamW's to use)."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import rgc


def _row_major(t: torch.Tensor) -> torch.Tensor:
    """t as rows of its last dimension, which follow each other without overlap (a broadcast tensor's do not)."""
    rows = t.reshape(-1, t.shape[-1])
    if rows.stride(1) != 1 or (rows.shape[0] > 1 and rows.stride(0) < rows.shape[1]):
        rows = rows.contiguous()
    return rows


class LayerNormFunction(torch.autograd.Function):
    """The norm of the last dimension; saves X and each row's mean and rstd."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, kind):
        x2 = _row_major(x)
        y, mean, rstd = rgc.rgc_layer_norm_forward(x2, weight, bias, eps=eps, kind=kind)
        ctx.save_for_backward(x2, weight, mean, rstd)
        ctx.kind = kind
        ctx.bias_dtype = None if bias is None else bias.dtype
        ctx.shape = x.shape
        return y.reshape(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x2, weight, mean, rstd = ctx.saved_tensors
        d2 = _row_major(dy if dy.dtype == x2.dtype else dy.to(x2.dtype))
        dx, dw, db = rgc.rgc_layer_norm_backward(d2, x2, weight, mean, rstd, bias=ctx.bias_dtype is not None, kind=ctx.kind)
        return (dx.reshape(ctx.shape), dw if weight is not None else None,
                None if db is None else db.to(ctx.bias_dtype), None, None)


class LayerNorm(torch.nn.Module):
    """Norm of the last dimension (kind "layer", or "rms" for the root-mean-square
    norm, which has no bias). Gains in float32 unless told otherwise: beside
    bf16 activations they cost nothing and their gradients stay float32.

    As with every torch parameter, a backward pass is captured into a graph
    only while no eager autograd graph over the same parameters is alive: torch
    would tie the capture to that graph's stream and end the process."""

    def __init__(self, features: int, eps: float = 1e-5, kind: str = "layer", bias: bool = True, device=None,
                 dtype: torch.dtype = torch.float32):
        super().__init__()
        if kind not in ("layer", "rms"):
            raise rgc.RgcError('kind must be "layer" or "rms"')
        device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.features, self.eps, self.kind = features, eps, kind
        self.weight = torch.nn.Parameter(torch.ones(features, dtype=dtype, device=device))
        with_bias = bias and kind == "layer"
        self.bias = torch.nn.Parameter(torch.zeros(features, dtype=dtype, device=device)) if with_bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.features:
            raise rgc.RgcError(f"the last dimension must be {self.features}")
        return LayerNormFunction.apply(x, self.weight, self.bias, self.eps, self.kind)
