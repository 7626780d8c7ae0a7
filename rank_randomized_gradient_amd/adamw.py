"""AdamW for the parameters that keep a dense gradient beside the sketched
layers: norm gains, biases, embeddings. All tensors of a step in few launches,
moments in 8 bits or 32, bf16 parameters rounded stochastically (no float32 copy).
"""
from __future__ import annotations

import torch

from . import rgc


class AdamW:
    """step() updates every parameter that has a gradient, in place.

    state_bits 8 holds both moments as e4m3 with a scale per 128 elements (2.06
    bytes an element), rounded stochastically, 32 as float32 (8 bytes). `seed` and the count of steps
    give the rounding bits, so a run repeats bit for bit. Parameters and
    gradients are contiguous bf16 or float32 tensors at multiples of 16 bytes. The step count and the
    rounding key are host values: a step captured into a graph would repeat
    both in every replay.
    """

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 state_bits: int = 8, seed: int = 0):
        if state_bits not in (8, 32):
            raise rgc.RgcError("state_bits must be 8 or 32")
        self.params = list(params)
        if len({id(p) for p in self.params}) != len(self.params):
            raise rgc.RgcError("a parameter is listed twice")
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.state_bits, self.seed = state_bits, seed
        # per parameter: None until its first gradient, then its step count and moments
        self.state = [None] * len(self.params)
        self.steps = 0

    def _fresh(self, p: torch.Tensor) -> dict:
        if self.state_bits == 32:
            return {"step": 0, "M": torch.zeros_like(p, dtype=torch.float32), "V": torch.zeros_like(p, dtype=torch.float32)}
        blocks = (p.numel() + rgc.ADAMW_BLOCK - 1) // rgc.ADAMW_BLOCK
        f8 = torch.float8_e4m3fn
        return {"step": 0, "M": torch.zeros(p.shape, dtype=f8, device=p.device),
                "V": torch.zeros(p.shape, dtype=f8, device=p.device),
                "M_scale": torch.zeros(blocks, dtype=torch.float32, device=p.device),
                "V_scale": torch.zeros(blocks, dtype=torch.float32, device=p.device)}

    @torch.no_grad()
    def step(self, grad_scale: torch.Tensor | None = None) -> None:
        """One step from the parameters' .grad, times grad_scale (a float32 on the
        device, e.g. a clipping coefficient; one that is not finite leaves the
        parameters and moments as they are, though the step is counted). A step that is
        refused changes nothing."""
        groups: dict = {}  # one call for each pair of types, device and step count
        for i, p in enumerate(self.params):
            if p.grad is None:
                continue
            if self.state[i] is None:
                self.state[i] = self._fresh(p)
            groups.setdefault((p.dtype, p.grad.dtype, p.device, self.state[i]["step"] + 1), []).append(i)
        eight, calls = self.state_bits == 8, []
        for n, ((_, _, _, t), at) in enumerate(groups.items()):
            s = [self.state[i] for i in at]
            # every call of a run has a key of its own: the seed, the step above bit 32 and the call above bit 56
            key = self.seed + ((self.steps + 1) << 32) + (n << 56)
            calls.append(rgc._adamw_call([self.params[i].data for i in at], [self.params[i].grad for i in at],
                                         [x["M"] for x in s], [x["V"] for x in s], self.lr, t, key, self.betas[0],
                                         self.betas[1], self.eps, self.weight_decay,
                                         [x["M_scale"] for x in s] if eight else None,
                                         [x["V_scale"] for x in s] if eight else None, grad_scale, "stochastic"))
        if len(calls) > 1:  # a call that would be refused is found before any is made
            for call in calls:
                call(rgc.RGC_ADAMW_CHECK_ONLY)
        for call, ((_, _, _, t), at) in zip(calls, groups.items()):
            call()
            for i in at:
                self.state[i]["step"] = t
        self.steps += 1

    def zero_grad(self, set_to_none: bool = True) -> None:
        for p in self.params:
            if p.grad is not None:
                if set_to_none:
                    p.grad = None
                else:
                    p.grad.zero_()

    def state_dict(self) -> dict:
        return {"steps": self.steps, "seed": self.seed, "state_bits": self.state_bits,
                "state": [None if s is None else dict(s) for s in self.state]}

    def load_state_dict(self, d: dict) -> None:
        """Takes copies of the moments, with their types as they are."""
        if d["state_bits"] != self.state_bits or len(d["state"]) != len(self.params):
            raise rgc.RgcError("the state belongs to another state_bits or parameter list")
        new = []
        for p, s in zip(self.params, d["state"]):
            if s is None:
                new.append(None)
                continue
            want = self._fresh(p)
            if set(s) != set(want) or any(torch.is_tensor(want[k]) and (s[k].shape != want[k].shape or s[k].dtype != want[k].dtype)
                                          for k in want):
                raise rgc.RgcError("the state does not fit the parameter")
            new.append({k: s[k].to(p.device, copy=True) if torch.is_tensor(s[k]) else s[k] for k in want})
        self.state, self.steps, self.seed = new, d["steps"], d["seed"]
