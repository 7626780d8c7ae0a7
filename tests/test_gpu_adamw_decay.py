"""AdamW's weight decay at rates near fp32's last place."""
import math

import pytest
import torch

from rank_randomized_gradient_amd import rgc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("decay", [1e-8, 3e-8, 1e-7, 1e-5])
def test_mean_decay_is_what_was_asked(decay):
    """Parameters from 1 to 2 take steps of random size and sign, so that each one's final rounding is as likely up as
    down, and the mean of many shows the decay. That rounding is off by at most half of fp32's step there, 2^-24
    (spread 2^-24 / sqrt(3)); the step's own errors, some 2^-21 of its 1e-3, have its random sign; the decay's rounding
    is 2^-23 of it."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev, n, lr, step = torch.device("cuda", 0), 1 << 22, 1e-3, 10
    gen = torch.Generator(device=dev).manual_seed(2)
    p = torch.rand(n, generator=gen, device=dev) + 1
    m = torch.randn(n, generator=gen, device=dev)
    v = torch.rand(n, generator=gen, device=dev) + 0.5
    m64, v64, want = 0.9 * m.double(), 0.999 * v.double(), p.double()
    want = want - decay * want - lr / (1 - 0.9 ** step) * m64 / (torch.sqrt(v64 / (1 - 0.999 ** step)) + 1e-8)
    rgc.rgc_adamw_batch([p], [torch.zeros(n, device=dev)], [m], [v], lr, step, weight_decay=decay / lr)
    off = abs(float((p.double() - want).mean()))
    tol = 6 * (2.0 ** -24 / math.sqrt(3) + 2.0 ** -21 * 1e-3) / math.sqrt(n) + 2.0 ** -22 * decay
    assert off < tol, (off, tol)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_infinite_parameters_stay(dtype, decay):
    """A parameter set to an infinity (a masked entry) keeps it; NaN stays NaN; the others do as without them."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev, n = torch.device("cuda", 0), 1000
    clean = torch.randn(n, generator=torch.Generator().manual_seed(4)).to(dtype).to(dev)
    at = {3: -float("inf"), 500: float("inf"), 999: float("nan")}
    out = []
    for marked in (False, True):
        p = clean.clone()
        for i, x in at.items():
            p[i] = x if marked else 0.0
        g = torch.ones(n, device=dev)
        rgc.rgc_adamw_batch([p], [g], [torch.zeros(n, device=dev)], [torch.zeros(n, device=dev)], 1e-2, 1, seed=1,
                            weight_decay=decay)
        out.append(p)
    assert float(out[1][3]) == -float("inf") and float(out[1][500]) == float("inf") and math.isnan(float(out[1][999]))
    keep = torch.ones(n, dtype=torch.bool, device=dev)
    keep[list(at)] = False
    assert torch.equal(out[0][keep], out[1][keep])
