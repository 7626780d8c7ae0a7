"""The gradient at forbidden entries (-inf) of logits: none, but for a forbidden token's own, which is the gradient of its log
probability as the formula has it: dz_v = gl ([v = y] - p_v) - ge p_v (log p_v + H) with p_v = 0. Against that in 64
bits; p's relative error is below 2^-15 here (rows' sums of at most 40 allowed entries of size up to 10, lse below
16 or the maximum taken off first), f's is below that of its terms' magnitudes, and the result is rounded once."""
import math

import pytest
import torch

from rank_randomized_gradient_amd import log_prob, rgc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INF = math.inf


@pytest.mark.parametrize("zt", [BF, F32])
@pytest.mark.parametrize("V", [9, 40, 9001, 20000])
@pytest.mark.parametrize("base", [0.0, 4096.0])
def test_a_forbidden_token(V, zt, base):
    """In rows of one allowed entry and of several, near and far from zero (|lse| above 1024), at a row's ends and within."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda", 0)
    g = torch.Generator().manual_seed(V)
    rows = 12
    z = torch.full((rows, V), -INF)
    y = torch.tensor([V - 1, 0, V // 2] * (rows // 3))
    for i in range(rows):
        free = [int(k) for k in torch.randperm(V, generator=g)[:1 if i < 3 else 40] if int(k) != int(y[i])][:1 if i < 3 else 40]
        free = free or [(int(y[i]) + 1) % V]
        z[i, free] = base + 32 * torch.randint(0, 4, (len(free),), generator=g) / (32.0 if base else 16.0)
    z = z.to(zt)
    gl, ge = torch.randn(rows, generator=g), 0.5 * torch.randn(rows, generator=g)
    zg, yg, glg, geg = (t.to(dev) for t in (z, y, gl, ge))
    logp, entropy, lse, _, _ = rgc.rgc_log_prob_forward(zg, yg)
    assert bool((logp == -INF).all()) and bool((lse.abs() >= 1024).all()) == (base > 0)
    dz = rgc.rgc_log_prob_backward(zg, yg, lse, entropy, glg, geg).double().cpu()
    z64 = z.double()
    p = torch.softmax(z64, 1)
    lp = torch.where(p > 0, torch.log_softmax(z64, 1), 0.0)
    H = -(p * lp).sum(1, keepdim=True)
    want = -p * (gl.double()[:, None] + ge.double()[:, None] * (lp + H))
    want[torch.arange(rows), y] += gl.double()
    size = p * (gl.abs()[:, None] + ge.abs()[:, None] * (lp.abs() + H))
    off = (torch.finfo(zt).eps / 2) * want.abs() + 2.0 ** -14 * size
    assert bool(((dz - want).abs() <= off).all())
    assert torch.equal(dz[torch.arange(rows), y], gl.to(zt).double())
    others = z == -INF
    others[torch.arange(rows), y] = False
    assert bool((dz[others] == 0).all())
    # in place, and through the function
    zi = zg.clone()
    rgc.rgc_log_prob_backward(zi, yg, lse, entropy, glg, geg, dZ=zi)
    assert torch.equal(zi.double().cpu(), dz)
    leaf = zg.clone().requires_grad_()
    a, b = log_prob(leaf, yg)
    torch.autograd.backward([a, b], [glg, geg])
    assert torch.equal(leaf.grad.double().cpu(), dz)
