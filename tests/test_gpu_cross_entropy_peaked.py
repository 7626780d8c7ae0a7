"""The head's input gradient where the softmax is peaked: a token's mass lies on
its target and on a rival whose row of W is near the target's, so that the two
large entries of D cancel in dX = D W and an error in either does not.

Bounds, element by element (as for flat logits, but for D's own precision): a
logit is off by at most 2^-20 of sum |x w|; D inherits p |g| times two such
errors and is held as two bf16 terms, each rounding leaving at most 2^-8 of what
it rounds and the second's half step at most 2^-17 of D; the targets' entries
are exact to fp32. dX adds the fp32 sums (2^-20 of sum |D W|) and its rounding
(2^-8 of itself).
"""
import pytest
import torch

from rank_randomized_gradient_amd import rgc, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _inputs(T, V, k, apart, seed):
    """Rows 2 i and 2 i + 1 of W differ by `apart` of their size; token t's logits are about 12 on one such pair
    (its target and the rival) and of size one elsewhere."""
    g = torch.Generator().manual_seed(seed)
    base = torch.randn(V // 2, k, generator=g)
    near = base * (1 + apart * torch.randn(V // 2, k, generator=g))
    w = torch.stack([base, near], 1).reshape(-1, k).bfloat16()
    pair = torch.randint(0, V // 2, (T,), generator=g)
    x = (12.0 * base[pair] / base[pair].square().sum(1, keepdim=True)).bfloat16()
    y = 2 * pair + torch.randint(0, 2, (T,), generator=g)
    y[4::9] = -100
    gr = torch.randn(T, generator=g)
    return x, w, y, gr


def _want(x, w, y, gr):
    x, w, gr = x.double(), w.double(), gr.double()
    z = x @ w.T
    live = (y >= 0) & (y < len(w))
    rows, at = torch.arange(len(y)), torch.where(live, y, 0)
    gl = torch.where(live, gr, torch.zeros(()).double())
    p = torch.exp(z - torch.logsumexp(z, 1)[:, None])
    d = p.clone()
    d[rows, at] -= 1
    d = d * gl[:, None]
    dz = 2.0 ** -20 * (x.abs() @ w.abs().T).amax(1)
    off = (2 * dz + 2.0 ** -20)[:, None] * p * gl.abs()[:, None]
    others = d.abs()
    others[rows, at] = 0
    dx = d @ w
    return dx, (off + 2.0 ** -17 * others + 2.0 ** -20 * d.abs()) @ w.abs() + 2.0 ** -8 * dx.abs()


# tokens in one tile of 64, of 128 and in several; every form of the sketch; a last tile of one token; two pieces
# of the vocabulary; a split sum
@pytest.mark.parametrize("T,V,k,r", [(1, 8, 64, 0), (5, 600, 64, 0), (64, 4104, 256, 16), (100, 1000, 136, 8),
                                     (128, 520, 264, 0), (129, 70008, 72, 16), (300, 2000, 264, 0), (385, 1032, 520, 128),
                                     (1025, 12000, 136, 0)])
@pytest.mark.parametrize("apart", [0.05, 0.5])
def test_rivals_near_the_target(dev, T, V, k, r, apart):
    print(T, V, k, r, apart, flush=True)
    x, w, y, gr = _inputs(T, V, k, apart, 7 * T + V)
    want, bound = _want(x, w, y, gr)
    xg, wg, yg, gg = (t.to(dev) for t in (x, w, y, gr))
    xp = synth.normal_bf16((T, r), 1.0, seed=1).to(dev) if r else None
    c = torch.zeros(V, r, device=dev) if r else None
    _, lse, _ = rgc.rgc_linear_cross_entropy_forward(xg, wg, yg)
    dx = rgc.rgc_linear_cross_entropy_backward(xg, wg, yg, lse, gg, xp, c)
    excess = (dx.double().cpu() - want).abs() - bound
    assert float(excess.max()) <= 1e-30, f"{float(excess.max()):.3e} over the bound"
