"""Outputs in the place of inputs: a norm's Y over X, its dX over X or dY, the
head's dX over X. The bits are those of separate outputs."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [100, 1003, 4096, 16384, 16392, 20001])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norms(dev, dtype, n, kind):
    g = torch.Generator().manual_seed(n)
    x, dy = (torch.randn(300, n, generator=g).to(dtype).to(dev) for _ in range(2))
    w = torch.randn(n, generator=g).to(dev)
    y, mean, rstd = rgc.rgc_layer_norm_forward(x, w, kind=kind)
    want = rgc.rgc_layer_norm_backward(dy, x, w, mean, rstd, kind=kind)
    for over in ("X", "dY"):
        xc, dc = x.clone(), dy.clone()
        got = rgc.rgc_layer_norm_backward(dc, xc, w, mean, rstd, kind=kind, dX=xc if over == "X" else dc)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), over
    xc = x.clone()
    rgc.rgc_layer_norm_forward(xc, w, kind=kind, Y=xc)
    assert torch.equal(xc, y)


# one tile of tokens, several; one piece and several; split and unsplit sums
@pytest.mark.parametrize("T,V,k,r", [(20, 1000, 64, 16), (300, 2000, 264, 16), (2000, 70000, 64, 0), (700, 264, 4096, 8)])
def test_head(dev, T, V, k, r):
    x, w = synth.normal_bf16((T, k), 1.0, seed=1).to(dev), synth.normal_bf16((V, k), k ** -0.5, seed=2).to(dev)
    y = (torch.arange(T) * 13 % V).to(dev)
    gr = synth.normal_f32((T,), 1.0, seed=3).to(dev)
    xp = synth.normal_bf16((T, r), 1.0, seed=4).to(dev) if r else None
    _, lse, _ = rgc.rgc_linear_cross_entropy_forward(x, w, y)
    out = []
    for inside in (False, True):
        c, xc = torch.zeros(V, r, device=dev) if r else None, x.clone()
        dx = rgc.rgc_linear_cross_entropy_backward(xc, w, y, lse, gr, xp, c, dX=xc if inside else None)
        out.append((dx.clone(), c))
    assert torch.equal(out[0][0], out[1][0]) and (r == 0 or torch.equal(out[0][1], out[1][1]))
