"""A sketched layer whose input requires no gradient (a model's first): its
sketch is trained all the same."""
import pytest
import torch

from rank_randomized_gradient_amd import LayerNorm, SketchedLinear, rgc, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


@pytest.mark.parametrize("T,k,d,r", [(20, 64, 128, 16), (300, 264, 136, 16), (40, 64, 72, 4)])
def test_the_sketch_is_added_to(dev, T, k, d, r):
    layer = SketchedLinear(k, d, r, device=dev)
    layer.begin_update(3)
    x = synth.normal_bf16((T, k), 1.0, seed=1).to(dev)
    dy = synth.normal_bf16((T, d), 0.1, seed=2).to(dev)
    layer(x).backward(dy)
    want = torch.zeros_like(layer.sketch)
    rgc.rgc_accumulate(dy, rgc.rgc_linear_forward(x, layer.weight, layer.proj)[1], want)
    assert torch.equal(layer.sketch, want) and bool((want != 0).any()) and x.grad is None


def test_below_a_layer_that_is_trained_otherwise(dev):
    """The norm's gradient alone used to end the backward before the layer."""
    layer, norm = SketchedLinear(64, 128, 16, device=dev), LayerNorm(128, device=dev)
    layer.begin_update(3)
    x = synth.normal_bf16((20, 64), 1.0, seed=1).to(dev)
    norm(layer(x)).square().sum().backward()
    got = layer.sketch.clone()
    layer.sketch.zero_()
    norm(layer(x.clone().requires_grad_(True))).square().sum().backward()
    rel = float((got - layer.sketch).norm() / layer.sketch.norm())
    assert bool((got != 0).any()) and rel < 2.0 ** -18, rel  # the same sums, of rgc_accumulate and of the layer's backward
    with torch.no_grad():
        assert not layer(x).requires_grad
