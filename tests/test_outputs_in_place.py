"""The modules' outputs are tensors of their own, which may be changed in place (a dropout, a scale, an
addition) with the gradient of what they became. What a backward reads again, autograd finds changed. On the CPU with
stand-ins for the library's calls; on the GPU with the calls themselves."""
import types

import pytest
import torch

from rank_randomized_gradient_amd import LayerNorm, SketchedCrossEntropy, SketchedLinear, layer_norm, rgc, sketched_head, sketched_linear, synth

BF = torch.bfloat16
SHAPES = [(6,), (2, 3), (2, 0)]


def _stand_ins():
    """Functions of the right shapes, and gradients that tell them apart."""
    def linear(x, w, p=None, **_):
        return x @ w.T, None if p is None else x @ p

    def loss(x, w, t, p):
        return x.float().sum(1), x.float().sum(1), x @ p

    return types.SimpleNamespace(
        RgcError=rgc.RgcError,
        rgc_layer_norm_forward=lambda x, w, b, **_: (2 * x, x[:, 0].float(), x[:, 0].float()),
        rgc_layer_norm_backward=lambda dy, x, *_, **__: (2 * dy, None, None),
        rgc_add_norm_forward=lambda x, r, w, b, **_: (x + r, 2 * (x + r), x[:, 0].float(), x[:, 0].float()),
        rgc_add_norm_backward=lambda dy, ds, s, *_, **__: (2 * dy if ds is None else 2 * dy + ds, None, None),
        rgc_linear_forward=linear, rgc_linear_backward=lambda d, w, *_, **__: d.float() @ w,
        rgc_linear_cross_entropy_forward=loss,
        rgc_linear_cross_entropy_backward=lambda x, w, t, lse, g, *_, **__: g[:, None].to(x.dtype).expand_as(x))


@pytest.fixture
def calls(monkeypatch):
    for module in (layer_norm, sketched_head, sketched_linear):
        monkeypatch.setattr(module, "rgc", _stand_ins())


def _x(shape, seed=1):
    return torch.randn(*shape, 8, generator=torch.Generator().manual_seed(seed))


def _same_gradient(make, leaves):
    """The gradients of `leaves` where the output is scaled in place, and where it is not."""
    grads = []
    for change in (lambda t: t.mul_(3.0), lambda t: t * 3.0):
        got = [t.clone().requires_grad_() for t in leaves]
        change(make(*got)).float().sum().backward()
        grads.append([t.grad for t in got])
    assert all(torch.equal(a, b) for a, b in zip(*grads))


@pytest.mark.parametrize("shape", SHAPES)
def test_each_function(calls, shape):
    w, p = torch.randn(4, 8), torch.randn(8, 2)
    anchor = lambda: torch.zeros((), requires_grad=True)  # noqa: E731
    t = torch.zeros(shape, dtype=torch.int64)
    norm = lambda x: layer_norm.LayerNormFunction.apply(x, None, None, 1e-5, "rms")  # noqa: E731
    add = lambda i: lambda x, r: layer_norm.AddNormFunction.apply(x, r, None, None, 1e-5, "rms")[i]  # noqa: E731
    linear = lambda x: sketched_linear.SketchedLinearFunction.apply(x, w, p, None, None, anchor())  # noqa: E731
    loss = lambda x: sketched_head.SketchedCrossEntropyFunction.apply(x, w, t, p, None, anchor())  # noqa: E731
    x = _x(shape)
    for make, size in ((norm, x.shape), (linear, (*shape, 4)), (loss, shape)):
        assert make(x).shape == torch.Size(size)
        _same_gradient(make, [x])
    assert all(t.shape == x.shape for t in layer_norm.AddNormFunction.apply(x, x, None, None, 1e-5, "rms"))
    _same_gradient(add(0), [x, _x(shape, 2)])
    # the sum, where nothing reads it again
    _same_gradient(add(1), [x, _x(shape, 2)])


@pytest.mark.parametrize("shape", SHAPES[:2])
def test_a_sum_that_the_backward_reads(calls, shape):
    y, s = layer_norm.AddNormFunction.apply(_x(shape).requires_grad_(), _x(shape, 2), None, None, 1e-5, "rms")
    s.add_(1.0)
    with pytest.raises(RuntimeError, match="in-?place"):
        (y + s).sum().backward()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(6,), (2, 3)])
def test_the_modules_themselves(shape):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda", 0)
    x, r = (synth.normal_bf16((*shape, 64), 1.0, seed=s).to(dev) for s in (1, 2))
    norm, layer = LayerNorm(64, device=dev), SketchedLinear(64, 64, 16, device=dev)
    head = SketchedCrossEntropy(64, 104, 16, device=dev)
    layer.begin_update(1), head.begin_update(2)
    t = torch.arange(6, device=dev).reshape(shape)
    _same_gradient(norm, [x])
    _same_gradient(lambda a, b: norm(a, b)[0], [x, r])
    _same_gradient(lambda a, b: norm(a, b)[1], [x, r])
    _same_gradient(layer, [x])
    _same_gradient(lambda a: head(a, t), [x])
    # a block's stream goes on in place behind the norm that read it: found, and not a wrong gradient
    leaf = x.clone().requires_grad_()
    n, stream = norm(leaf, r)
    stream += layer(n)
    with pytest.raises(RuntimeError, match="in-?place"):
        stream.float().sum().backward()
