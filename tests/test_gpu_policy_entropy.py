"""The entropies' gradient through a policy's whole model, in a backward of its own: beside the log probabilities' it is
too small a part to be seen. Against the same model in 64 bits, with the bound of the whole step's test: about sixteen
tensors on the way are rounded to bf16, each by at most 2^-8 of itself, so 24 * 2^-8 of the norm bounds what adds up. (D = -ge p
(log p + H) takes the logits' error twice, as p's and as log p's beside a spread of about two; the logits' own error is
one of those sixteen and small beside its bound: rows' errors are independent and 2^-9 at their largest.)"""
import pytest
import torch

from rank_randomized_gradient_amd import LayerNorm, SketchedCrossEntropy, SketchedLinear, synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_entropy_alone(sign):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev, k, V, r = torch.device("cuda", 0), 256, 1000, 32
    norm1, norm2 = LayerNorm(k, kind="rms", device=dev), LayerNorm(k, device=dev)
    layer = SketchedLinear(k, k, r, device=dev, weight=synth.normal_bf16((k, k), k ** -0.5, seed=1))
    head = SketchedCrossEntropy(k, V, r, device=dev, weight=synth.normal_bf16((V, k), 2 * k ** -0.5, seed=2))
    layer.begin_update(5), head.begin_update(6)
    x = synth.normal_bf16((3, 40, k), 1.0, seed=3).to(dev).requires_grad_()
    g = torch.Generator().manual_seed(4)
    y = torch.randint(0, V, (3, 40), generator=g)
    y[:, :3] = -100
    ge = sign * (0.5 + torch.rand(3, 40, generator=g))
    n, _ = norm2(layer(norm1(x)), x)
    logp, entropy = head.log_prob(n, y.to(dev))
    (entropy * ge.to(dev)).sum().backward()

    d = lambda t: t.detach().double().cpu()  # noqa: E731
    leaf = lambda t: d(t).requires_grad_()  # noqa: E731
    x64, w1, w2, b2, wl, wh = (leaf(t) for t in (x, norm1.weight, norm2.weight, norm2.bias, layer.weight, head.weight))
    rms = lambda h, w: h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-5) * w  # noqa: E731
    s = x64 + rms(x64, w1) @ wl.T
    h = rms(s - s.mean(-1, keepdim=True), w2) + b2
    lp = torch.log_softmax(h @ wh.T, -1)
    ent = -(lp.exp() * lp).sum(-1)
    (torch.where(y >= 0, ent, 0.0) * ge.double()).sum().backward()
    for name, got, want in (("x", x.grad, x64.grad), ("norm1", norm1.weight.grad, w1.grad), ("norm2", norm2.weight.grad, w2.grad),
                            ("bias", norm2.bias.grad, b2.grad), ("layer", layer.sketch, wl.grad @ d(layer.proj)),
                            ("head", head.sketch, wh.grad @ d(head.proj))):
        rel = float((d(got) - want).norm() / want.norm())
        print(name, rel, flush=True)
        assert rel < 24 * 2.0 ** -8, (name, rel)
