"""The operators together, as a training step uses them: norms, sketched
layers and the vocabulary head's loss, their backward pass, and the two kinds
of update. Every module gives the bits of the calls it stands for; the whole
gives the gradients of the same model in 64 bits."""
import pytest
import torch

from rank_randomized_gradient_amd import AdamW, LayerNorm, SketchedCrossEntropy, SketchedLinear, rgc, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


class Model(torch.nn.Module):
    """norm -> sketched layer -> residual -> norm -> head and loss."""

    def __init__(self, k, V, r, dev, seed=0):
        super().__init__()
        self.norm1 = LayerNorm(k, kind="rms", device=dev)
        self.layer = SketchedLinear(k, k, r, device=dev, weight=synth.normal_bf16((k, k), k ** -0.5, seed=seed))
        self.norm2 = LayerNorm(k, device=dev)
        self.head = SketchedCrossEntropy(k, V, r, device=dev, weight=synth.normal_bf16((V, k), k ** -0.5, seed=seed + 1))
        with torch.no_grad():
            for i, p in enumerate((self.norm1.weight, self.norm2.weight, self.norm2.bias)):
                p.add_(0.1 * torch.randn(k, generator=torch.Generator().manual_seed(seed + 2 + i)).to(dev))

    def begin(self, seed):
        self.layer.begin_update(seed)
        self.head.begin_update(seed + 1)

    def forward(self, x, y):
        h = x + self.layer(self.norm1(x))
        return self.head(self.norm2(h), y)


def _batch(dev, B, S, k, V, seed):
    x = synth.normal_bf16((B, S, k), 1.0, seed=seed)
    g = torch.Generator().manual_seed(seed)
    y = torch.randint(0, V, (B, S), generator=g)
    y[:, 0] = -100
    return x.to(dev), y.to(dev)


def test_modules_give_the_bits_of_their_calls(dev):
    k, V, r = 256, 1000, 32
    m = Model(k, V, r, dev)
    m.begin(5)
    x, y = _batch(dev, 3, 40, k, V, 1)
    x.requires_grad_(True)
    loss = m(x, y)
    g = torch.randn(loss.shape, generator=torch.Generator().manual_seed(3)).to(dev) / loss.numel()
    loss.backward(g)
    assert m.layer.weight.grad is None and m.head.weight.grad is None
    # the same, call by call
    x2, y2 = x.detach().reshape(-1, k), y.reshape(-1)
    n1, _, r1 = rgc.rgc_layer_norm_forward(x2, m.norm1.weight.data, None, kind="rms")
    o, xp = rgc.rgc_linear_forward(n1, m.layer.weight, m.layer.proj)
    h = x2 + o
    n2, mu, r2 = rgc.rgc_layer_norm_forward(h, m.norm2.weight.data, m.norm2.bias.data)
    want, lse, xph = rgc.rgc_linear_cross_entropy_forward(n2, m.head.weight, y2, m.head.proj)
    assert torch.equal(loss.detach().reshape(-1), want) and bool((loss[:, 0] == 0).all())
    ch, cl = torch.zeros_like(m.head.sketch), torch.zeros_like(m.layer.sketch)
    d2 = rgc.rgc_linear_cross_entropy_backward(n2, m.head.weight, y2, lse, g.reshape(-1), xph, ch)
    dh, dw2, db2 = rgc.rgc_layer_norm_backward(d2, h, m.norm2.weight.data, mu, r2)
    do = rgc.rgc_linear_backward(dh, m.layer.weight, xp, cl)
    dx, dw1, _ = rgc.rgc_layer_norm_backward(do, x2, m.norm1.weight.data, None, r1, bias=False, kind="rms")
    assert torch.equal(m.head.sketch, ch) and torch.equal(m.layer.sketch, cl)
    assert torch.equal(m.norm2.weight.grad, dw2) and torch.equal(m.norm2.bias.grad, db2)
    assert torch.equal(m.norm1.weight.grad, dw1)
    assert torch.equal(x.grad.reshape(-1, k), dh + dx)


def test_gradients_agree_with_64_bits(dev):
    """Against autograd of the same model in float64 on the CPU. About ten tensors on the way are rounded to bf16,
    each by at most 2^-8 of itself; norms and a layer of unit scale pass a relative error on with a factor of
    about one, so 16 * 2^-8 of the norm bounds what adds up."""
    k, V, r = 256, 1000, 32
    m = Model(k, V, r, dev)
    m.begin(5)
    x, y = _batch(dev, 2, 60, k, V, 2)
    x.requires_grad_(True)
    g = torch.randn(y.shape, generator=torch.Generator().manual_seed(3)) / y.numel()
    for _ in range(2):  # two microbatches of the same tokens: everything adds up
        m(x, y).backward(g.to(dev))
    w = {n: p.detach().double().cpu().requires_grad_(True) for n, p in m.named_parameters()}
    x64 = x.detach().double().cpu().requires_grad_(True)
    n1 = x64 / torch.sqrt(x64.square().mean(-1, keepdim=True) + 1e-5) * w["norm1.weight"]
    h = x64 + n1 @ w["layer.weight"].T
    c = h - h.mean(-1, keepdim=True)
    n2 = c / torch.sqrt(c.square().mean(-1, keepdim=True) + 1e-5) * w["norm2.weight"] + w["norm2.bias"]
    z = n2 @ w["head.weight"].T
    live = y.cpu() >= 0
    loss = torch.where(live, torch.logsumexp(z, -1) - z.gather(-1, y.cpu().clamp(min=0)[..., None])[..., 0], 0.0)
    (2 * (loss * g.double()).sum()).backward()

    def close(got, want, what):
        rel = float((got.detach().double().cpu() - want).norm() / want.norm())
        assert rel < 16 * 2.0 ** -8, (what, rel)

    close(x.grad, x64.grad, "x")
    close(m.norm1.weight.grad, w["norm1.weight"].grad, "norm1")
    close(m.norm2.weight.grad, w["norm2.weight"].grad, "norm2")
    close(m.norm2.bias.grad, w["norm2.bias"].grad, "norm2 bias")
    close(m.layer.sketch, w["layer.weight"].grad @ m.layer.proj.double().cpu(), "the layer's sketch")
    close(m.head.sketch, w["head.weight"].grad @ m.head.proj.double().cpu(), "the head's sketch")


@pytest.mark.parametrize("bits", [8, 32])
def test_a_whole_step_runs_and_repeats(dev, bits):
    """Two steps of two microbatches, sketched updates and AdamW; a second run from the same seeds gives the same
    bits, and the weights have moved."""
    runs = []
    for _ in range(2):
        m = Model(128, 520, 16, dev)
        first = [p.detach().clone() for p in m.parameters()]
        opt = AdamW([p for p in m.parameters() if p.requires_grad], lr=1e-2, state_bits=bits, seed=7)
        for step in range(2):
            m.begin(10 * step)
            opt.zero_grad()
            for mb in range(2):
                x, y = _batch(dev, 2, 33, 128, 520, 20 + 2 * step + mb)
                m(x, y).mean().backward()
            norm = torch.stack([p.grad.norm() for p in opt.params]).norm()
            opt.step(grad_scale=torch.clamp(1.0 / (norm + 1e-6), max=1.0).reshape(1))
            m.layer.apply_update(step, tau=1e-2)
            m.head.apply_update(step, tau=1e-2)
        assert all(not torch.equal(a, b) and bool(torch.isfinite(b).all()) for a, b in zip(first, m.parameters()))
        runs.append([p.detach().clone() for p in m.parameters()])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_inputs_that_need_no_gradient_and_broadcast_gradients(dev):
    k, V, r = 64, 104, 16
    head = SketchedCrossEntropy(k, V, r, device=dev)
    head.begin_update(1)
    x, y = _batch(dev, 2, 9, k, V, 4)
    w = head.weight
    # only the sketch is wanted: a parameter of the graph behind the loss asks for it
    s = torch.ones((), device=dev, requires_grad=True)
    x.requires_grad_(True)
    (head(x, y) * s).sum().backward()
    want = head.sketch.clone()
    head.sketch.zero_()
    xd, yd = x.detach().reshape(-1, k), y.reshape(-1)
    _, lse, xp = rgc.rgc_linear_cross_entropy_forward(xd, w, yd, head.proj)
    none = rgc.rgc_linear_cross_entropy_backward(xd, w, yd, lse, torch.ones(18, device=dev), xp, head.sketch, input_grad=False)
    assert none is None and torch.equal(head.sketch, want)
    with pytest.raises(rgc.RgcError):
        rgc.rgc_linear_cross_entropy_backward(xd, w, yd, lse, torch.ones(18, device=dev), input_grad=False)
    norm = LayerNorm(k, device=dev)
    z = x.detach()[:1, :1].expand(2, 9, k).requires_grad_(True)  # rows that are one row
    norm(z).sum().backward()  # and a gradient that is one number
    ref = LayerNorm(k, device=dev)
    zc = z.detach().contiguous().requires_grad_(True)
    ref(zc).backward(torch.ones(2, 9, k, dtype=torch.bfloat16, device=dev))
    assert torch.equal(z.grad, zc.grad) and torch.equal(norm.weight.grad, ref.weight.grad)


def test_optimizer_state_travels(dev):
    """Five steps; or three, a saved and loaded state, and two: the same bits. A parameter without a gradient keeps
    its own step count."""
    def params():
        g = torch.Generator().manual_seed(1)
        return [torch.nn.Parameter(torch.randn(n, generator=g).to(t).to(dev)) for n, t in
                ((300, torch.bfloat16), (77, torch.float32), (4096, torch.bfloat16))]

    def run(opt, lo, hi):
        for t in range(lo, hi):
            for i, p in enumerate(opt.params):
                g = torch.randn(p.shape, generator=torch.Generator().manual_seed(100 * t + i)).to(dev)
                p.grad = None if (i == 1 and t == 1) else g.to(p.dtype)
            opt.step()

    a = AdamW(params(), lr=1e-2, seed=3)
    run(a, 0, 5)
    b = AdamW(params(), lr=1e-2, seed=3)
    run(b, 0, 3)
    c = AdamW([torch.nn.Parameter(p.detach().clone()) for p in b.params], lr=1e-2)
    c.load_state_dict(b.state_dict())
    run(b, 3, 5)
    run(c, 3, 5)
    assert a.state[1]["step"] == 4 and a.state[0]["step"] == 5
    for p, q, r in zip(a.params, b.params, c.params):
        assert torch.equal(p, q) and torch.equal(p, r)
    with pytest.raises(rgc.RgcError):
        AdamW(params(), state_bits=32).load_state_dict(b.state_dict())
    with pytest.raises(rgc.RgcError):
        AdamW([a.params[0], a.params[0]])


def test_a_tensor_listed_twice_is_refused(dev):
    p, g = torch.zeros(64, device=dev), torch.ones(64, device=dev)
    m, v = [torch.zeros(64, device=dev) for _ in range(2)], [torch.zeros(64, device=dev) for _ in range(2)]
    with pytest.raises(rgc.RgcError):
        rgc.rgc_adamw_batch([p, p], [g, g], m, v, 0.1, 1)
    assert bool((p == 0).all())
