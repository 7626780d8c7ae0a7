"""A policy's training step on the operators together: residual norms, a
sketched layer, the head's log probabilities and entropies, a clipped objective
against the rollout's log probabilities (taken from logits), global clipping
and both kinds of update. Gradients against the same model in 64 bits; a captured
step against eager ones."""
import pytest
import torch

from rank_randomized_gradient_amd import AdamW, LayerNorm, SketchedCrossEntropy, SketchedLinear, clip_grad_norm, log_prob, rgc, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


class Policy(torch.nn.Module):
    """A pre-norm block with its stream kept beside it: norm, layer, (addition, norm), head."""

    def __init__(self, k, V, r, dev, seed=0):
        super().__init__()
        self.norm1 = LayerNorm(k, kind="rms", device=dev)
        self.layer = SketchedLinear(k, k, r, device=dev, weight=synth.normal_bf16((k, k), k ** -0.5, seed=seed))
        self.norm2 = LayerNorm(k, kind="rms", device=dev)
        self.layer2 = SketchedLinear(k, k, r, device=dev, weight=synth.normal_bf16((k, k), k ** -0.5, seed=seed + 1))
        self.norm3 = LayerNorm(k, device=dev)
        self.head = SketchedCrossEntropy(k, V, r, device=dev, weight=synth.normal_bf16((V, k), 2 * k ** -0.5, seed=seed + 2))

    def begin(self, seed):
        for i, m in enumerate((self.layer, self.layer2, self.head)):
            m.begin_update(seed + i)

    def update(self, seed):
        for i, m in enumerate((self.layer, self.layer2, self.head)):
            m.apply_update(seed + i, tau=1e-2)

    def hidden(self, x):
        n, s = self.norm2(self.layer(self.norm1(x)), x)
        n, s = self.norm3(self.layer2(n), s)
        return n

    def forward(self, x, tokens):
        return self.head.log_prob(self.hidden(x), tokens)


def objective(logp, entropy, old, advantage, mask):
    ratio = torch.exp(logp - old)
    gain = torch.minimum(ratio * advantage, ratio.clamp(0.8, 1.2) * advantage)
    return -((gain + 0.01 * entropy) * mask).sum() / mask.sum()


def _batch(dev, B, L, k, V, seed):
    x = synth.normal_bf16((B, L, k), 1.0, seed=seed)
    g = torch.Generator().manual_seed(seed)
    y = torch.randint(0, V, (B, L), generator=g)
    y[:, :3] = -100
    adv, noise = torch.randn(B, 1, generator=g), 0.1 * torch.randn(B, L, generator=g)
    return x.to(dev), y.to(dev), adv.to(dev), noise.to(dev)


def test_gradients_agree_with_64_bits(dev):
    """About sixteen tensors on the way are rounded to bf16, each by at most 2^-8 of itself, with factors of about one
    behind them (norms and layers of unit scale), so 24 * 2^-8 of the norm bounds what adds up."""
    k, V, r = 256, 1000, 32
    m = Policy(k, V, r, dev)
    m.begin(5)
    x, y, adv, noise = _batch(dev, 3, 40, k, V, 1)
    x.requires_grad_(True)
    mask = (y >= 0).float()
    with torch.no_grad():
        old = m.forward(x, y)[0] + noise * mask
    objective(*m(x, y), old, adv, mask).backward()
    w = {n: p.detach().double().cpu().requires_grad_(True) for n, p in m.named_parameters()}
    x64 = x.detach().double().cpu().requires_grad_(True)
    rms = lambda h, g: h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-5) * g  # noqa: E731
    s = x64 + rms(x64, w["norm1.weight"]) @ w["layer.weight"].T
    s = s + rms(s, w["norm2.weight"]) @ w["layer2.weight"].T
    n = rms(s - s.mean(-1, keepdim=True), w["norm3.weight"]) + w["norm3.bias"]
    lp = torch.log_softmax(n @ w["head.weight"].T, -1)
    live = y.cpu() >= 0
    logp = torch.where(live, lp.gather(-1, y.cpu().clamp(min=0)[..., None])[..., 0], 0.0)
    ent = torch.where(live, -(lp.exp() * lp).sum(-1), 0.0)
    objective(logp, ent, old.double().cpu(), adv.double().cpu(), mask.double().cpu()).backward()

    def close(got, want, what):
        rel = float((got.detach().double().cpu() - want).norm() / want.norm())
        assert rel < 24 * 2.0 ** -8, (what, rel)

    close(x.grad, x64.grad, "x")
    for name in ("norm1.weight", "norm2.weight", "norm3.weight", "norm3.bias"):
        close(dict(m.named_parameters())[name].grad, w[name].grad, name)
    for name in ("layer", "layer2", "head"):
        mod = getattr(m, name)
        close(mod.sketch, w[name + ".weight"].grad @ mod.proj.double().cpu(), name)


def test_rollout_and_training_agree(dev):
    """The rollout's log probabilities, from the plain head's bf16 logits, and its alternatives, against the training
    forward without logits: the logits' rounding to bf16, at most 2^-9 of their largest, is between the two."""
    k, V, r = 128, 5000, 16
    m = Policy(k, V, r, dev)
    m.begin(1)
    x, y, _, _ = _batch(dev, 2, 30, k, V, 2)
    h = m.hidden(x).detach()
    logits, _ = rgc.rgc_linear_forward(h.reshape(-1, k), m.head.weight)
    a, ea = log_prob(logits.reshape(2, 30, V), y)
    b, eb = (t.detach() for t in m.head.log_prob(h, y))
    off = 2.0 ** -8 * float(logits.float().abs().max())  # of the token's logit, and of lse at most the same
    assert float((a - b).abs().max()) <= off + 1e-4
    # dH is a covariance of log p with the logits' errors: at most their size times the mean of |log p + H|, below 2 H
    assert bool(((ea - eb).abs() <= 0.5 * off * (2 * eb + 1) + 1e-4).all())
    top, ids = m.head.alternatives(h, 4)
    lp = torch.log_softmax(logits.double().reshape(2, 30, V), -1)
    best = torch.sort(logits.float().reshape(2, 30, V), dim=-1, descending=True, stable=True)
    assert torch.equal(ids, best.indices[..., :4])
    assert float((top - lp.gather(-1, ids)).abs().max()) < 1e-4


@pytest.mark.parametrize("in_place", [False, True])
def test_a_whole_step_runs_and_repeats(dev, in_place):
    """Two steps of two microbatches; a second run from the same seeds gives the same bits, and the weights move.
    Clipping as the optimizer reads the gradients or in place before."""
    runs = []
    for _ in range(2):
        m = Policy(128, 520, 16, dev)
        first = [p.detach().clone() for p in m.parameters()]
        opt = AdamW([p for p in m.parameters() if p.requires_grad], lr=1e-2, seed=7)
        norms = []
        for step in range(2):
            m.begin(10 * step)
            opt.zero_grad()
            for mb in range(2):
                x, y, adv, noise = _batch(dev, 2, 33, 128, 520, 20 + 2 * step + mb)
                mask = (y >= 0).float()
                logp, entropy = m(x, y)
                objective(logp, entropy, logp.detach() + noise * mask, adv, mask).backward()
            if in_place:
                norms.append(clip_grad_norm(opt.params, 0.01))
                opt.step()
            else:
                norms.append(opt.step(max_norm=0.01))
            m.update(step)
        assert all(not torch.equal(a, b) and bool(torch.isfinite(b).all()) for a, b in zip(first, m.parameters()))
        runs.append([p.detach().clone() for p in m.parameters()] + norms)
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_calls_captured_and_replayed(dev):
    """The step's calls in one graph, the sketch and the clipped gradients among its outputs, replayed over new inputs
    with eager calls between."""
    T, k, V, r = 90, 128, 1000, 16
    w = synth.normal_bf16((V, k), 2 * k ** -0.5, seed=1).to(dev)
    p = synth.normal_bf16((k, r), 1.0, seed=2).to(dev)
    gain = torch.ones(k, device=dev)
    x, res = (synth.normal_bf16((T, k), 1.0, seed=s).to(dev) for s in (3, 4))
    y = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(5)).to(dev)
    gl, ge = synth.normal_f32((T,), 1.0, seed=6).to(dev), torch.full((T,), -0.01, device=dev)

    def call():
        s, n, _, rstd = rgc.rgc_add_norm_forward(x, res, gain, kind="rms")
        logp, entropy, lse, xp = rgc.rgc_linear_log_prob_forward(n, w, y, p)
        c = torch.zeros(V, r, device=dev)
        dn = rgc.rgc_linear_log_prob_backward(n, w, y, lse, entropy, gl, ge, xp, c)
        dx, dg, _ = rgc.rgc_add_norm_backward(dn, x, s, gain, None, rstd, bias=False, kind="rms")
        norm, scale = rgc.rgc_grad_norm_batch([dg, c], 0.5)
        rgc.rgc_scale_batch([dg, c], scale)
        return logp, entropy, dx, dg, c, norm, scale

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for rep in range(3):
        x.copy_(synth.normal_bf16((T, k), 1.0, seed=10 + rep).to(dev))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, call())), rep
        torch.cuda.synchronize()
