"""The vocabulary head's log probabilities with entropies:
rgc_linear_log_prob_forward and _backward against the same formulas in 64 bits.

Bounds, element by element, u = 2^-24 the fp32 half step. A product of K terms is an
fp32 sum in steps of 32 terms, with at most two roundings a step: off by
u (K / 16 + 16) of the sum of magnitudes (call it dz for a row's logits, at their
largest). exp(d) is off by |d| 2^-22 of itself for its rounded exponent and 2^-21 for
the rest. The sums s = sum exp(z - m) and q = sum exp(z - m) (z - m) take at most 80
roundings one after the other (16 entries of a lane, the lanes, the waves, a tile of
many a lane, the lanes again), so with p the probabilities and d = z - m
  lse: dz + 2^-17 + 2^-22 sum p |d| + 2^-22 (|lse| + |m|)
  H = log s - q / s: 2^-16 (1 + sum p (|d| + d^2)) + 2 dz (1 + H)
(dH / dz_v = -p_v (log p_v + H), whose magnitudes sum to 2 H at most). D = p f + gl
[v = y], f = -gl - ge (log p + H): p's relative error is dz + lse's + 2^-21 + 2^-21
|log p|, f is off by |ge| (dz + lse's + H's) + 2^-22 (|gl| + |ge| (|log p| + H)). As two bf16 terms D is
off by 2^-16 of itself more. dX and C add their sums' errors, and dX its rounding, half a step of bf16 (2^-8).
"""
import pytest
import torch

from rank_randomized_gradient_amd import SketchedCrossEntropy, rgc, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _inputs(T, V, k, r, seed, ignored=0.1, spread=2.0):
    x = synth.normal_bf16((T, k), 1.0, seed=seed)
    w = synth.normal_bf16((V, k), spread / k ** 0.5, seed=seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    y = torch.randint(0, V, (T,), generator=g)
    y[torch.rand(T, generator=g) < ignored] = -100
    gl, ge = synth.normal_f32((T,), 1.0, seed=seed + 3), synth.normal_f32((T,), 0.3, seed=seed + 6)
    xp = synth.normal_bf16((T, r), 3.0, seed=seed + 4) if r else None
    c = synth.normal_f32((V, r), 1e-3, seed=seed + 5) if r else None
    return x, w, y, gl, ge, xp, c


def _steps(K):
    return (K / 16 + 16) * 2.0 ** -24


def _reference(x, w, y, gl, ge, xp, c):
    T, V = len(x), len(w)
    x, w = x.double(), w.double()
    zero = torch.zeros(T, dtype=torch.float64)
    gl, ge = (zero if g is None else g.double() for g in (gl, ge))
    z = x @ w.T
    live = (y >= 0) & (y < V)
    at = torch.where(live, y, 0)
    gl, ge = torch.where(live, gl, 0.0), torch.where(live, ge, 0.0)
    m = z.amax(1)
    d = z - m[:, None]
    lse = torch.logsumexp(z, 1)
    lp = z - lse[:, None]
    p = torch.exp(lp)
    H = -(p * lp).sum(1)
    rows = torch.arange(T)
    dz = _steps(x.shape[1]) * (x.abs() @ w.abs().T).amax(1)
    e_lse = dz + 2.0 ** -17 + 2.0 ** -22 * ((p * d.abs()).sum(1) + lse.abs() + m.abs())
    e_h = 2.0 ** -16 * (1 + (p * (d.abs() + d * d)).sum(1)) + 2 * dz * (1 + H)
    out = {"lse": lse, "logp": torch.where(live, lp[rows, at], 0.0), "entropy": torch.where(live, H, 0.0)}
    bound = {"lse": e_lse, "logp": dz + e_lse + 2.0 ** -22 * (lse.abs() + z.abs().amax(1)), "entropy": e_h}
    f = -gl[:, None] - ge[:, None] * (lp + H[:, None])
    D = p * f
    size = gl.abs()[:, None] + ge.abs()[:, None] * (lp.abs() + H[:, None])
    off = p * (size * ((dz + e_lse)[:, None] + 2.0 ** -20 + 2.0 ** -21 * lp.abs()) + (ge.abs() * (dz + e_lse + e_h))[:, None])
    D[rows, at] += gl
    off = off + 2.0 ** -16 * D.abs() + 1e-37  # (and what exp flushes to zero)
    out["dX"] = D @ w
    bound["dX"] = (off + _steps(V) * D.abs()) @ w.abs() + 2.0 ** -8 * out["dX"].abs()
    if c is not None:
        xa = torch.where(live[:, None], xp.double(), 0.0)
        out["C"] = c.double() + D.T @ xa
        bound["C"] = (off + _steps(2 * T) * D.abs()).T @ xa.abs() + 2.0 ** -22 * c.double().abs()
    return out, bound


def _check(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    excess = (got.double().cpu() - want).abs() - bound
    assert excess.numel() == 0 or float(excess.max()) <= 1e-30, f"{what}: {float(excess.max()):.3e} over the bound"


def _to(dev, *ts):
    return [None if t is None else t.to(dev) for t in ts]


def _run(dev, T, V, k, r, seed, **kw):
    x, w, y, gl, ge, xp, c = _inputs(T, V, k, r, seed, **kw)
    want, bound = _reference(x, w, y, gl, ge, xp, c)
    xg, wg, yg, glg, geg, xpg, cg = _to(dev, x, w, y, gl, ge, xp, c)
    logp, entropy, lse, none = rgc.rgc_linear_log_prob_forward(xg, wg, yg)
    assert none is None
    dx = rgc.rgc_linear_log_prob_backward(xg, wg, yg, lse, entropy, glg, geg, xpg, cg)
    torch.cuda.synchronize()
    what = f"T={T} V={V} k={k} r={r}"
    for name, got in (("lse", lse), ("logp", logp), ("entropy", entropy), ("dX", dx)):
        _check(got, want[name], bound[name], f"{name} {what}")
    assert bool((logp.cpu()[y < 0] == 0).all()) and bool((entropy.cpu()[y < 0] == 0).all())
    assert bool((dx.cpu()[y < 0] == 0).all()) and bool((entropy >= 0).all())
    if r:
        _check(cg, want["C"], bound["C"], f"C {what}")


# one token, one entry; K ending anywhere in a step; every kind of tile (64, 128 and 256 rows, pairs) and of rank; more
# entries than one piece; rounds of large tiles with small ones behind
SHAPES = [(1, 1, 8, 0), (1, 8, 8, 8), (2, 7, 16, 0), (24, 1000, 64, 16), (300, 777, 520, 0), (257, 2056, 72, 4),
          (513, 264, 1000, 8), (129, 1025, 136, 0), (255, 17, 264, 0), (64, 4104, 2048, 128), (33, 70008, 64, 16),
          (5, 70001, 24, 0), (65, 1000, 72, 4), (100, 2056, 136, 48), (128, 520, 264, 256), (7, 1288, 264, 240),
          (100, 33000, 72, 0), (300, 20001, 136, 0), (520, 11016, 136, 16), (700, 24008, 72, 4), (1025, 16385, 72, 0)]


@pytest.mark.parametrize("T,V,k,r", SHAPES)
def test_against_64_bits(dev, T, V, k, r):
    print(T, V, k, r, flush=True)
    _run(dev, T, V, k, r, seed=100 + T + V)


@pytest.mark.parametrize("spread", [0.0, 0.01, 12.0])
def test_flat_and_peaked(dev, spread):
    """Entropies from log V to nearly nothing."""
    _run(dev, 200, 3000, 64, 16, seed=3, spread=spread)


def test_more_tokens_than_the_stacked_terms_hold(dev):
    _run(dev, 33000, 72, 32, 16, seed=7)


@pytest.mark.parametrize("which", ["logp", "entropy"])
def test_one_gradient_alone(dev, which):
    x, w, y, gl, ge, xp, c = _inputs(150, 1032, 72, 16, 21)
    gl, ge = (gl, None) if which == "logp" else (None, ge)
    want, bound = _reference(x, w, y, gl, ge, xp, c)
    xg, wg, yg, glg, geg, xpg, cg = _to(dev, x, w, y, gl, ge, xp, c)
    _, entropy, lse, _ = rgc.rgc_linear_log_prob_forward(xg, wg, yg)
    dx = rgc.rgc_linear_log_prob_backward(xg, wg, yg, lse, None if which == "logp" else entropy, glg, geg, xpg, cg)
    _check(dx, want["dX"], bound["dX"], "dX")
    _check(cg, want["C"], bound["C"], "C")
    c2 = c.to(dev)
    assert rgc.rgc_linear_log_prob_backward(xg, wg, yg, lse, entropy, glg, geg, xpg, c2, input_grad=False) is None
    _check(c2, want["C"], bound["C"], "C alone")


def test_log_probability_is_the_loss_negated(dev):
    """The same tiles and joins in the same order: lse and, negated, the losses, bit for bit, and their gradient."""
    x, w, y, gl, _, xp, c = _inputs(300, 5000, 136, 16, 31)
    xg, wg, yg, gg, xpg = _to(dev, x, w, y, gl, xp)
    loss, lse0, _ = rgc.rgc_linear_cross_entropy_forward(xg, wg, yg)
    logp, entropy, lse, _ = rgc.rgc_linear_log_prob_forward(xg, wg, yg)
    assert torch.equal(lse, lse0) and torch.equal(-logp, loss)
    a, b = c.to(dev), c.to(dev)
    dx0 = rgc.rgc_linear_cross_entropy_backward(xg, wg, yg, lse, -gg, xpg, a)
    dx = rgc.rgc_linear_log_prob_backward(xg, wg, yg, lse, entropy, gg, None, xpg, b)
    assert torch.equal(dx, dx0) and torch.equal(a, b)


@pytest.mark.parametrize("r", [0, 4, 16])
def test_ignored_tokens_may_hold_anything(dev, r):
    T, V, k = 70, 520, 72
    x, w, y, gl, ge, xp, c = _inputs(T, V, k, r, 11, ignored=0.0)
    y[::3] = -1
    y[1::9] = V
    y[4::9] = 2 ** 40
    out = (y < 0) | (y >= V)
    want, bound = _reference(x, w, y, gl, ge, xp, c)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")])[torch.arange(T) % 3]
    x[out] = bad[out, None].to(torch.bfloat16)
    gl[out] = bad[out]
    ge[out] = -bad[out]
    if r:
        xp[out] = bad[out, None].to(torch.bfloat16)
    xg, wg, yg, glg, geg, xpg, cg = _to(dev, x, w, y, gl, ge, xp, c)
    logp, entropy, lse, _ = rgc.rgc_linear_log_prob_forward(xg, wg, yg)
    dx = rgc.rgc_linear_log_prob_backward(xg, wg, yg, lse, entropy, glg, geg, xpg, cg)
    for name, got in (("logp", logp), ("entropy", entropy), ("dX", dx)):
        _check(got, want[name], bound[name], name)
        assert bool((got.cpu()[out] == 0).all())
    if r:
        _check(cg, want["C"], bound["C"], "C")


def test_nan_reaches_only_its_token(dev):
    T, V, k = 20, 600, 64
    x, w, y, gl, ge, _, _ = _inputs(T, V, k, 0, 12, ignored=0.0)
    want, bound = _reference(x, w, y, gl, ge, None, None)
    x[5, 3] = float("nan")
    xg, wg, yg, glg, geg = _to(dev, x, w, y, gl, ge)
    logp, entropy, lse, _ = rgc.rgc_linear_log_prob_forward(xg, wg, yg)
    dx = rgc.rgc_linear_log_prob_backward(xg, wg, yg, lse, entropy, glg, geg)
    assert torch.isnan(logp[5]) and torch.isnan(entropy[5]) and torch.isnan(lse[5]) and torch.isnan(dx[5]).all()
    rest = torch.arange(T) != 5
    for name, got in (("logp", logp), ("entropy", entropy), ("dX", dx)):
        _check(got.cpu()[rest], want[name][rest], bound[name][rest], name)


def test_extreme_logits(dev):
    """Logits of +-1e4 (a saturated softmax) stay finite, and an entry at -inf has no part in the entropy."""
    k, V = 8, 300
    x, w = torch.zeros(3, k), torch.zeros(V, k)
    x[:, 0] = torch.tensor([100.0, -100.0, 1.0])
    w[:, 0] = torch.linspace(-100, 100, V)
    x, w = x.bfloat16(), w.bfloat16()
    y, g = torch.tensor([V - 1, V - 1, 5]), torch.ones(3)
    want, bound = _reference(x, w, y, g, g, None, None)
    xg, wg, yg, gg = _to(dev, x, w, y, g)
    logp, entropy, lse, _ = rgc.rgc_linear_log_prob_forward(xg, wg, yg)
    dx = rgc.rgc_linear_log_prob_backward(xg, wg, yg, lse, entropy, gg, gg)
    for name, got in (("logp", logp), ("entropy", entropy), ("dX", dx)):
        _check(got, want[name], bound[name], name)
    w = torch.zeros(V, k).bfloat16()
    w[7, 0] = -float("inf")
    logp, entropy, lse, _ = rgc.rgc_linear_log_prob_forward(torch.ones(2, k).bfloat16().to(dev), w.to(dev),
                                                            torch.tensor([3, 7]).to(dev))
    ref = float(torch.log(torch.tensor(V - 1.0, dtype=torch.float64)))
    assert abs(float(entropy[0]) - ref) < 1e-5 and abs(float(logp[0]) + ref) < 1e-5 and float(logp[1]) == -float("inf")


def test_gradient_agrees_with_differences(dev):
    """Both outputs' change along dX, by central differences of the forward."""
    T, V, k = 8, 300, 64
    x, w, y, gl, ge, _, _ = _inputs(T, V, k, 0, 18, ignored=0.0)
    xq = ((x.float().clamp(-1, 1) * 256).round() / 256).bfloat16()  # steps of 1/8 are exact then
    wg, yg, glg, geg = _to(dev, w, y, gl, ge)
    _, entropy, lse, _ = rgc.rgc_linear_log_prob_forward(xq.to(dev), wg, yg)
    dx = rgc.rgc_linear_log_prob_backward(xq.to(dev), wg, yg, lse, entropy, glg, geg).double().cpu()
    for t, i in ((0, 3), (5, 60), (7, 0)):
        sides = []
        for step in (0.125, -0.125):
            xs = xq.clone()
            xs[t, i] = float(xs[t, i]) + step
            logp, ent, _, _ = rgc.rgc_linear_log_prob_forward(xs.to(dev), wg, yg)
            value = (logp.double().cpu() * gl.double() + ent.double().cpu() * ge.double()).sum()
            sides.append((float(value), float(xs[t, i])))
        h = (sides[0][1] - sides[1][1]) / 2
        slope = (sides[0][0] - sides[1][0]) / (2 * h)
        # third derivatives along one element: of logp a third cumulant of W[:, i] under p, of the entropy (its
        # derivative is a covariance of log p with W[:, i]) a sum of cumulants up to the fourth with one log p, each
        # at most (2 w)^3 times 1 and 6 (L + log V), L the spread of log p, which is below 2 log V + 8 here
        wm, lv = float(w[:, i].abs().max()), float(torch.log(torch.tensor(float(V))))
        third = (2 * wm) ** 3 * (abs(float(gl[t])) + abs(float(ge[t])) * 6 * (3 * lv + 8))
        tol = third * h * h / 6 + 2.0 ** -7 * abs(slope) + 2.0 ** -8 * (abs(float(gl[t])) + abs(float(ge[t])) * 8) * wm
        assert abs(slope - float(dx[t, i])) <= tol, (t, i, slope, float(dx[t, i]), tol)


def test_strided_operands_and_what_lies_around_them(dev):
    T, V, k, r = 301, 1032, 200, 16
    x, w, y, gl, ge, xp, c = _inputs(T, V, k, r, 13)
    want, bound = _reference(x, w, y, gl, ge, xp, c)
    xf = torch.full((T, k + 24), float("nan"), dtype=torch.bfloat16, device=dev)
    wf = torch.full((V, k + 8), float("nan"), dtype=torch.bfloat16, device=dev)
    df = torch.full((T + 2, k + 16), 5.0, dtype=torch.bfloat16, device=dev)
    cf = torch.full((V + 2, r), 7.0, device=dev)
    xf[:, 8:8 + k], wf[:, :k], cf[1:-1] = x.to(dev), w.to(dev), c.to(dev)
    xs, ws, ds = xf[:, 8:8 + k], wf[:, :k], df[1:-1, 8:8 + k]
    yg, glg, geg, xpg = _to(dev, y, gl, ge, xp)
    _, entropy, lse, _ = rgc.rgc_linear_log_prob_forward(xs, ws, yg)
    rgc.rgc_linear_log_prob_backward(xs, ws, yg, lse, entropy, glg, geg, xpg, cf[1:-1], dX=ds)
    _check(entropy, want["entropy"], bound["entropy"], "entropy")
    _check(ds, want["dX"], bound["dX"], "dX")
    _check(cf[1:-1], want["C"], bound["C"], "C")
    assert bool((df[0] == 5).all()) and bool((df[-1] == 5).all())
    assert bool((df[:, :8] == 5).all()) and bool((df[:, 8 + k:] == 5).all())
    assert bool((cf[0] == 7).all()) and bool((cf[-1] == 7).all())


def test_forward_makes_xp_as_the_project_does(dev):
    x, w, y = _to(dev, *_inputs(300, 520, 264, 0, 14)[:3])
    p = synth.normal_bf16((264, 16), 1.0, seed=15).to(dev)
    assert torch.equal(rgc.rgc_linear_log_prob_forward(x, w, y, p)[3], rgc.rgc_project(x, p))


def _both(st):
    x, w, y, gl, ge, xp, c = st
    cg = c.clone() if c is not None else None
    logp, entropy, lse, _ = rgc.rgc_linear_log_prob_forward(x, w, y)
    return logp, entropy, rgc.rgc_linear_log_prob_backward(x, w, y, lse, entropy, gl, ge, xp, cg), cg


def _same(a, b):
    return all(p is None and q is None or torch.equal(p, q) for p, q in zip(a, b))


def test_captured_and_replayed(dev):
    """Two graphs, replayed in turn with eager calls between, each replay with new inputs."""
    jobs = []
    for T, V, k, r in [(200, 1000, 136, 16), (90, 2000, 136, 0)]:
        st = _to(dev, *_inputs(T, V, k, r, 19))
        _both(st)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = _both(st)
        jobs.append((st, graph, outs))
    for rep in range(3):
        for n, (st, graph, outs) in enumerate(jobs):
            st[0].copy_(synth.normal_bf16(tuple(st[0].shape), 1.0, seed=50 + 7 * rep + n).to(dev))
            graph.replay()
        torch.cuda.synchronize()
        for st, graph, outs in jobs:
            assert _same(outs, _both(st)), rep


def test_two_streams_at_once(dev):
    jobs = [_to(dev, *_inputs(300, 3000, 264, r, 60 + r)) for r in (0, 16)]
    want = [_both(j) for j in jobs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(4):
        for n in (0, 1):
            with torch.cuda.stream(streams[n]):
                got[n].append(_both(jobs[n]))
    torch.cuda.synchronize()
    for n in (0, 1):
        assert all(_same(g, want[n]) for g in got[n])


# ---- the module ---------------------------------------------------------------

def _head(dev, k, V, r, seed):
    w = synth.normal_bf16((V, k), 2.0 / k ** 0.5, seed=seed)
    head = SketchedCrossEntropy(k, V, r, kind="rademacher", device=dev, weight=w)
    head.begin_update(5)
    return head, w


@pytest.mark.parametrize("leaf", [True, False])
def test_module_gradients(dev, leaf):
    """A policy's loss through log_prob: x's gradient and the sketch are the calls', whether or not x needs one."""
    B, L, k, V, r = 3, 17, 72, 1032, 16
    head, w = _head(dev, k, V, r, 1)
    x = synth.normal_bf16((B, L, k), 1.0, seed=2).to(dev).requires_grad_(leaf)
    y = torch.randint(0, V, (B, L), generator=torch.Generator().manual_seed(3)).to(dev)
    y[0, :5] = -100
    adv = synth.normal_f32((B, L), 1.0, seed=4).to(dev)
    logp, entropy = head.log_prob(x, y)
    assert logp.shape == entropy.shape == (B, L)
    (-(logp * adv).sum() - 0.01 * entropy.sum()).backward()
    x2, y2 = x.detach().reshape(-1, k), y.reshape(-1)
    a, e, lse, xp = rgc.rgc_linear_log_prob_forward(x2, w.to(dev), y2, head.proj)
    c = torch.zeros(V, r, device=dev)
    dx = rgc.rgc_linear_log_prob_backward(x2, w.to(dev), y2, lse, e, -adv.reshape(-1), torch.full((B * L,), -0.01, device=dev), xp, c)
    assert torch.equal(logp.reshape(-1), a) and torch.equal(entropy.reshape(-1), e) and torch.equal(head.sketch, c)
    assert (x.grad is None) if not leaf else torch.equal(x.grad.reshape(-1, k), dx)


def test_module_one_output_used(dev):
    head, w = _head(dev, 64, 520, 8, 6)
    x = synth.normal_bf16((9, 64), 1.0, seed=7).to(dev).requires_grad_()
    y = torch.arange(9, device=dev)
    head.log_prob(x, y)[1].sum().backward()
    _, e, lse, xp = rgc.rgc_linear_log_prob_forward(x.detach(), w.to(dev), y, head.proj)
    c = torch.zeros(520, 8, device=dev)
    dx = rgc.rgc_linear_log_prob_backward(x.detach(), w.to(dev), y, lse, e, None, torch.ones(9, device=dev), xp, c)
    assert torch.equal(x.grad, dx) and torch.equal(head.sketch, c)


def test_module_alternatives(dev):
    """Of the plain head's bf16 logits, rows in pieces or not."""
    head, w = _head(dev, 64, 70008, 8, 8)
    x = synth.normal_bf16((2, 1003, 64), 1.0, seed=9).to(dev)  # 2006 rows: more than a piece of 1917
    logp, ids = head.alternatives(x, 5)
    z, _ = rgc.rgc_linear_forward(x.reshape(-1, 64), w.to(dev))
    # (a row's sums are joined in another order in a call of few rows, so the pieces are the module's)
    a, b = (torch.cat(t) for t in zip(*[rgc.rgc_log_prob_forward(p, top=5)[3:] for p in (z[:1917], z[1917:])]))
    assert torch.equal(b, rgc.rgc_log_prob_forward(z, top=5)[4])
    assert ids.shape == (2, 1003, 5) and torch.equal(ids.reshape(-1, 5), b) and torch.equal(logp.reshape(-1, 5), a)
