"""The vocabulary head's loss: rgc_linear_cross_entropy_forward and _backward
against the same formulas in 64 bits.

Bounds, element by element. A logit is an fp32 sum of exact products of bf16:
it is off by at most 2^-20 of A = sum |x w| (as for the layer products). lse
inherits the largest logit error of its row (it is a weighted mean of them),
plus a few fp32 roundings of values of the size of lse; loss is lse minus one
logit. D = g (p - [v = y]) then is off by p |g| times the two logit errors in
its exponent, and rounded to bf16 for dX (half a step, 2^-8 of D) except at the
targets, whose rest is added in fp32; dX adds its own rounding (2^-8) and the
fp32 sum (2^-20 of sum |D W|). For C, D's two bf16 terms leave 2^-16 of D.
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


def _inputs(T, V, k, r, seed, ignored=0.1):
    x = synth.normal_bf16((T, k), 1.0, seed=seed)
    w = synth.normal_bf16((V, k), 2.0 / k ** 0.5, seed=seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    y = torch.randint(0, V, (T,), generator=g)
    y[torch.rand(T, generator=g) < ignored] = -100
    gr = synth.normal_f32((T,), 1.0, seed=seed + 3)
    xp = synth.normal_bf16((T, r), 3.0, seed=seed + 4) if r else None
    c = synth.normal_f32((V, r), 1e-3, seed=seed + 5) if r else None
    return x, w, y, gr, xp, c


def _reference(x, w, y, gr, xp, c):
    x, w, gr = x.double(), w.double(), gr.double()
    z = x @ w.T
    live = (y >= 0) & (y < w.shape[0])
    at = torch.where(live, y, 0)
    lse = torch.logsumexp(z, 1)
    loss = torch.where(live, lse - z.gather(1, at[:, None])[:, 0], torch.zeros(()).double())
    p = torch.exp(z - lse[:, None])
    dz = 2.0 ** -20 * (x.abs() @ w.abs().T).amax(1)  # a row's largest logit error
    d = p.clone()
    d[torch.arange(len(y)), at] -= 1
    gl = torch.where(live, gr, torch.zeros(()).double())
    d = d * gl[:, None]
    off = (2 * dz + 2.0 ** -20)[:, None] * p * gl.abs()[:, None]  # of D, before any rounding to bf16
    rounded = d.abs()  # entries that dX takes rounded to bf16: all but the targets'
    rounded[torch.arange(len(y)), at] = 0
    out = {"lse": lse, "loss": loss, "dX": d @ w}
    few = 2.0 ** -21 * (lse.abs() + z.abs().amax(1) + 1)
    bound = {"lse": dz + few, "loss": 2 * dz + 2 * few,
             "dX": (off + 2.0 ** -8 * rounded + 2.0 ** -20 * d.abs()) @ w.abs() + 2.0 ** -8 * (d @ w).abs()}
    if c is not None:
        xa = xp.double()
        xa = torch.where(live[:, None], xa, torch.zeros(()).double())
        out["C"] = c.double() + d.T @ xa
        bound["C"] = (off + (2.0 ** -16 + 2.0 ** -20) * d.abs()).T @ xa.abs() + 2.0 ** -22 * c.double().abs()
    return out, bound


def _check(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    excess = (got.double().cpu() - want).abs() - bound
    assert excess.numel() == 0 or float(excess.max()) <= 1e-30, f"{what}: {float(excess.max()):.3e} over the bound"


def _run(dev, T, V, k, r, seed, **kw):
    x, w, y, gr, xp, c = _inputs(T, V, k, r, seed, **kw)
    want, bound = _reference(x, w, y, gr, xp, c)
    xg, wg, yg = x.to(dev), w.to(dev), y.to(dev)
    cg = c.to(dev) if r else None
    loss, lse, none = rgc.rgc_linear_cross_entropy_forward(xg, wg, yg)
    assert none is None
    dx = rgc.rgc_linear_cross_entropy_backward(xg, wg, yg, lse, gr.to(dev), xp.to(dev) if r else None, cg)
    torch.cuda.synchronize()
    what = f"T={T} V={V} k={k} r={r}"
    _check(lse, want["lse"], bound["lse"], f"lse {what}")
    _check(loss, want["loss"], bound["loss"], f"loss {what}")
    _check(dx, want["dX"], bound["dX"], f"dX {what}")
    assert bool((loss.cpu()[y < 0] == 0).all()) and bool((dx.cpu()[y < 0] == 0).all())
    if r:
        _check(cg, want["C"], bound["C"], f"C {what}")
        # the targets' entries carry most of C and are exact to fp32: far below one bf16 term's 2^-9
        rel = float((cg.double().cpu() - want["C"]).norm() / want["C"].norm())
        assert rel < 2.0 ** -18, (what, rel)


# one token, one entry; widths of one 16-byte chunk; K of the logits (k) and of dX (V) ending anywhere in a step of
# 64; tiles ending anywhere; every kind of rank; more entries than one piece of the vocabulary; one tile of tokens
# (up to 64, up to 128), which makes its own part of the sketch, and one more
SHAPES = [(1, 1, 8, 0), (1, 8, 8, 8), (2, 7, 16, 0), (24, 1000, 64, 16), (300, 777, 520, 0), (257, 2056, 72, 4),
          (513, 264, 1000, 8), (129, 1025, 136, 0), (255, 17, 264, 0), (256, 256, 256, 256), (64, 4104, 2048, 128),
          (1000, 1048, 200, 48), (33, 70008, 64, 16), (5, 70001, 24, 0), (65, 1000, 72, 4), (100, 2056, 136, 48),
          (128, 520, 264, 256), (129, 1000, 64, 16), (7, 1288, 264, 240)]


@pytest.mark.parametrize("T,V,k,r", SHAPES)
def test_against_64_bits(dev, T, V, k, r):
    print(T, V, k, r, flush=True)
    _run(dev, T, V, k, r, seed=100 + T + V)


# two workgroups to a compute unit (more 128 x 128 tiles than compute units, no larger ones): one row of tiles, three,
# six; more than two rounds of them at a width where the forward takes the other form
@pytest.mark.parametrize("T,V,k,r", [(100, 33000, 72, 0), (300, 20001, 136, 0), (700, 9000, 72, 8), (66, 65800, 1032, 0)])
def test_tiles_in_pairs(dev, T, V, k, r):
    print(T, V, k, r, flush=True)
    _run(dev, T, V, k, r, seed=500 + T + V)


# 256 x 256 tiles alone (129 and 144 of them), and rounds of them with small tiles behind (on 256 compute units)
@pytest.mark.parametrize("T,V,k,r", [(520, 11016, 136, 16), (2100, 4001, 264, 0), (700, 24008, 72, 4), (1025, 16385, 72, 0)])
def test_large_tiles_against_64_bits(dev, T, V, k, r):
    print(T, V, k, r, flush=True)
    _run(dev, T, V, k, r, seed=T + V)


@pytest.mark.parametrize("left", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64])
def test_every_kind_of_last_step(dev, left):
    """dX's K ends `left` rows into a step of 64; the logits' K likewise where a layer's width allows it."""
    print(left, flush=True)
    _run(dev, 40, 128 + left, 64 + 8 * ((left + 7) // 8), 0, seed=left)


def test_more_tokens_than_the_stacked_terms_hold(dev):
    _run(dev, 33000, 72, 32, 16, seed=7)


def test_no_tokens(dev):
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=dev)
    w = synth.normal_bf16((100, 64), 1.0, seed=1).to(dev)
    y = torch.zeros(0, dtype=torch.int64, device=dev)
    e = torch.zeros(0, device=dev)
    loss, lse, _ = rgc.rgc_linear_cross_entropy_forward(x, w, y)
    dx = rgc.rgc_linear_cross_entropy_backward(x, w, y, lse, e)
    assert loss.shape == lse.shape == (0,) and dx.shape == (0, 64)


@pytest.mark.parametrize("r", [0, 4, 16])
def test_ignored_tokens_may_hold_anything(dev, r):
    """Ignored tokens (negative targets, targets behind the vocabulary) with Inf and NaN in their rows of X and
    XP and in their grad: no loss, zero gradients, and the other tokens as without them. All tokens ignored too."""
    T, V, k = 70, 520, 72
    x, w, y, gr, xp, c = _inputs(T, V, k, r, 11, ignored=0.0)
    y[::3] = -1
    y[1::9] = V
    y[4::9] = 2 ** 40
    out = (y < 0) | (y >= V)
    want, bound = _reference(x, w, y, gr, xp, c)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")])[torch.arange(T) % 3]
    x[out] = bad[out, None].to(torch.bfloat16)
    gr[out] = bad[out]
    if r:
        xp[out] = bad[out, None].to(torch.bfloat16)
    cg = c.to(dev) if r else None
    loss, lse, _ = rgc.rgc_linear_cross_entropy_forward(x.to(dev), w.to(dev), y.to(dev))
    dx = rgc.rgc_linear_cross_entropy_backward(x.to(dev), w.to(dev), y.to(dev), lse, gr.to(dev),
                                               xp.to(dev) if r else None, cg)
    _check(loss, want["loss"], bound["loss"], "loss")
    _check(dx, want["dX"], bound["dX"], "dX")
    assert bool((loss.cpu()[out] == 0).all()) and bool((dx.cpu()[out] == 0).all())
    if r:
        _check(cg, want["C"], bound["C"], "C")
    none = torch.full((T,), -100, device=dev)
    loss, lse, _ = rgc.rgc_linear_cross_entropy_forward(x.to(dev), w.to(dev), none)
    c2 = c.to(dev) if r else None
    dx = rgc.rgc_linear_cross_entropy_backward(x.to(dev), w.to(dev), none, lse, gr.to(dev), xp.to(dev) if r else None, c2)
    assert bool((loss == 0).all()) and bool((dx == 0).all())
    if r:
        assert torch.equal(c2.cpu(), c)


def test_infinite_and_extreme_logits(dev):
    """Logits of +-1e4 (a saturated softmax) stay finite; a vocabulary entry at -Inf has no probability."""
    k, V = 8, 300
    x = torch.zeros(3, k)
    x[:, 0] = torch.tensor([100.0, -100.0, 1.0])
    w = torch.zeros(V, k)
    w[:, 0] = torch.linspace(-100, 100, V)
    x, w = x.bfloat16(), w.bfloat16()
    y = torch.tensor([V - 1, V - 1, 5])
    want, bound = _reference(x, w, y, torch.ones(3), None, None)
    loss, lse, _ = rgc.rgc_linear_cross_entropy_forward(x.to(dev), w.to(dev), y.to(dev))
    dx = rgc.rgc_linear_cross_entropy_backward(x.to(dev), w.to(dev), y.to(dev), lse, torch.ones(3, device=dev))
    _check(lse, want["lse"], bound["lse"], "lse")
    _check(loss, want["loss"], bound["loss"], "loss")
    _check(dx, want["dX"], bound["dX"], "dX")
    x = torch.ones(2, k).bfloat16()
    w = torch.zeros(V, k).bfloat16()
    w[7, 0] = -float("inf")
    loss, lse, _ = rgc.rgc_linear_cross_entropy_forward(x.to(dev), w.to(dev), torch.tensor([3, 7]).to(dev))
    ref = torch.log(torch.tensor(V - 1.0, dtype=torch.float64))
    assert abs(float(lse[0]) - float(ref)) < 1e-6 and abs(float(loss[0]) - float(ref)) < 1e-6
    assert float(loss[1]) == float("inf")


def test_nan_reaches_only_its_token(dev):
    T, V, k = 20, 600, 64
    x, w, y, gr, _, _ = _inputs(T, V, k, 0, 12, ignored=0.0)
    want, bound = _reference(x, w, y, gr, None, None)
    x[5, 3] = float("nan")
    loss, lse, _ = rgc.rgc_linear_cross_entropy_forward(x.to(dev), w.to(dev), y.to(dev))
    dx = rgc.rgc_linear_cross_entropy_backward(x.to(dev), w.to(dev), y.to(dev), lse, gr.to(dev))
    assert torch.isnan(loss[5]) and torch.isnan(lse[5]) and torch.isnan(dx[5]).all()
    rest = torch.arange(T) != 5
    _check(loss.cpu()[rest], want["loss"][rest], bound["loss"][rest], "loss")
    _check(dx.cpu()[rest], want["dX"][rest], bound["dX"][rest], "dX")


def test_strided_operands_and_what_lies_around_them(dev):
    T, V, k, r = 301, 1032, 200, 16
    x, w, y, gr, xp, c = _inputs(T, V, k, r, 13)
    want, bound = _reference(x, w, y, gr, xp, c)
    xf = torch.full((T, k + 24), float("nan"), dtype=torch.bfloat16, device=dev)
    wf = torch.full((V, k + 8), float("nan"), dtype=torch.bfloat16, device=dev)
    df = torch.full((T + 2, k + 16), 5.0, dtype=torch.bfloat16, device=dev)
    cf = torch.full((V + 2, r), 7.0, device=dev)
    xf[:, 8:8 + k] = x.to(dev)
    wf[:, :k] = w.to(dev)
    cf[1:-1] = c.to(dev)
    xs, ws, ds = xf[:, 8:8 + k], wf[:, :k], df[1:-1, 8:8 + k]
    loss, lse, _ = rgc.rgc_linear_cross_entropy_forward(xs, ws, y.to(dev))
    rgc.rgc_linear_cross_entropy_backward(xs, ws, y.to(dev), lse, gr.to(dev), xp.to(dev), cf[1:-1], dX=ds)
    _check(loss, want["loss"], bound["loss"], "loss")
    _check(ds, want["dX"], bound["dX"], "dX")
    _check(cf[1:-1], want["C"], bound["C"], "C")
    assert bool((df[0] == 5).all()) and bool((df[-1] == 5).all())
    assert bool((df[:, :8] == 5).all()) and bool((df[:, 8 + k:] == 5).all())
    assert bool((cf[0] == 7).all()) and bool((cf[-1] == 7).all())


@pytest.mark.parametrize("r", [4, 16, 128])
def test_forward_makes_xp_as_the_project_does(dev, r):
    x, w, y, _, _, _ = _inputs(300, 520, 264, 0, 14)
    p = synth.normal_bf16((264, r), 1.0, seed=15).to(dev)
    _, _, xp = rgc.rgc_linear_cross_entropy_forward(x.to(dev), w.to(dev), y.to(dev), p)
    assert torch.equal(xp, rgc.rgc_project(x.to(dev), p))


def test_same_target_for_every_token(dev):
    """All tokens' largest entries of D fall on one row of C, added in token order."""
    T, V, k, r = 700, 264, 264, 256
    x, w, y, gr, xp, c = _inputs(T, V, k, r, 16, ignored=0.0)
    y[:] = 17
    want, bound = _reference(x, w, y, gr, xp, c)
    cg = c.to(dev)
    _, lse, _ = rgc.rgc_linear_cross_entropy_forward(x.to(dev), w.to(dev), y.to(dev))
    rgc.rgc_linear_cross_entropy_backward(x.to(dev), w.to(dev), y.to(dev), lse, gr.to(dev), xp.to(dev), cg)
    _check(cg, want["C"], bound["C"], "C")


def test_repeated_calls_give_the_same_bits(dev):
    x, w, y, gr, xp, c = [t.to(dev) for t in _inputs(500, 3000, 264, 64, 17)]
    runs = []
    for _ in range(3):
        cg = c.clone()
        loss, lse, _ = rgc.rgc_linear_cross_entropy_forward(x, w, y)
        dx = rgc.rgc_linear_cross_entropy_backward(x, w, y, lse, gr, xp, cg)
        runs.append((loss, lse, dx, cg))
    for run in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], run))


def test_gradient_agrees_with_differences(dev):
    """The loss's change along dX, by central differences of the forward."""
    T, V, k = 8, 300, 64
    x, w, y, gr, _, _ = _inputs(T, V, k, 0, 18, ignored=0.0)
    xg, wg, yg, gg = x.to(dev), w.to(dev), y.to(dev), gr.to(dev)
    _, lse, _ = rgc.rgc_linear_cross_entropy_forward(xg, wg, yg)
    dx = rgc.rgc_linear_cross_entropy_backward(xg, wg, yg, lse, gg).double()
    # steps of 1/8 in single elements of X of size up to 1 are exact in bf16 for values that are multiples of 2^-8
    xq = (x.float().clamp(-1, 1) * 256).round() / 256
    xq = xq.bfloat16()
    _, lse, _ = rgc.rgc_linear_cross_entropy_forward(xq.to(dev), wg, yg)
    dx = rgc.rgc_linear_cross_entropy_backward(xq.to(dev), wg, yg, lse, gg).double().cpu()
    for t, i in ((0, 3), (5, 60), (7, 0)):
        h = 0.125
        xq64 = xq.double()
        loss = []
        for s in (h, -h):
            xs = xq64.clone()
            xs[t, i] = torch.tensor(float(xs[t, i]) + s).bfloat16().double()
            loss.append((rgc.rgc_linear_cross_entropy_forward(xs.bfloat16().to(dev), wg, yg)[0].double().cpu(),
                         float(xs[t, i])))
        slope = float(((loss[0][0] - loss[1][0]) * gr.double()).sum()) / (loss[0][1] - loss[1][1])
        # third derivative of the loss along one element: at most |w|^3 (a third cumulant of a variable of that
        # range, |w| <= max |W[:, i]|, is at most w^3), so the difference is off by h^2 / 6 of it
        wm = float(w[:, i].abs().max())
        tol = abs(float(gr[t])) * (2 * wm) ** 3 * h * h / 6 + 2.0 ** -7 * abs(slope) + 2.0 ** -8 * float(gr[t].abs()) * wm
        assert abs(slope - float(dx[t, i])) <= tol, (t, i, slope, float(dx[t, i]), tol)


def test_captured_and_replayed(dev):
    """Two graphs of forward and backward, replayed in turn with eager calls between, each replay with new inputs."""
    shapes = [(200, 1000, 136, 16), (90, 2000, 136, 0)]
    jobs = []
    for T, V, k, r in shapes:
        st = [t.to(dev) if t is not None else None for t in _inputs(T, V, k, r, 19)]

        def call(st=st):
            x, w, y, gr, xp, c = st
            cg = c.clone() if c is not None else None
            loss, lse, _ = rgc.rgc_linear_cross_entropy_forward(x, w, y)
            return loss, rgc.rgc_linear_cross_entropy_backward(x, w, y, lse, gr, xp, cg), cg

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = call()
        jobs.append((st, call, graph, outs))
    for rep in range(3):
        for n, (st, call, graph, outs) in enumerate(jobs):
            st[0].copy_(synth.normal_bf16(tuple(st[0].shape), 1.0, seed=50 + 7 * rep + n).to(dev))
            graph.replay()
        torch.cuda.synchronize()
        for st, call, graph, outs in jobs:
            eager = call()
            torch.cuda.synchronize()
            for a, b in zip(outs, eager):
                assert a is None and b is None or torch.equal(a, b), rep


def test_two_streams_at_once(dev):
    jobs = [[t.to(dev) if t is not None else None for t in _inputs(300, 3000, 264, r, 60 + r)] for r in (0, 16)]

    def call(st):
        x, w, y, gr, xp, c = st
        cg = c.clone() if c is not None else None
        loss, lse, _ = rgc.rgc_linear_cross_entropy_forward(x, w, y)
        return loss, rgc.rgc_linear_cross_entropy_backward(x, w, y, lse, gr, xp, cg), cg

    want = [call(j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for n in (0, 1):
            with torch.cuda.stream(streams[n]):
                got[n].append(call(jobs[n]))
    torch.cuda.synchronize()
    for n in (0, 1):
        for g in got[n]:
            assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(g, want[n]))
