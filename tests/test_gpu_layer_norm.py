"""rgc_layer_norm_forward and _backward against the formulas in 64 bits.

Bounds, element by element, u = 2^-24 the fp32 half step. Sums over a row of n
elements are taken in at most n / (lanes) + 10 additions a lane; 2^-19 of the
sum of magnitudes covers every width tested (n <= 65536: at most 64 terms a lane
and ten joining steps, 74 u < 2^-17.7 for the widest, 32 u = 2^-19 up to 16384).
mu is off by that of mean |x|, and so are the centred values (call it dc); the
variance's relative error is that of its sum plus 2 dc / sigma; xhat's is dc rstd
plus half of the variance's. Outputs add their own rounding: half a step of
their type (2^-8 for bf16, 2^-24 for fp32) and a few u.
"""
import pytest
import torch

from rank_randomized_gradient_amd import rgc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
S = 2.0 ** -17  # of a sum of magnitudes, see above


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _inputs(rows, n, xt, wt, seed):
    g = torch.Generator().manual_seed(seed)
    x = ((torch.randn(rows, n, generator=g) + torch.randn(rows, 1, generator=g)) * 2).to(xt)
    dy = torch.randn(rows, n, generator=g).to(xt)
    w = (1 + 0.2 * torch.randn(n, generator=g)).to(wt)
    b = torch.randn(n, generator=g).to(wt)
    return x, dy, w, b


def _half(t):
    return torch.finfo(t).eps / 2


def _reference(x, dy, w, b, kind, wt):
    xt, n = x.dtype, x.shape[1]
    x, dy = x.double(), dy.double()
    w64 = w.double() if w is not None else torch.ones(n, dtype=torch.float64)
    b64 = b.double() if b is not None else torch.zeros(n, dtype=torch.float64)
    mu = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros(len(x), 1, dtype=torch.float64)
    c = x - mu
    var = c.square().mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + EPS)
    xhat = c * rstd
    dc = S * x.abs().mean(1, keepdim=True) + 2.0 ** -23 * x.abs()
    dvar = S + 2 * (dc * c.abs()).mean(1, keepdim=True) / (var + EPS) + 2.0 ** -21  # relative, of var + eps
    dxhat = dc * rstd + xhat.abs() * (dvar / 2 + 2.0 ** -22)
    out, bound = {}, {}
    out["Y"] = xhat * w64 + b64
    bound["Y"] = dxhat * w64.abs() + (_half(xt) + 2.0 ** -23) * out["Y"].abs() + 2.0 ** -23 * (xhat * w64).abs()
    h = dy * w64
    flat = h.mean(1, keepdim=True) if kind == "layer" else 0.0
    along = (h * xhat).mean(1, keepdim=True)
    out["dX"] = (h - flat - xhat * along) * rstd
    dflat = S * h.abs().mean(1, keepdim=True)
    dalong = S * (h * xhat).abs().mean(1, keepdim=True) + (h.abs() * dxhat).mean(1, keepdim=True)
    size = h.abs() + h.abs().mean(1, keepdim=True) + (xhat * along).abs()
    bound["dX"] = ((dflat + dxhat * along.abs() + xhat.abs() * dalong + 2.0 ** -21 * size) * rstd
                   + out["dX"].abs() * (dvar / 2 + _half(xt)))
    out["dw"] = (dy * xhat).sum(0)
    # column sums: at most rows additions in sequence and sixteen joining ones
    steps = (len(x) + 32) * 2.0 ** -24
    bound["dw"] = (dy.abs() * dxhat).sum(0) + steps * (dy * xhat).abs().sum(0) + _half(wt) * out["dw"].abs()
    out["db"] = dy.sum(0)
    bound["db"] = steps * dy.abs().sum(0) + _half(wt) * out["db"].abs()
    return out, bound


def _check(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    excess = (got - want).abs() - bound
    assert excess.numel() == 0 or float(excess.max()) <= 1e-30, f"{what}: {float(excess.max()):.3e} over the bound"


def _run(dev, rows, n, xt, wt, kind, seed, weight=True, bias=True):
    x, dy, w, b = _inputs(rows, n, xt, wt, seed)
    w, b = w if weight else None, b if bias else None
    want, bound = _reference(x, dy, w, b, kind, wt if weight else F32)
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    xg, wg = to(x), to(w)
    y, mean, rstd = rgc.rgc_layer_norm_forward(xg, wg, to(b), eps=EPS, kind=kind)
    assert (mean is None) == (kind == "rms") and y.dtype == xt and rstd.dtype == F32
    dx, dw, db = rgc.rgc_layer_norm_backward(to(dy), xg, wg, mean, rstd, bias=bias, kind=kind)
    torch.cuda.synchronize()
    what = f"{rows}x{n} {xt} {wt} {kind}"
    _check(y, want["Y"], bound["Y"], "Y " + what)
    _check(dx, want["dX"], bound["dX"], "dX " + what)
    _check(dw, want["dw"], bound["dw"], "dweight " + what)
    assert dw.dtype == (wt if weight else F32)
    if bias:
        _check(db, want["db"], bound["db"], "dbias " + what)
    else:
        assert db is None


# one element, one row; every width class of both paths and one past each; odd widths
WIDTHS = [1, 2, 7, 8, 64, 65, 120, 128, 136, 256, 257, 512, 520, 1000, 1003, 1024, 1032, 2048, 2056, 4095, 4096, 4097, 4104,
          8192, 8200, 16384]


@pytest.mark.parametrize("n", WIDTHS)
def test_every_width(dev, n):
    print(n, flush=True)
    _run(dev, 37, n, BF, F32, "layer", n)
    _run(dev, 5, n, F32, BF, "rms", n + 1)


@pytest.mark.parametrize("n", [16385, 16392, 40000, 65536])
def test_rows_wider_than_the_registers(dev, n):
    print(n, flush=True)
    _run(dev, 70, n, BF, BF, "layer", n)
    _run(dev, 3, n, F32, F32, "rms", n)


@pytest.mark.parametrize("rows", [1, 2, 3, 255, 256, 257, 1025, 5000])
@pytest.mark.parametrize("n", [128, 1003, 2048])
def test_row_counts(dev, rows, n):
    print(rows, n, flush=True)
    _run(dev, rows, n, BF, F32, "layer", rows)


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("wt", [BF, F32])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("weight,bias", [(True, True), (True, False), (False, False), (False, True)])
def test_types_kinds_and_missing_parameters(dev, xt, wt, kind, weight, bias):
    if not weight and bias:
        # without a weight dbias is float32 whatever the bias's type
        x, dy, _, b = _inputs(20, 264, xt, wt, 3)
        want, bound = _reference(x, dy, None, b, kind, F32)
        y, mean, rstd = rgc.rgc_layer_norm_forward(x.to(dev), None, b.to(dev), eps=EPS, kind=kind)
        _, _, db = rgc.rgc_layer_norm_backward(dy.to(dev), x.to(dev), None, mean, rstd, kind=kind)
        _check(y, want["Y"], bound["Y"], "Y")
        _check(db, want["db"], bound["db"], "dbias")
        return
    _run(dev, 20, 264, xt, wt, kind, 3, weight, bias)


def test_no_rows(dev):
    x = torch.zeros(0, 100, dtype=BF, device=dev)
    w = torch.ones(100, device=dev)
    y, mean, rstd = rgc.rgc_layer_norm_forward(x, w, w)
    dx, dw, db = rgc.rgc_layer_norm_backward(x, x, w, mean, rstd)
    assert y.shape == dx.shape == (0, 100) and bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("xt,n,off", [(BF, 264, 8), (BF, 264, 1), (F32, 260, 4), (F32, 261, 3), (BF, 1003, 5)])
def test_strided_rows_and_what_lies_around_them(dev, xt, n, off):
    rows = 50
    x, dy, w, b = _inputs(rows, n, xt, F32, 9)
    want, bound = _reference(x, dy, w, b, "layer", F32)
    wide = n + 24
    full = [torch.full((rows + 2, wide), v, dtype=xt, device=dev) for v in (float("nan"), float("nan"), 3.0, 5.0)]
    xs, ds, ys, gs = [f[1:-1, off:off + n] for f in full]
    xs.copy_(x.to(dev))
    ds.copy_(dy.to(dev))
    _, mean, rstd = rgc.rgc_layer_norm_forward(xs, w.to(dev), b.to(dev), eps=EPS, Y=ys)
    _, dw, db = rgc.rgc_layer_norm_backward(ds, xs, w.to(dev), mean, rstd, dX=gs)
    _check(ys, want["Y"], bound["Y"], "Y")
    _check(gs, want["dX"], bound["dX"], "dX")
    _check(dw, want["dw"], bound["dw"], "dweight")
    _check(db, want["db"], bound["db"], "dbias")
    for f, v in ((full[2], 3.0), (full[3], 5.0)):
        inside = torch.zeros_like(f, dtype=torch.bool)
        inside[1:-1, off:off + n] = True
        assert bool((f[~inside] == v).all())


def test_constant_rows_and_large_means(dev):
    """A row of one value has variance 0: y is the bias. A mean far above the spread keeps the spread (the
    variance is taken of centred values)."""
    n = 512
    x = torch.full((3, n), 7.0, device=dev)
    w, b = torch.ones(n, device=dev), torch.full((n,), 0.25, device=dev)
    y, _, rstd = rgc.rgc_layer_norm_forward(x, w, b, eps=EPS)
    assert bool((y == 0.25).all())
    _, dw, _ = rgc.rgc_layer_norm_backward(torch.ones_like(x), x, w, torch.full((3,), 7.0, device=dev), rstd)
    assert bool((dw == 0).all())
    # 4096 + {-1, 1}: exact in fp32, mean exact, variance 1
    x = 4096 + torch.tensor([-1.0, 1.0], device=dev).repeat(n // 2)[None]
    y, mean, rstd = rgc.rgc_layer_norm_forward(x, None, None, eps=0.0)
    assert float(mean) == 4096 and float(rstd) == 1 and torch.equal(y, x - 4096)


def test_nan_and_inf_stay_in_their_rows(dev):
    x, dy, w, b = _inputs(9, 264, BF, F32, 5)
    want, bound = _reference(x, dy, w, b, "layer", F32)
    x[4, 7] = float("nan")
    x[6, 0] = float("inf")
    y, mean, rstd = rgc.rgc_layer_norm_forward(x.to(dev), w.to(dev), b.to(dev), eps=EPS)
    dx, _, _ = rgc.rgc_layer_norm_backward(dy.to(dev), x.to(dev), w.to(dev), mean, rstd)
    keep = torch.tensor([i not in (4, 6) for i in range(9)])
    _check(y.cpu()[keep], want["Y"][keep], bound["Y"][keep], "Y")
    _check(dx.cpu()[keep], want["dX"][keep], bound["dX"][keep], "dX")
    assert torch.isnan(y[4]).all() and torch.isnan(dx[4]).all()


def test_gradient_agrees_with_differences(dev):
    """dX, dweight and dbias against central differences of the forward in fp32."""
    n, h = 40, 2.0 ** -5
    g = torch.Generator().manual_seed(2)
    x = torch.randn(3, n, generator=g)
    x = (x * 32).round() / 32
    w, b, dy = 1 + 0.1 * torch.randn(n, generator=g), torch.randn(n, generator=g), torch.randn(3, n, generator=g)
    for kind in ("layer", "rms"):
        _, mean, rstd = rgc.rgc_layer_norm_forward(x.to(dev), w.to(dev), b.to(dev), eps=EPS, kind=kind)
        dx, dw, db = rgc.rgc_layer_norm_backward(dy.to(dev), x.to(dev), w.to(dev), mean, rstd, kind=kind)

        def loss(x_, w_, b_):
            y, _, _ = rgc.rgc_layer_norm_forward(x_.to(dev), w_.to(dev), b_.to(dev), eps=EPS, kind=kind)
            return float((y.double().cpu() * dy.double()).sum())

        size = float(dy.abs().sum())
        for i, j in ((0, 0), (1, 17), (2, 39)):
            for base, grad, at in ((x, dx, (i, j)), (w, dw, (j,)), (b, db, (j,))):
                up, down = base.clone(), base.clone()
                up[at] += h
                down[at] -= h
                args = [(up if base is t else t, down if base is t else t) for t in (x, w, b)]
                slope = (loss(*[a[0] for a in args]) - loss(*[a[1] for a in args])) / float(up[at] - down[at])
                # third derivatives of xhat along one element are below 30 rstd^3 (each derivative divides by sigma
                # and |xhat| <= sqrt(n) enters at most cubed over n); fp32 rounding of y enters over 2 h
                r = float(rstd[i] if base is x else 1.0)
                tol = size * (30 * r ** 3 / n ** 0.5 * h * h / 6 * (base is x) + 8 * 2.0 ** -22 / (2 * h))
                assert abs(slope - float(grad[at])) <= tol, (kind, at, slope, float(grad[at]), tol)


def test_repeated_calls_give_the_same_bits(dev):
    x, dy, w, b = [t.to(dev) for t in _inputs(3000, 1024, BF, F32, 6)]
    runs = []
    for _ in range(3):
        y, mean, rstd = rgc.rgc_layer_norm_forward(x, w, b)
        runs.append((y, mean, rstd, *rgc.rgc_layer_norm_backward(dy, x, w, mean, rstd)))
    for r in runs[1:]:
        assert all(torch.equal(a, c) for a, c in zip(runs[0], r))


def test_captured_and_replayed(dev):
    jobs = []
    for rows, n in ((300, 1024), (77, 1003)):
        st = [t.to(dev) for t in _inputs(rows, n, BF, F32, 8)]

        def call(st=st):
            x, dy, w, b = st
            y, mean, rstd = rgc.rgc_layer_norm_forward(x, w, b)
            return (y, *rgc.rgc_layer_norm_backward(dy, x, w, mean, rstd))

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = call()
        jobs.append((st, call, graph, outs))
    for rep in range(3):
        for st, call, graph, outs in jobs:
            st[0].add_(0.5 * (rep + 1))
            graph.replay()
        torch.cuda.synchronize()
        for st, call, graph, outs in jobs:
            for a, c in zip(outs, call()):
                assert torch.equal(a, c), rep
