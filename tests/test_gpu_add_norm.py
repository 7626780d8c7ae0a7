"""The residual norm, rgc_add_norm_forward and _backward. The sum is one rounding of
an fp32 sum: torch's bits. Y, mean and rstd are those of rgc_layer_norm_forward of the
sum, bit for bit, and so are dX, dweight and dbias without a gradient of the sum. With one, dX is
the norm's own dx in fp32 plus it, rounded once, and the column sums may be taken of other rows together:
all three are compared with the formulas in 64 bits. Row sums are off by 2^-17 of their magnitudes, as
rgc_layer_norm_backward's tests derive; a column's sum takes at most `rows` additions in sequence and 32 joining ones.
"""
import pytest
import torch

from rank_randomized_gradient_amd import LayerNorm, rgc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
SUM = 2.0 ** -17  # of a sum of magnitudes


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _inputs(rows, n, xt, wt, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, n, generator=g).to(xt)
    r = ((torch.randn(rows, n, generator=g) + torch.randn(rows, 1, generator=g)) * 2).to(xt)
    dy, ds = torch.randn(rows, n, generator=g).to(xt), torch.randn(rows, n, generator=g).to(xt)
    w, b = (1 + 0.2 * torch.randn(n, generator=g)).to(wt), torch.randn(n, generator=g).to(wt)
    return x, r, dy, ds, w, b


def _dx(s, dy, ds, w, kind):
    """dX, dweight and dbias in 64 bits with their bounds (the last two before their rounding): what
    rgc_layer_norm_backward's tests derive, and one rounding of the whole of dX."""
    half = torch.finfo(s.dtype).eps / 2
    x, dy, ds = s.double(), dy.double(), ds.double()
    w = w.double() if w is not None else torch.ones(s.shape[1], dtype=torch.float64)
    mu = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros(len(x), 1, dtype=torch.float64)
    c = x - mu
    var = c.square().mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + EPS)
    xhat = c * rstd
    dc = SUM * x.abs().mean(1, keepdim=True) + 2.0 ** -23 * x.abs()
    dvar = SUM + 2 * (dc * c.abs()).mean(1, keepdim=True) / (var + EPS) + 2.0 ** -21
    dxhat = dc * rstd + xhat.abs() * (dvar / 2 + 2.0 ** -22)
    h = dy * w
    flat = h.mean(1, keepdim=True) if kind == "layer" else 0.0
    along = (h * xhat).mean(1, keepdim=True)
    own = (h - flat - xhat * along) * rstd
    dflat = SUM * h.abs().mean(1, keepdim=True)
    dalong = SUM * (h * xhat).abs().mean(1, keepdim=True) + (h.abs() * dxhat).mean(1, keepdim=True)
    size = h.abs() + h.abs().mean(1, keepdim=True) + (xhat * along).abs()
    off = (dflat + dxhat * along.abs() + xhat.abs() * dalong + 2.0 ** -21 * size) * rstd + own.abs() * dvar / 2
    out = own + ds
    steps = (len(s) + 32) * 2.0 ** -24
    dw, db = (dy * xhat).sum(0), dy.sum(0)
    columns = ((dw, (dy.abs() * dxhat).sum(0) + steps * (dy * xhat).abs().sum(0)), (db, steps * dy.abs().sum(0)))
    return (out, off + (half + 2.0 ** -23) * out.abs() + 2.0 ** -23 * own.abs()), *columns


def _check(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    excess = (got - want).abs() - bound
    assert excess.numel() == 0 or float(excess.max()) <= 1e-30, f"{what}: {float(excess.max()):.3e} over the bound"


def _equal(a, b):
    return a is None and b is None or torch.equal(a, b)


def _run(dev, rows, n, xt, wt, kind, seed, weight=True, bias=True):
    x, r, dy, ds, w, b = [t.to(dev) for t in _inputs(rows, n, xt, wt, seed)]
    w, b = w if weight else None, b if bias else None
    s, y, mean, rstd = rgc.rgc_add_norm_forward(x, r, w, b, eps=EPS, kind=kind)
    assert torch.equal(s, (x.float() + r.float()).to(xt))
    plain = rgc.rgc_layer_norm_forward(s, w, b, eps=EPS, kind=kind)
    assert all(_equal(p, q) for p, q in zip((y, mean, rstd), plain)) and (mean is None) == (kind == "rms")
    # without the sum's gradient: the plain norm's
    want = rgc.rgc_layer_norm_backward(dy, s, w, mean, rstd, bias=bias, kind=kind)
    got = rgc.rgc_add_norm_backward(dy, None, s, w, mean, rstd, bias=bias, kind=kind)
    assert all(_equal(p, q) for p, q in zip(got, want))
    dx, dw, db = rgc.rgc_add_norm_backward(dy, ds, s, w, mean, rstd, bias=bias, kind=kind)
    torch.cuda.synchronize()
    what = f"{rows}x{n} {xt} {wt} {kind}"
    (ref, bound), *columns = _dx(s.cpu(), dy.cpu(), ds.cpu(), w.cpu() if weight else None, kind)
    _check(dx, ref, bound, "dX " + what)
    for got, plain, (ref, bound), name in zip((dw, db), want[1:], columns, ("dweight ", "dbias ")):
        assert (got is None) == (plain is None)
        if got is not None:
            assert got.dtype == plain.dtype
            _check(got, ref, bound + torch.finfo(got.dtype).eps / 2 * ref.abs(), name + what)


WIDTHS = [1, 2, 7, 8, 64, 65, 128, 136, 257, 512, 520, 1000, 1003, 1024, 1032, 2048, 2056, 4095, 4096, 4097, 8192, 8200,
          16384, 16385, 16392, 40000, 65536]


@pytest.mark.parametrize("n", WIDTHS)
def test_every_width(dev, n):
    print(n, flush=True)
    _run(dev, 37, n, BF, F32, "layer", n)
    _run(dev, 5, n, F32, BF, "rms", n + 1)
    _run(dev, 5, n, BF, BF, "rms", n + 2, bias=False)


@pytest.mark.parametrize("rows", [1, 2, 255, 257, 5000])
@pytest.mark.parametrize("n", [128, 1003, 1800, 4096])
def test_row_counts(dev, rows, n):
    _run(dev, rows, n, BF, F32, "rms", rows, bias=False)
    _run(dev, rows, n, BF, F32, "layer", rows)


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("wt", [BF, F32])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("weight,bias", [(True, True), (True, False), (False, False)])
def test_types_kinds_and_missing_parameters(dev, xt, wt, kind, weight, bias):
    _run(dev, 20, 264, xt, wt, kind, 3, weight, bias)


def test_no_rows(dev):
    x, w = torch.zeros(0, 100, dtype=BF, device=dev), torch.ones(100, device=dev)
    s, y, mean, rstd = rgc.rgc_add_norm_forward(x, x, w, w)
    dx, dw, db = rgc.rgc_add_norm_backward(x, x, x, w, mean, rstd)
    assert s.shape == y.shape == dx.shape == (0, 100) and bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("xt,n,off", [(BF, 264, 8), (BF, 264, 1), (F32, 261, 3), (BF, 1003, 5), (BF, 20000, 3)])
def test_strided_rows_and_what_lies_around_them(dev, xt, n, off):
    rows = 30
    x, r, dy, ds, w, b = [t.to(dev) for t in _inputs(rows, n, xt, F32, 9)]
    s0, y0, mean, rstd = rgc.rgc_add_norm_forward(x, r, w, b)
    g0 = rgc.rgc_add_norm_backward(dy, ds, s0, w, mean, rstd)
    full = [torch.full((rows + 2, n + 24 + 8 * i), float("nan") if i < 4 else 3.0, dtype=xt, device=dev) for i in range(7)]
    xs, rs, ys_, gs, ss, yy, dd = [f[1:-1, off:off + n] for f in full]
    for a, v in ((xs, x), (rs, r), (ys_, dy), (gs, ds)):
        a.copy_(v)
    _, _, mean, rstd = rgc.rgc_add_norm_forward(xs, rs, w, b, S=ss, Y=yy)
    _, dw, db = rgc.rgc_add_norm_backward(ys_, gs, ss, w, mean, rstd, dX=dd)
    assert torch.equal(ss, s0) and torch.equal(yy, y0) and torch.equal(dd, g0[0])
    assert torch.equal(dw, g0[1]) and torch.equal(db, g0[2])
    for f in full[4:]:
        inside = torch.zeros_like(f, dtype=torch.bool)
        inside[1:-1, off:off + n] = True
        assert bool((f[~inside] == 3).all())


@pytest.mark.parametrize("n", [264, 1003, 4096, 20000])
def test_in_place(dev, n):
    """The sum in the residual's place, y in x's; dX in the place of each of its operands."""
    x, r, dy, ds, w, b = [t.to(dev) for t in _inputs(50, n, BF, F32, 10)]
    s, y, mean, rstd = rgc.rgc_add_norm_forward(x, r, w, b)
    dx = rgc.rgc_add_norm_backward(dy, ds, s, w, mean, rstd)[0]
    for flip in (False, True):
        a, c = x.clone(), r.clone()
        to = (c, a) if not flip else (a, c)
        rgc.rgc_add_norm_forward(a, c, w, b, S=to[0], Y=to[1])
        assert torch.equal(to[0], s) and torch.equal(to[1], y)
    for i in range(3):
        ops = [dy.clone(), ds.clone(), s.clone()]
        rgc.rgc_add_norm_backward(*ops, w, mean, rstd, dX=ops[i])
        assert torch.equal(ops[i], dx), i


def test_offsets_past_two_to_the_32(dev):
    """Rows 2^31 elements apart."""
    n, ld = 4096, (1 << 31) - 8
    flat = torch.empty(2 * ld + n, dtype=BF, device=dev)
    far = flat.as_strided((3, n), (ld, 1))
    x, r, dy, ds, w, b = [t.to(dev) for t in _inputs(3, n, BF, F32, 11)]
    s, y, mean, rstd = rgc.rgc_add_norm_forward(x, r, w, b)
    far.copy_(r)
    rgc.rgc_add_norm_forward(x, far, w, b, S=far)
    assert torch.equal(far, s)
    dx = rgc.rgc_add_norm_backward(dy, ds, s, w, mean, rstd)[0]
    assert torch.equal(rgc.rgc_add_norm_backward(dy, ds, far, w, mean, rstd)[0], dx)
    far.copy_(ds)
    rgc.rgc_add_norm_backward(dy, far, s, w, mean, rstd, dX=far)
    assert torch.equal(far, dx)


def test_refusals(dev):
    x, w, f = torch.zeros(5, 40, dtype=BF, device=dev), torch.ones(40, device=dev), torch.ones(5, device=dev)
    fwd, bwd = rgc.rgc_add_norm_forward, rgc.rgc_add_norm_backward
    for call in (lambda: fwd(x, x.float(), w), lambda: fwd(x, x[:4], w), lambda: fwd(x, x.cpu(), w), lambda: fwd(x, x, w[:39]),
                 lambda: fwd(x, x, w, kind="batch"), lambda: fwd(x, x, w, eps=-1.0), lambda: fwd(x, x, w, S=x.float()),
                 lambda: fwd(x, x, w, S=x, Y=x), lambda: fwd(x, x[:1].expand(5, 40), w), lambda: fwd(x.half(), x.half(), w),
                 lambda: bwd(x, x.float(), x, w, f, f), lambda: bwd(x, x[:4], x, w, f, f), lambda: bwd(x, x, x, w, None, f),
                 lambda: bwd(x, x, x, w, f, f[:4]), lambda: bwd(x, x, x, w, f, f, dX=x[:4])):
        with pytest.raises(rgc.RgcError):
            call()


def _both(st):
    x, r, dy, ds, w, b = st
    s, y, mean, rstd = rgc.rgc_add_norm_forward(x, r, w, b)
    return (s, y, *rgc.rgc_add_norm_backward(dy, ds, s, w, mean, rstd))


def test_captured_and_replayed(dev):
    jobs = []
    for rows, n in ((300, 1024), (77, 1003)):
        st = [t.to(dev) for t in _inputs(rows, n, BF, F32, 8)]
        _both(st)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = _both(st)
        jobs.append((st, graph, outs))
    for rep in range(3):
        for st, graph, outs in jobs:
            st[0].add_(0.5 * (rep + 1))
            graph.replay()
        torch.cuda.synchronize()
        for st, graph, outs in jobs:
            assert all(torch.equal(a, c) for a, c in zip(outs, _both(st))), rep


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("used", ["both", "y", "sum"])
def test_module(dev, kind, used):
    """LayerNorm(x, residual): gradients of x, residual and the parameters, whichever outputs are used; a broadcast
    gradient of the sum among them."""
    B, L, n = 3, 7, 264
    x, r, dy, _, _, _ = _inputs(B * L, n, BF, F32, 12)
    x, r = (t.reshape(B, L, n).to(dev).requires_grad_() for t in (x, r))
    dy = dy.reshape(B, L, n).to(dev)
    norm = LayerNorm(n, kind=kind, device=dev)
    y, s = norm(x, r)
    assert y.shape == s.shape == x.shape
    loss = 0
    if used != "sum":
        loss = loss + (y * dy).sum()
    if used != "y":
        loss = loss + s.sum()
    loss.backward()
    ones = torch.ones(B * L, n, dtype=BF, device=dev)
    if used == "sum":
        assert torch.equal(x.grad, ones.reshape(B, L, n)) and torch.equal(r.grad, x.grad) and norm.weight.grad is None
        return
    s2, _, mean, rstd = rgc.rgc_add_norm_forward(x.detach().reshape(-1, n), r.detach().reshape(-1, n), norm.weight.detach(),
                                                 None if norm.bias is None else norm.bias.detach(), kind=kind)
    dx, dw, db = rgc.rgc_add_norm_backward(dy.reshape(-1, n), ones if used == "both" else None, s2, norm.weight.detach(), mean,
                                           rstd, bias=norm.bias is not None, kind=kind)
    assert torch.equal(s.reshape(-1, n), s2) and torch.equal(x.grad.reshape(-1, n), dx) and torch.equal(r.grad, x.grad)
    assert x.grad.data_ptr() != r.grad.data_ptr()
    assert torch.equal(norm.weight.grad, dw) and _equal(None if norm.bias is None else norm.bias.grad, db)


def test_module_refuses_another_shape(dev):
    norm = LayerNorm(64, device=dev)
    x = torch.zeros(4, 64, dtype=BF, device=dev)
    for bad in (x[:2], x.float(), x[:, :32]):
        with pytest.raises(rgc.RgcError):
            norm(x, bad)
