"""The residual norm's forward on rows above 16384, whose last elements, where they are no whole
vector of eight, are one thread's: the sum is torch's, and the norm, mean and rstd are those of rgc_layer_norm_forward of
it, bit for bit, wherever that end lies."""
import pytest
import torch

from rank_randomized_gradient_amd import rgc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _inputs(rows, n, xt, seed, dev):
    g = torch.Generator().manual_seed(seed)
    x, r = (torch.randn(rows, n, generator=g).to(xt).to(dev) for _ in range(2))
    return x, r, (1 + 0.2 * torch.randn(n, generator=g)).to(dev), torch.randn(n, generator=g).to(dev)


# one element and seven in the last vector; that vector the first, a middle and the last thread's, of the third to the
# eighth of a thread's; no such vector
WIDTHS = [16385, 16391, 16384 + 8 * 511 + 3, 16384 + 8 * 1023 + 5, 16384 + 8 * 1024 + 1, 32768, 32769, 40003, 57345, 65528,
          65529, 65535, 65536]


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("n", WIDTHS)
def test_the_plain_norms_bits(dev, n, xt):
    print(n, xt, flush=True)
    for rows, kind, wt in ((5, "layer", F32), (3, "rms", BF)):
        x, r, w, b = _inputs(rows, n, xt, n, dev)
        w, b = w.to(wt), b.to(wt)
        for weight, bias in ((w, b), (w, None), (None, None)):
            s, y, mean, rstd = rgc.rgc_add_norm_forward(x, r, weight, bias, kind=kind)
            assert torch.equal(s, (x.float() + r.float()).to(xt))
            want = rgc.rgc_layer_norm_forward(s, weight, bias, kind=kind)
            assert all(p is None and q is None or torch.equal(p, q) for p, q in zip((y, mean, rstd), want))
        y64 = s.double() - (s.double().mean(1, keepdim=True) if kind == "layer" else 0.0)
        y64 = y64 / torch.sqrt(y64.square().mean(1, keepdim=True) + 1e-5)
        # half a step of the type, and a row's sums off by 2^-17 of their magnitudes (of x: mean |x| < 2 |y|'s scale)
        assert bool(((y - y64).abs() <= (torch.finfo(xt).eps / 2 + 2.0 ** -16) * (y64.abs() + 1)).all())


# (2100 rows: more than a launch has workgroups)
@pytest.mark.parametrize("xt,n,off,rows", [(BF, 20003, 1, 2100), (F32, 40001, 3, 300), (BF, 65535, 0, 300)])
def test_in_place_strided_and_what_lies_around(dev, xt, n, off, rows):
    x, r, w, b = _inputs(rows, n, xt, 7, dev)
    s0, y0, _, _ = rgc.rgc_add_norm_forward(x, r, w, b)
    full = [torch.full((rows + 2, n + 13), 3.0, dtype=xt, device=dev) for _ in range(2)]
    views = [f[1:-1, off:off + n] for f in full]
    for into in ((0, 1), (1, 0)):
        views[0].copy_(x), views[1].copy_(r)
        rgc.rgc_add_norm_forward(views[0], views[1], w, b, S=views[into[0]], Y=views[into[1]])
        assert torch.equal(views[into[0]], s0) and torch.equal(views[into[1]], y0)
    for f in full:
        inside = torch.zeros_like(f, dtype=torch.bool)
        inside[1:-1, off:off + n] = True
        assert bool((f[~inside] == 3).all())
