"""Log probabilities, entropies and alternatives of logits at hand:
rgc_log_prob_forward and _backward against the same formulas in 64 bits.

Bounds, element by element, u = 2^-24 the fp32 half step. The logits are exact.
exp(d) is off by |d| 2^-22 of itself for its rounded exponent and 2^-21 for the
rest. A row's sums take at most N = 100 + V / 1600 roundings one after the other
(a batch of 8192 entries adds 13 of them to a thread, or 4 and the rescaling's; the lanes' and
the waves' or parts' joins 64 at most), so with p the probabilities, d = z - m
  log s: u N + 2^-21 + 2^-22 sum p |d|
  lse = m + log s: 2^-23 (|lse| + |m|) more;  logp = z - m - log s: 2^-22 |logp| more
  H: 2 (u N + 2^-21) (1 + sum p (|d| + d^2))
dz = p f + gl [v = y], f = -gl - ge (log p + H): p's relative error is lse's (log s's alone where |lse| >= 1024: there
the backward takes z - m - log s) + 2^-21 + 2^-21 |log p|, f is off by |ge| (as much
+ H's) + 2^-22 (|gl| + |ge| (|log p| + H)); then half a step of the logits' type.
Indices are equal, whatever ties.
"""
import math

import pytest
import torch

from rank_randomized_gradient_amd import log_prob, rgc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _inputs(rows, V, zt, seed, ignored=0.1, masked=0.05, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(rows, V, generator=g) * spread).to(zt)
    if masked and V > 4:
        z[torch.rand(rows, V, generator=g) < masked] = -INF
    y = torch.randint(0, V, (rows,), generator=g)
    y = torch.where(z.gather(1, y[:, None])[:, 0] == -INF, z.float().argmax(1), y)
    y[torch.rand(rows, generator=g) < ignored] = -100
    return z, y, torch.randn(rows, generator=g), 0.3 * torch.randn(rows, generator=g)


def _reference(z, y, gl, ge, top):
    zt, (rows, V) = z.dtype, z.shape
    z = z.double()
    zero = torch.zeros(rows, dtype=torch.float64)
    gl, ge = (zero if g is None else g.double() for g in (gl, ge))
    live = (y >= 0) & (y < V)
    at = torch.where(live, y, 0)
    gl, ge = torch.where(live, gl, 0.0), torch.where(live, ge, 0.0)
    m = z.amax(1)
    ls = torch.logsumexp(z - m[:, None], 1)
    lse = m + ls
    some = torch.where(z == -INF, m[:, None], z)  # (p is 0 there)
    d = some - m[:, None]
    lp = d - ls[:, None]
    p = torch.exp(z - m[:, None] - ls[:, None])
    H = -(p * lp).sum(1)
    r = torch.arange(rows)
    uN = (100 + V / 1600) * 2.0 ** -24
    e_ls = uN + 2.0 ** -21 + 2.0 ** -22 * (p * d.abs()).sum(1)
    e_lse = e_ls + 2.0 ** -23 * (lse.abs() + m.abs())
    e_p = torch.where(lse.abs() < 1024, e_lse, e_ls)
    e_h = 2 * (uN + 2.0 ** -21) * (1 + (p * (d.abs() + d * d)).nan_to_num(0.0).sum(1))  # (d^2 overflows where p is 0)
    given = torch.where(live, z[r, at] - m - ls, 0.0)
    out = {"lse": lse, "logp": given, "entropy": torch.where(live, H, 0.0), "entropy of all": H}
    bound = {"lse": e_lse, "logp": e_ls + 2.0 ** -22 * given.abs(), "entropy": e_h, "entropy of all": e_h}
    f = -gl[:, None] - ge[:, None] * (lp + H[:, None])
    D = p * f
    size = gl.abs()[:, None] + ge.abs()[:, None] * (lp.abs() + H[:, None])
    off = p * (size * (e_p[:, None] + 2.0 ** -20 + 2.0 ** -21 * lp.abs()) + (ge.abs() * (e_p + e_h))[:, None])
    D[r, at] += gl
    out["dZ"] = D
    bound["dZ"] = off + (torch.finfo(zt).eps / 2 + 2.0 ** -23) * D.abs() + 1e-37  # (and what exp flushes to zero)
    if top:
        best = torch.sort(z, dim=1, descending=True, stable=True)
        out["top_ids"] = best.indices[:, :top]
        out["top_logp"] = best.values[:, :top] - m[:, None] - ls[:, None]
        bound["top_logp"] = e_ls[:, None] + 2.0 ** -22 * torch.nan_to_num(out["top_logp"], neginf=0.0).abs()
    return out, bound


def _check(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    same = got == want  # infinities among them
    excess = torch.where(same, 0.0, (got - want).abs() - bound)
    assert excess.numel() == 0 or float(excess.max()) <= 1e-30, f"{what}: {float(excess.max()):.3e} over the bound"


def _to(dev, *ts):
    return [None if t is None else t.to(dev) for t in ts]


def _compare(dev, z, y, gl, ge, top, what, zg=None):
    want, bound = _reference(z, y, gl, ge, top)
    yg, glg, geg = _to(dev, y, gl, ge)
    zg = z.to(dev) if zg is None else zg
    logp, entropy, lse, top_logp, top_ids = rgc.rgc_log_prob_forward(zg, yg, top)
    dz = rgc.rgc_log_prob_backward(zg, yg, lse, entropy, glg, geg)
    torch.cuda.synchronize()
    for name, got in (("lse", lse), ("logp", logp), ("entropy", entropy), ("dZ", dz)):
        _check(got, want[name], bound[name], f"{name} {what}")
    assert dz.dtype == z.dtype and bool((entropy >= 0).all())
    if top:
        assert torch.equal(top_ids.cpu(), want["top_ids"]), f"top_ids {what}"
        _check(top_logp, want["top_logp"], bound["top_logp"], f"top_logp {what}")
    else:
        assert top_logp is None and top_ids is None
    return logp, entropy, lse, top_logp, top_ids, dz


# one row, one entry; fewer entries than alternatives hold lanes; ends anywhere in a vector, a batch (8192) and a part
# of a row; rows in one part and in many
SHAPES = [(1, 1, 1), (1, 7, 7), (3, 8, 2), (2, 9, 9), (4, 63, 63), (5, 64, 64), (5, 65, 64), (5, 1000, 5), (64, 4097, 20),
          (300, 8191, 8), (7, 8192, 3), (3, 8193, 64), (33, 16385, 50), (2100, 300, 4), (2049, 8200, 1), (2, 70001, 20),
          (1, 131072, 20), (9, 131071, 64), (2048, 20003, 8), (1000, 12345, 0)]


@pytest.mark.parametrize("zt", [BF, F32])
@pytest.mark.parametrize("rows,V,top", SHAPES)
def test_against_64_bits(dev, rows, V, top, zt):
    print(rows, V, top, zt, flush=True)
    _compare(dev, *_inputs(rows, V, zt, rows + V), top, f"{rows}x{V} {zt} top {top}")


@pytest.mark.parametrize("V", [4096, 4104, 4095, 2056, 40003])
@pytest.mark.parametrize("rows", [1, 40, 700])
def test_parts_of_rows(dev, rows, V):
    _compare(dev, *_inputs(rows, V, BF, rows + V), 10, f"{rows}x{V}")


@pytest.mark.parametrize("order", ["rising", "falling", "equal", "two values", "late"])
@pytest.mark.parametrize("rows", [2, 2100])
def test_ties_and_orders(dev, order, rows):
    """Rows in which every entry is a new largest, none is, all are equal, or the largest come last."""
    V = 9000
    v = {"rising": torch.arange(V) / 512.0, "falling": -torch.arange(V) / 512.0, "equal": torch.full((V,), 0.25),
         "two values": (torch.arange(V) % 7 == 3).float(), "late": torch.where(torch.arange(V) >= V - 100, 3.0, 1.0)}[order]
    z = v.repeat(rows, 1)
    z[1] = v.roll(4321)
    y = torch.arange(rows) % V
    gl, ge = torch.ones(rows), torch.full((rows,), 0.5)
    _compare(dev, z, y, gl, ge, 33, f"{order} fp32")
    _compare(dev, z.to(BF), y, gl, ge, 33, f"{order} bf16")


@pytest.mark.parametrize("zt", [BF, F32])
@pytest.mark.parametrize("V", [40, 20000])
def test_masks(dev, zt, V):
    """Rows of -inf alone, of one allowed entry, with the type's lowest value as a mask, and of that alone."""
    low = torch.finfo(zt).min
    z = torch.randn(6, V, generator=torch.Generator().manual_seed(1)).to(zt)
    z[0] = -INF
    z[1] = -INF
    z[1, V - 3] = 2.0
    z[2, ::2] = low
    z[3] = low
    z[4, 1:] = -INF
    z[5, 5] = 0.0
    z[5, 6] = -0.0
    y = torch.tensor([3, V - 3, 1, V - 1, 7, 5])  # (row 4's token is forbidden)
    gl, ge = torch.ones(6), torch.ones(6)
    zg, yg, glg, geg = _to(dev, z, y, gl, ge)
    logp, entropy, lse, top_logp, top_ids = rgc.rgc_log_prob_forward(zg, yg, 10)
    dz = rgc.rgc_log_prob_backward(zg, yg, lse, entropy, glg, geg)
    assert float(lse[0]) == -INF and float(logp[0]) == -INF and float(entropy[0]) == 0 and bool((dz[0] == 0).all())
    assert top_ids[0].tolist() == list(range(10)) and bool((top_logp[0] == -INF).all())
    assert float(logp[1]) == 0 and float(entropy[1]) == 0 and float(lse[1]) == 2 and top_ids[1, 0] == V - 3
    assert bool((dz[1] == 0).all()) and float(logp[4]) == -INF and float(entropy[4]) == 0
    keep = torch.tensor([1, 2, 3, 5])
    want, bound = _reference(z[keep], y[keep], gl[keep], ge[keep], 10)
    for name, got in (("lse", lse), ("logp", logp), ("entropy", entropy), ("dZ", dz), ("top_logp", top_logp)):
        _check(got.cpu()[keep], want[name], bound[name], name)
    assert torch.equal(top_ids.cpu()[keep], want["top_ids"])


@pytest.mark.parametrize("zt", [BF, F32])
@pytest.mark.parametrize("V", [50, 30000])
def test_nan_and_infinity_stay_in_their_rows(dev, zt, V):
    z, y, gl, ge = _inputs(5, V, zt, 3, ignored=0.0)
    good, gbound = _reference(z, y, gl, ge, 4)
    z[1, 17] = NAN
    z[1, 33] = -NAN
    z[1, 20] = INF
    z[3, V - 1] = INF
    zg, yg, glg, geg = _to(dev, z, y, gl, ge)
    logp, entropy, lse, top_logp, top_ids = rgc.rgc_log_prob_forward(zg, yg, 4)
    dz = rgc.rgc_log_prob_backward(zg, yg, lse, entropy, glg, geg)
    for r in (1, 3):
        assert all(bool(torch.isnan(t[r]).all()) for t in (logp, entropy, lse, top_logp, dz)), r
    assert top_ids[1].tolist()[:3] == [17, 33, 20] and top_ids[3, 0] == V - 1
    keep = torch.tensor([0, 2, 4])
    for name, got in (("lse", lse), ("logp", logp), ("entropy", entropy), ("dZ", dz), ("top_logp", top_logp)):
        _check(got.cpu()[keep], good[name][keep], gbound[name][keep], name)
    assert torch.equal(top_ids.cpu()[keep], good["top_ids"][keep])


@pytest.mark.parametrize("spread", [1e-3, 30.0, 300.0, 2000.0, 2e4, 1e30])
def test_flat_peaked_and_extreme(dev, spread):
    _compare(dev, *_inputs(20, 5003, F32, 5, spread=spread, masked=0.0), 6, f"spread {spread}")


@pytest.mark.parametrize("rows", [3, 2100])
def test_without_tokens(dev, rows):
    z, y, gl, ge = _inputs(rows, 5000, BF, 6)
    want, bound = _reference(z, y, gl, ge, 3)
    logp, entropy, lse, top_logp, top_ids = rgc.rgc_log_prob_forward(z.to(dev), top=3)
    assert logp is None and torch.equal(top_ids.cpu(), want["top_ids"])
    _check(entropy, want["entropy of all"], bound["entropy of all"], "entropy")
    _check(lse, want["lse"], bound["lse"], "lse")


@pytest.mark.parametrize("which", ["logp", "entropy"])
def test_one_gradient_alone(dev, which):
    z, y, gl, ge = _inputs(50, 3001, BF, 7)
    gl, ge = (gl, None) if which == "logp" else (None, ge)
    want, bound = _reference(z, y, gl, ge, 0)
    zg, yg, glg, geg = _to(dev, z, y, gl, ge)
    _, entropy, lse, _, _ = rgc.rgc_log_prob_forward(zg, yg)
    dz = rgc.rgc_log_prob_backward(zg, yg, lse, None if which == "logp" else entropy, glg, geg)
    _check(dz, want["dZ"], bound["dZ"], "dZ")


def test_tokens_that_take_no_part(dev):
    """Their rows may hold anything; their gradient is zero, their alternatives their row's."""
    z, y, gl, ge = _inputs(30, 9000, F32, 8, ignored=0.0)
    out = torch.arange(30) % 3 == 0
    y[out] = torch.tensor([-1, -100, 9000, 2 ** 40, -(2 ** 40)])[torch.arange(int(out.sum())) % 5]
    want, bound = _reference(z, y, gl, ge, 2)
    gl[out], ge[out] = NAN, INF
    zg, yg, glg, geg = _to(dev, z, y, gl, ge)
    logp, entropy, lse, top_logp, top_ids = rgc.rgc_log_prob_forward(zg, yg, 2)
    zg[0] = NAN
    dz = rgc.rgc_log_prob_backward(zg, yg, lse, entropy, glg, geg)
    assert bool((logp.cpu()[out] == 0).all()) and bool((entropy.cpu()[out] == 0).all()) and bool((dz.cpu()[out] == 0).all())
    for name, got in (("lse", lse), ("logp", logp), ("entropy", entropy), ("dZ", dz)):
        _check(got, want[name], bound[name], name)
    assert torch.equal(top_ids.cpu(), want["top_ids"])


@pytest.mark.parametrize("zt", [BF, F32])
@pytest.mark.parametrize("V,off,pad", [(4096, 1, 3), (1003, 5, 0), (20001, 0, 64), (9, 7, 1)])
def test_strided_rows_and_what_lies_around_them(dev, zt, V, off, pad):
    rows = 12
    z, y, gl, ge = _inputs(rows, V, zt, 9)
    full = torch.full((rows + 2, off + V + pad), NAN, dtype=zt, device=dev)
    zs = full[1:-1, off:off + V]
    zs.copy_(z.to(dev))
    dz = _compare(dev, z, y, gl, ge, 5, f"strided {V}", zg=zs)[-1]
    out = torch.full((rows + 2, off + V + pad), 3.0, dtype=zt, device=dev)
    yg, glg, geg = _to(dev, y, gl, ge)
    _, entropy, lse, _, _ = rgc.rgc_log_prob_forward(zs, yg)
    rgc.rgc_log_prob_backward(zs, yg, lse, entropy, glg, geg, dZ=out[1:-1, off:off + V])
    assert torch.equal(out[1:-1, off:off + V], dz)
    inside = torch.zeros_like(out, dtype=torch.bool)
    inside[1:-1, off:off + V] = True
    assert bool((out[~inside] == 3).all())
    rgc.rgc_log_prob_backward(zs, yg, lse, entropy, glg, geg, dZ=zs)  # in place
    assert torch.equal(zs, dz) and bool(torch.isnan(full[~inside]).all())


def test_no_rows(dev):
    z, y, f = torch.zeros(0, 50, device=dev), torch.zeros(0, dtype=torch.int64, device=dev), torch.zeros(0, device=dev)
    logp, entropy, lse, top_logp, top_ids = rgc.rgc_log_prob_forward(z, y, 4)
    assert logp.shape == entropy.shape == lse.shape == (0,) and top_logp.shape == top_ids.shape == (0, 4)
    assert rgc.rgc_log_prob_backward(z, y, lse, entropy, f, f).shape == (0, 50)


def test_offsets_past_two_to_the_32(dev):
    """Three rows 2^31 elements apart: 17 GB of bf16, of which the rows alone are written."""
    V, ld = 50001, 2 ** 31 - 8
    try:
        flat = torch.empty(2 * ld + V, dtype=BF, device=dev)
    except torch.cuda.OutOfMemoryError:
        pytest.skip("memory")
    zs = flat.as_strided((3, V), (ld, 1))
    z, y, gl, ge = _inputs(3, V, BF, 10, ignored=0.0)
    zs.copy_(z.to(dev))
    dz = _compare(dev, z, y, gl, ge, 9, "far rows", zg=zs)[-1]
    yg, glg, geg = _to(dev, y, gl, ge)
    _, entropy, lse, _, _ = rgc.rgc_log_prob_forward(zs, yg)
    rgc.rgc_log_prob_backward(zs, yg, lse, entropy, glg, geg, dZ=zs)
    assert torch.equal(zs, dz)


@pytest.mark.parametrize("zt", [BF, F32])
def test_far_rows_in_place(dev, zt):
    """Rows with |lse| above 1024 between near ones, over several batches: one workgroup makes each, in place too."""
    z, y, gl, ge = _inputs(6, 20003, zt, 21, ignored=0.0)
    z[1] += 3000
    z[2] = torch.finfo(zt).min
    z[4] = torch.where(z[4] == -INF, z[4], z[4] * 500 - 5000)
    y[1], y[4] = int(z[1].float().argmax()), int(z[4].float().argmax())
    dz = _compare(dev, z, y, gl, ge, 3, f"far {zt}")[-1]
    zg, yg, glg, geg = _to(dev, z, y, gl, ge)
    _, entropy, lse, _, _ = rgc.rgc_log_prob_forward(zg, yg)
    assert int((lse.abs() >= 1024).sum()) >= 2
    rgc.rgc_log_prob_backward(zg, yg, lse, entropy, glg, geg, dZ=zg)
    assert torch.equal(zg, dz)


def test_more_rows_than_a_launch_has_workgroups(dev):
    rows, V = (1 << 20) + 5, 9
    z = torch.randn(rows, V, generator=torch.Generator(device=dev).manual_seed(1), device=dev)
    y = torch.arange(rows, device=dev) % V
    g = torch.ones(rows, device=dev)
    logp, entropy, lse, top_logp, top_ids = rgc.rgc_log_prob_forward(z, y, 2)
    dz = rgc.rgc_log_prob_backward(z, y, lse, entropy, g, g)
    lp = torch.log_softmax(z.double(), 1)
    h = -(lp.exp() * lp).sum(1)
    best = torch.sort(z, dim=1, descending=True, stable=True)
    want = -lp.exp() * (1 + lp + h[:, None])
    want[torch.arange(rows, device=dev), y] += 1
    # (u N + 2^-21) (1 + sum p (|d| + d^2)) with N = 100, |d| < 12 and the sums below 20; gradients of size up to 8
    assert torch.equal(top_ids, best.indices[:, :2])
    for got, ref in ((logp, lp.gather(1, y[:, None])[:, 0]), (entropy, h), (top_logp, lp.gather(1, top_ids))):
        assert float((got.double() - ref).abs().max()) <= 2 * 20 * (100 * 2.0 ** -24 + 2.0 ** -21)
    assert float((dz.double() - want).abs().max()) <= 8 * 2 * 20 * (100 * 2.0 ** -24 + 2.0 ** -21)


def test_the_largest_vocabulary(dev):
    V = 1 << 24
    z = torch.randn(2, V, generator=torch.Generator(device=dev).manual_seed(1), device=dev)
    y = torch.tensor([V - 1, 0], device=dev)
    logp, entropy, lse, top_logp, top_ids = rgc.rgc_log_prob_forward(z, y, 64)
    best = torch.sort(z, dim=1, descending=True, stable=True)
    want = torch.logsumexp(z.double(), 1)
    p = torch.softmax(z.double(), 1)
    h = -(p * torch.log_softmax(z.double(), 1)).sum(1)
    # u N with 64 parts of a row: 100 + V / 64 / 1600 roundings, and the terms in d (sum p (|d| + d^2) < 40)
    bound = 2 * ((100 + V / 64 / 1600) * 2.0 ** -24 + 2.0 ** -21) * 41
    assert torch.equal(top_ids, best.indices[:, :64])
    assert float((lse - want).abs().max()) <= bound and float((entropy - h).abs().max()) <= bound
    assert float((top_logp - (best.values[:, :64] - want[:, None])).abs().max()) <= bound


def test_gradient_agrees_with_differences(dev):
    V, h = 60, 2.0 ** -5
    z, y, gl, ge = _inputs(4, V, F32, 11, ignored=0.0, masked=0.0)
    z = (z * 256).round() / 256
    yg, glg, geg = _to(dev, y, gl, ge)
    _, entropy, lse, _, _ = rgc.rgc_log_prob_forward(z.to(dev), yg)
    dz = rgc.rgc_log_prob_backward(z.to(dev), yg, lse, entropy, glg, geg).double().cpu()
    for t, i in ((0, 3), (1, int(y[1])), (3, int(z[3].argmax()))):
        sides = []
        for step in (h, -h):
            zs = z.clone()
            zs[t, i] += step
            logp, ent, _, _, _ = rgc.rgc_log_prob_forward(zs.to(dev), yg)
            sides.append(float((logp.double().cpu() * gl.double() + ent.double().cpu() * ge.double()).sum()))
        slope = (sides[0] - sides[1]) / (2 * h)
        # third derivatives along one logit: of logp a third cumulant of an indicator (below 1), of the entropy sums of
        # such with one log p (below 12 in size here); fp32 errors of 4 values of each over 2 h
        tol = (abs(float(gl[t])) + 40 * abs(float(ge[t]))) * h * h / 6 + 4 * 2.0 ** -18 / (2 * h)
        assert abs(slope - float(dz[t, i])) <= tol, (t, i, slope, float(dz[t, i]), tol)


def _both(st):
    z, y, gl, ge = st
    out = rgc.rgc_log_prob_forward(z, y, 6)
    return (*out, rgc.rgc_log_prob_backward(z, y, out[2], out[1], gl, ge))


def _same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_repeated_calls_give_the_same_bits(dev):
    st = _to(dev, *_inputs(40, 30001, BF, 12))
    first = _both(st)
    assert all(_same(first, _both(st)) for _ in range(3))


def test_captured_and_replayed(dev):
    jobs = []
    for rows, V in ((3, 40000), (2100, 1003)):
        st = _to(dev, *_inputs(rows, V, BF, 13))
        _both(st)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = _both(st)
        jobs.append((st, graph, outs))
    for rep in range(3):
        for st, graph, outs in jobs:
            st[0].copy_(_inputs(*st[0].shape, BF, 14 + rep)[0].to(dev))
            graph.replay()
        torch.cuda.synchronize()
        for st, graph, outs in jobs:
            assert _same(outs, _both(st)), rep


def test_two_streams_at_once(dev):
    jobs = [_to(dev, *_inputs(rows, V, F32, 20)) for rows, V in ((5, 50000), (3000, 700))]
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


def test_autograd(dev):
    """log_prob on a view of masked, scaled logits: the calls' gradient reaches what made them."""
    B, L, V = 2, 9, 1003
    z = torch.randn(B, L, V + 5, generator=torch.Generator().manual_seed(1)).to(dev).requires_grad_()
    y = torch.randint(0, V, (B, L), generator=torch.Generator().manual_seed(2)).to(dev)
    y[1, 3] = -100
    logp, entropy = log_prob((z * 0.5)[..., :V], y)
    a, b = torch.randn(B, L, generator=torch.Generator().manual_seed(3)).to(dev), 0.1
    (logp * a + b * entropy).sum().backward()
    zr = (z.detach().double().cpu() * 0.5)[..., :V].requires_grad_()
    lp = torch.log_softmax(zr, -1)
    live = (y.cpu() >= 0)
    got = lp.gather(-1, y.cpu().clamp(min=0)[..., None])[..., 0]
    ent = -(lp.exp() * lp).sum(-1)
    (torch.where(live, got * a.cpu().double() + b * ent, 0.0)).sum().backward()
    want = torch.zeros(B, L, V + 5, dtype=torch.float64)
    want[..., :V] = 0.5 * zr.grad
    # fp32 throughout: errors of lse and H (2^-18) on gradients of size up to |a| + b (|log p| + H) <= 5
    assert float((z.grad.double().cpu() - want).abs().max()) <= 5 * 2.0 ** -17
    z.grad = None
    log_prob(z[..., :V], y)[1].sum().backward()  # one output alone
    assert bool(torch.isfinite(z.grad).all()) and float(z.grad.abs().max()) > 0
    assert math.isclose(float(z.grad.sum()), 0.0, abs_tol=1e-3)  # (an entropy's gradient sums to zero in each row)
