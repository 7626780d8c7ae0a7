"""The gradients' global norm and clipping: rgc_grad_norm_batch, rgc_scale_batch,
clip_grad_norm and AdamW's max_norm.

The squares are added in fp64, at most 2^20 additions one after the other here, so that
a norm is off by 2^-33 of itself before its one rounding to fp32 (2^-24), and so is the
scale. The multiplication in place is one fp32 product and one rounding: the
same bits as torch's.
"""
import math

import pytest
import torch

from rank_randomized_gradient_amd import AdamW, clip_grad_norm, rgc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
U = 2.0 ** -24 + 2.0 ** -32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _tensors(sizes, dtypes, seed, dev, off=0, std=1e-2):
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = dtypes[i % len(dtypes)]
        whole = torch.full((off + n + 3,), 7.0, dtype=t, device=dev)
        whole[off:off + n] = (torch.randn(n, generator=g) * std * (1 + i % 5)).to(t).to(dev)
        out.append(whole[off:off + n])
    return out


def _norm(ts):
    return math.sqrt(math.fsum(float((t.double().cpu() ** 2).sum()) for t in ts))


def _near(got, want):
    assert abs(float(got) - want) <= U * abs(want), (float(got), want)


# one element; ends anywhere in a vector and in a round of the workgroup (2048); one chunk and one past (8192); more
# tensors than a launch's table holds; tensors of nothing among them
LISTS = [[1], [7, 8, 9], [2047, 2048, 2049], [8191, 8192, 8193, 8200], [0, 5, 0, 0, 100003, 0], [1000003],
         [4096] * 145, [17 + 13 * i for i in range(161)], [33] * 500, [0] * 200 + [3]]


@pytest.mark.parametrize("dtypes", [(BF,), (F32,), (BF, F32, F32)])
@pytest.mark.parametrize("i", range(len(LISTS)))
def test_norm_and_scale(dev, i, dtypes):
    sizes = LISTS[i]
    print(i, dtypes, flush=True)
    ts = _tensors(sizes, dtypes, i, dev, off=i % 3)
    before = [t.clone() for t in ts]
    n = _norm(ts)
    norm, scale = rgc.rgc_grad_norm_batch(ts)
    assert norm.shape == scale.shape == (1,) and norm.dtype == F32
    _near(norm, n)
    assert float(scale) == 1
    norm, scale = rgc.rgc_grad_norm_batch(ts, 0.25 * n)
    _near(norm, n)
    _near(scale, 0.25)
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    assert rgc.rgc_scale_batch(ts, scale) is ts
    for a, b in zip(ts, before):
        assert torch.equal(a, (b.float() * scale).to(b.dtype))
        whole = a._base if a._base is not None else a
        assert bool((whole[:i % 3] == 7).all()) and bool((whole[i % 3 + len(a):] == 7).all())


def test_limits_of_max_norm(dev):
    ts = _tensors([1000], (F32,), 1, dev)
    n = _norm(ts)
    for limit, want in ((INF, 1.0), (2 * n, 1.0), (0.0, 0.0), (1e-300, 1e-300 / n)):
        norm, scale = rgc.rgc_grad_norm_batch(ts, limit)
        _near(norm, n)
        assert abs(float(scale) - want) <= U * want + 1e-45
    norm, scale = rgc.rgc_grad_norm_batch([torch.zeros(50, device=dev)], 0.0)
    assert float(norm) == 0 and float(scale) == 1


def test_a_factor_that_comes_first(dev):
    """grad_scale multiplies the norm by its size and joins the scale."""
    ts = _tensors([3000, 41], (BF, F32), 2, dev)
    n = _norm(ts)
    for s in (0.125, -3.0, 0.0):
        f = torch.tensor([s], device=dev)
        norm, scale = rgc.rgc_grad_norm_batch(ts, 0.5 * n, f)
        _near(norm, abs(s) * n)
        _near(scale, s * min(1.0, 0.5 / abs(s)) if s else 0.0)
    for s in (INF, NAN):
        norm, scale = rgc.rgc_grad_norm_batch(ts, 1.0, torch.tensor(s, device=dev))
        assert not math.isfinite(float(norm)) and math.isnan(float(scale))


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_is_not_finite(dev, bad, dtype):
    """One such gradient anywhere: the norm says so, the scale is NaN, and nothing is multiplied."""
    for at in (0, 2000, 20006):
        ts = _tensors([5, 20007, 9], (dtype,), 3, dev)
        ts[1][at] = bad
        norm, scale = rgc.rgc_grad_norm_batch(ts, 1.0)
        assert not math.isfinite(float(norm)) and math.isnan(float(scale))
        before = [t.clone() for t in ts]
        rgc.rgc_scale_batch(ts, scale)
        assert all(torch.equal(a.nan_to_num(3.0), b.nan_to_num(3.0)) for a, b in zip(ts, before))


@pytest.mark.parametrize("size", [1e-44, 1e-30, 1e30, 3e38])
def test_squares_neither_overflow_nor_vanish(dev, size):
    for dtype in (BF, F32):
        t = torch.full((3000,), size, device=dev).to(dtype)
        n = float(t[0].double()) * math.sqrt(3000)
        norm, scale = rgc.rgc_grad_norm_batch([t], 0.5 * n)
        if n > 3.4e38:
            assert float(norm) == INF  # fp32 holds no such number, the scale is one all the same
        else:
            assert abs(float(norm) - n) <= U * n + 2e-45
        _near(scale, 0.5 if n else 1.0)  # (bf16 has no 1e-44: zeros, and a max_norm of zero clips nothing of them)


def test_tensors_of_nothing(dev):
    empty = [torch.zeros(0, device=dev), torch.zeros(0, 5, dtype=BF, device=dev)]
    norm, scale = rgc.rgc_grad_norm_batch(empty, 1.0)
    assert float(norm) == 0 and float(scale) == 1
    rgc.rgc_scale_batch(empty, scale)


def test_many_chunks(dev):
    """More elements than the join has partial sums for at the smallest chunk, past 2^32 bytes."""
    n = (1 << 31) + 4099
    t = torch.full((n,), 0.5, dtype=BF, device=dev)
    t[n - 1] = 300.0
    norm, scale = rgc.rgc_grad_norm_batch([t, torch.full((3,), 2.0, device=dev)], 1000.0)
    want = math.sqrt(0.25 * (n - 1) + 9e4 + 12)
    _near(norm, want)
    _near(scale, 1000 / want)
    half = torch.tensor([0.5], device=dev)
    rgc.rgc_scale_batch([t], half)
    assert float(t[0]) == float(t[1 << 31]) == float(t[n - 2]) == 0.25 and float(t[n - 1]) == 150
    assert float(rgc.rgc_grad_norm_batch([t])[0]) == float(torch.tensor(math.sqrt(0.0625 * (n - 1) + 22500), dtype=torch.float64).float())


def test_a_tensor_twice(dev):
    t = _tensors([500], (F32,), 4, dev)[0]
    _near(rgc.rgc_grad_norm_batch([t, t])[0], math.sqrt(2) * _norm([t]))
    one = torch.ones(1, device=dev)
    for bad in ([t, t], [t, t[10:20]], [t[:100], t[99:]]):
        with pytest.raises(rgc.RgcError):
            rgc.rgc_scale_batch(bad, one)
    rgc.rgc_scale_batch([t[:100], t[100:]], one)


def test_refusals(dev):
    t, s = torch.ones(10, device=dev), torch.ones(1, device=dev)
    for call in (lambda: rgc.rgc_grad_norm_batch([]), lambda: rgc.rgc_grad_norm_batch([t.double()]),
                 lambda: rgc.rgc_grad_norm_batch([t.half()]), lambda: rgc.rgc_grad_norm_batch([t, t.cpu()]),
                 lambda: rgc.rgc_grad_norm_batch([t.cpu()]), lambda: rgc.rgc_grad_norm_batch([t[::2]]),
                 lambda: rgc.rgc_grad_norm_batch([t, None]), lambda: rgc.rgc_grad_norm_batch([t], -1.0),
                 lambda: rgc.rgc_grad_norm_batch([t], NAN), lambda: rgc.rgc_grad_norm_batch([t], 1.0, s.double()),
                 lambda: rgc.rgc_grad_norm_batch([t], 1.0, torch.ones(2, device=dev)),
                 lambda: rgc.rgc_grad_norm_batch([t], 1.0, s.cpu()), lambda: rgc.rgc_scale_batch([t], s.cpu()),
                 lambda: rgc.rgc_scale_batch([t], torch.ones(2, device=dev)), lambda: rgc.rgc_scale_batch([t.half()], s)):
        with pytest.raises(rgc.RgcError):
            call()
    assert rgc.rgc_scale_batch([], s) == []


def test_repeated_calls_give_the_same_bits(dev):
    ts = _tensors([100003, 5, 777777], (BF, F32), 5, dev)
    first = rgc.rgc_grad_norm_batch(ts, 0.1)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, rgc.rgc_grad_norm_batch(ts, 0.1)))


def test_captured_and_replayed(dev):
    jobs = []
    for seed, sizes in ((1, [1000, 20, 30000]), (2, [64] * 300)):
        ts = _tensors(sizes, (BF, F32), seed, dev)

        def call(ts=ts):
            norm, scale = rgc.rgc_grad_norm_batch(ts, 0.01)
            rgc.rgc_scale_batch(ts, scale)
            return norm, scale

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = call()
        jobs.append((ts, graph, outs, sizes))
    for rep in range(3):
        for seed, (ts, graph, outs, sizes) in enumerate(jobs):
            new = _tensors(sizes, (BF, F32), 10 * rep + seed, dev)
            for a, b in zip(ts, new):
                a.copy_(b)
            graph.replay()
            torch.cuda.synchronize()
            norm, scale = rgc.rgc_grad_norm_batch(new, 0.01)
            rgc.rgc_scale_batch(new, scale)
            assert torch.equal(norm, outs[0]) and torch.equal(scale, outs[1])
            assert all(torch.equal(a, b) for a, b in zip(ts, new)), rep


def test_two_streams_at_once(dev):
    jobs = [_tensors([300001, 17], (F32,), 6, dev), _tensors([100] * 200, (BF,), 7, dev)]
    want = [rgc.rgc_grad_norm_batch(j, 0.1) for j in jobs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(4):
        for n in (0, 1):
            with torch.cuda.stream(streams[n]):
                got[n].append(rgc.rgc_grad_norm_batch(jobs[n], 0.1))
    torch.cuda.synchronize()
    for n in (0, 1):
        assert all(torch.equal(a, b) for g in got[n] for a, b in zip(g, want[n]))


def _params(dev, seed):
    g = torch.Generator().manual_seed(seed)
    ps = [torch.nn.Parameter(torch.randn(n, generator=g).to(t).to(dev)) for n, t in ((1000, F32), (777, BF), (64, F32))]
    for p in ps[:2]:
        p.grad = torch.randn(p.shape, generator=g).to(p.dtype).to(dev)
    return ps


def test_clip_grad_norm(dev):
    ps = _params(dev, 1)
    before = [p.grad.clone() for p in ps[:2]]
    n = _norm(before)
    norm = clip_grad_norm([ps[0], ps[1], ps[2], ps[0]], 0.5 * n)  # (listed twice, and one without a gradient)
    assert norm.dim() == 0
    _near(norm, n)
    scale = rgc.rgc_grad_norm_batch(before, 0.5 * n)[1]
    assert all(torch.equal(p.grad, (b.float() * scale).to(b.dtype)) for p, b in zip(ps, before))
    kept = [p.grad.clone() for p in ps[:2]]
    clip_grad_norm(ps, 10 * n)
    assert all(torch.equal(p.grad, b) for p, b in zip(ps, kept))
    assert float(clip_grad_norm([ps[2]], 1.0)) == 0


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_clips_as_it_reads(dev, bits):
    """step(max_norm) is the step with the scale handed over, over parameters of both types, and leaves the gradients."""
    runs = []
    for own in (True, False):
        ps = _params(dev, 2)
        opt = AdamW(ps, lr=1e-2, state_bits=bits, seed=3)
        for _ in range(3):
            grads = [p.grad.clone() for p in ps[:2]]
            if own:
                norm = opt.step(max_norm=1.5)
                _near(norm, _norm(grads))
            else:
                _, scale = rgc.rgc_grad_norm_batch([p.grad for p in ps[:2]], 1.5)
                assert opt.step(grad_scale=scale) is None
            assert all(torch.equal(p.grad, g) for p, g in zip(ps, grads))
        runs.append([p.detach().clone() for p in ps])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_adamw_skips_a_step_that_is_not_finite(dev):
    ps = _params(dev, 4)
    opt = AdamW(ps, lr=1e-2)
    opt.step(max_norm=1.0)
    ps[1].grad[5] = INF
    before = [p.detach().clone() for p in ps]
    norm = opt.step(max_norm=1.0)
    assert float(norm) == INF and all(torch.equal(p, b) for p, b in zip(ps, before))
    scaled = opt.step(grad_scale=torch.tensor([0.5], device=dev), max_norm=1.0)
    assert float(scaled) == INF
    ps[1].grad[5] = 0.0
    norm = opt.step(grad_scale=torch.tensor([0.5], device=dev), max_norm=1.0)
    _near(norm, 0.5 * _norm([p.grad for p in ps[:2]]))
    assert not torch.equal(ps[0], before[0])
