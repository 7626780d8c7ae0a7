"""rgc_adamw_batch against the same step in 64 bits.

Bounds, u = 2^-24: m and v are sums of two products of three factors at most,
rounded at every operation: 4 u of the sum of the terms' magnitudes. The step's
quotient takes a square root, three products, a sum and a division: 10 u more;
the new parameter is off by that of the step, 2 u of the old one and the
rounding of its type (a whole step for a stochastic one). 8-bit moments are
compared as codes: nearest rounding of m may differ from the oracle's only
where the 64-bit value lies within 2^-20 of a rounding border; sqrt(v) likewise
at its random threshold.
"""
import math

import numpy as np
import pytest
import torch

import oracle as orc
from rank_randomized_gradient_amd import rgc

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
B = rgc.ADAMW_BLOCK
U = 2.0 ** -24
# UNDECIDED: elements whose 64-bit value lies on a rounding border, so that either neighbour is right. They say
# nothing about the kernel and must be few for a test to say much. With 8-bit moments and bf16 gradients they are
# not only chance: m = (9 c + g) / 10 of an e4m3 c and a bf16 g falls exactly on a border of e4m3 for some pairs (c
# = 88 units of 2^-12, g = 0.08984375 is one), 11 of the 300 elements of one tensor here. Sixteen steps of e4m3 to a
# binade and borders half way between make one in sixteen a bound for values on the lattice of the steps' halves.
HP = dict(beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _bits(n, tensor, seed):
    """The parameters' and the second moments' 16 random bits of n elements, by the oracle's Philox."""
    group = np.arange((n + 7) // 8, dtype=np.uint64)
    words = orc.philox4x32_10(group & np.uint64(0xFFFFFFFF), group >> np.uint64(32), np.full_like(group, 4),
                              np.full_like(group, tensor), *orc.seed_to_key(seed))
    words = np.stack([np.asarray(w, dtype=np.uint64) for w in words], 1)
    low, high = (words & 0xFFFF).astype(np.int64), (words >> 16).astype(np.int64)
    p = np.stack([low, high], 2).reshape(-1)[:n]
    v = np.stack([high, low], 2).reshape(-1)[:n]
    return torch.from_numpy(p), torch.from_numpy(v)


def _make(n, pt, gt, eight, seed):
    g = torch.Generator().manual_seed(seed)
    t = {"P": torch.randn(n, generator=g).to(pt), "G": (torch.randn(n, generator=g) * 0.1).to(gt)}
    if eight:
        k = (n + B - 1) // B
        t["M"] = (torch.randn(n, generator=g) * 60).clamp(-240, 240).to(F8)
        t["V"] = (torch.rand(n, generator=g) * 200).to(F8)
        t["Ms"] = torch.exp2(torch.randint(-14, -9, (k,), generator=g).float())
        t["Vs"] = torch.exp2(torch.randint(-12, -8, (k,), generator=g).float())
    else:
        t["M"] = torch.randn(n, generator=g) * 0.01
        t["V"] = (torch.randn(n, generator=g) * 0.1).square()
    return t


def _blocks(x):
    n = x.numel()
    out = torch.zeros((n + B - 1) // B * B, dtype=torch.float64)
    out[:n] = x
    return out.view(-1, B)


def _step(t, lr, step, scale, beta1, beta2, eps, weight_decay):
    """(p, m, v, bound of p) in 64 bits, before any rounding."""
    g = t["G"].double() * scale
    if "Ms" in t:
        m = (_blocks(t["M"].double()) * t["Ms"].double()[:, None]).view(-1)[:g.numel()]
        v = (_blocks(t["V"].double()) * t["Vs"].double()[:, None]).view(-1)[:g.numel()].square()
    else:
        m, v = t["M"].double(), t["V"].double()
    em = 4 * U * ((beta1 * m).abs() + ((1 - beta1) * g).abs())
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    denom = torch.sqrt(v / (1 - beta2 ** step)) + eps
    size = lr / (1 - beta1 ** step)
    p = t["P"].double()
    new = p * (1 - lr * weight_decay) - size * m / denom
    bound = size * (em + 10 * U * m.abs()) / denom + 3 * U * p.abs() + U * new.abs()
    return new, m, v, em, bound


def _e4m3(x):
    """e4m3 value of a 64-bit one at or below 448, rounded down, and the step there."""
    e = torch.floor(torch.log2(x.clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.floor(x / step) * step, step


def _check_eight(old, new, m, v, em, seed, tensor):
    n = m.numel()
    root = torch.sqrt(v)
    for vals, err, code, scale in ((m, em, "M", "Ms"), (root, 6 * U * root, "V", "Vs")):
        rows = _blocks(vals)
        top = rows.abs().amax(1)
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - 7
        want = torch.exp2(e.clamp(min=-126))
        got = new[scale].double().cpu()
        # a block whose largest value lies within rounding of a power of two may go either way
        edge = ((torch.log2(top.clamp(min=2.0 ** -140)) + 0.5).remainder(1) - 0.5).abs() < 2.0 ** -20
        assert bool(((got == want) | edge).all()), scale
        unit = got.repeat_interleave(B)[:n]
        q = new[code].double().cpu()
        x = vals / unit
        low, step = _e4m3(x.abs())
        frac = (x.abs() - low) / step
        if code == "M":
            up = frac > 0.5
            tie = (frac - 0.5).abs() <= err / unit / step + 2.0 ** -20
        else:
            bits = _bits(n, tensor, seed)[1].double() / 65536
            up = frac + bits >= 1
            tie = (frac + bits - 1).abs() <= err / unit / step + 2.0 ** -15
        mag = torch.where(up, low + step, low)
        if code == "V":
            mag = torch.where(vals > 0, mag.clamp(min=2.0 ** -9), mag)
        off = (q.abs() - mag).abs()
        assert bool((off == 0)[~tie].all()), f"{code}: {int((off != 0)[~tie].sum())} codes differ"
        assert bool((off[tie] <= step[tie] * 1.0001).all()), code
        assert int(tie.sum()) <= n / 16 + 2  # see UNDECIDED
        assert bool(((q == 0) | (torch.sign(q) == torch.sign(x))).all())
    assert bool((new["V"].double().cpu()[v > 0] > 0).all())


def _run(dev, sizes, pt, gt, eight, step, scale=None, lr=1e-2, seed=0x123456789ABC):
    ts = [_make(n, pt, gt, eight, 10 + i) for i, n in enumerate(sizes)]
    on = [{k: v.to(dev) for k, v in t.items()} for t in ts]
    gs = torch.tensor([scale], device=dev) if scale is not None else None
    names = lambda k: [t[k] for t in on]  # noqa: E731
    rgc.rgc_adamw_batch(names("P"), names("G"), names("M"), names("V"), lr, step, seed=seed,
                        M_scales=names("Ms") if eight else None, V_scales=names("Vs") if eight else None, grad_scale=gs,
                        **HP)
    torch.cuda.synchronize()
    s32 = float(torch.tensor(scale if scale is not None else 1.0, dtype=F32))
    for i, (t, new) in enumerate(zip(ts, on)):
        n = sizes[i]
        if n == 0:
            continue
        p, m, v, em, bound = _step(t, lr, step, s32, **HP)
        got = new["P"].double().cpu()
        if pt == BF:
            # v + 16 random bits in the low half, then the high half: exact but for the error before rounding
            ulp = torch.exp2(torch.floor(torch.log2(p.abs().clamp(min=2.0 ** -126))) - 7)
            low = torch.floor(p.abs() / ulp) * ulp
            bits = _bits(n, i, seed)[0].double() / 65536
            mag = torch.where((p.abs() - low) / ulp + bits >= 1, low + ulp, low)
            tie = ((p.abs() - low) / ulp + bits - 1).abs() <= bound / ulp + 2.0 ** -15
            edge = (p.abs() - low <= bound) | (low + ulp - p.abs() <= bound)
            off = (got.abs() - mag).abs()
            assert bool((off == 0)[~tie & ~edge].all()), f"P {i}"
            assert bool((off <= ulp * 2.0001 + bound).all()), f"P {i}"
            assert int((tie | edge).sum()) <= n / 16 + 2  # see UNDECIDED
        else:
            assert bool(((got - p).abs() <= bound).all()), f"P {i}: {float(((got - p).abs() - bound).max())}"
        if eight:
            _check_eight(t, new, m, v, em, seed, i)
        else:
            assert bool(((new["M"].double().cpu() - m).abs() <= em).all()), f"M {i}"
            assert bool(((new["V"].double().cpu() - v).abs() <= 4 * U * v.abs()).all()), f"V {i}"


SIZES = [1, 7, 8, 9, 127, 128, 129, 0, 2047, 2048, 2049, 5000, 4096, 100003]


@pytest.mark.parametrize("pt", [BF, F32])
@pytest.mark.parametrize("gt", [BF, F32])
@pytest.mark.parametrize("eight", [False, True])
def test_against_64_bits(dev, pt, gt, eight):
    print(pt, gt, eight, flush=True)
    _run(dev, SIZES, pt, gt, eight, step=7, scale=0.37)


@pytest.mark.parametrize("step", [1, 2, 1000, 10 ** 7])
@pytest.mark.parametrize("eight", [False, True])
def test_steps(dev, step, eight):
    _run(dev, [1000], F32, F32, eight, step=step)


def test_more_tensors_than_a_launch_holds(dev):
    _run(dev, [300 + 13 * i for i in range(101)], BF, BF, True, step=3)


def test_tensors_of_nothing(dev):
    _run(dev, [0, 0], BF, BF, False, step=1)
    _run(dev, [0], F32, F32, True, step=1)
    _run(dev, [], F32, F32, False, step=1)


def test_what_lies_between_the_tensors_stays(dev):
    flat = {k: torch.full((1024,), 3.0, device=dev) for k in "PGMV"}
    cut = [(16, 37), (64, 99), (512, 513)]
    args = [[flat[k][a:b] for a, b in cut] for k in "PGMV"]
    rgc.rgc_adamw_batch(*args, 0.5, 1)
    for k in "PMV":
        inside = torch.zeros(1024, dtype=torch.bool, device=dev)
        for a, b in cut:
            inside[a:b] = True
        assert bool((flat[k][~inside] == 3).all()) and bool((flat[k][inside] != 3).all())
    assert bool((flat["G"] == 3).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("eight", [False, True])
def test_a_scale_that_is_not_finite_skips_the_step(dev, bad, eight):
    t = {k: v.to(dev) for k, v in _make(1000, BF, BF, eight, 1).items()}
    old = {k: v.clone() for k, v in t.items()}
    kw = dict(M_scales=[t["Ms"]], V_scales=[t["Vs"]]) if eight else {}
    rgc.rgc_adamw_batch([t["P"]], [t["G"]], [t["M"]], [t["V"]], 0.1, 1, grad_scale=torch.tensor([bad], device=dev), **kw)
    for k in t:
        a, b = (x.view(torch.uint8) if x.dtype == F8 else x for x in (t[k], old[k]))
        assert torch.equal(a, b), k


def test_states_of_zero_bytes_and_zero_gradients(dev):
    """Fresh 8-bit states, and gradients that are all zero: nothing moves but the decay, and no NaN appears."""
    n = 300
    p = torch.linspace(-1, 1, n, device=dev)
    old = p.clone()
    m, v = torch.zeros(n, dtype=F8, device=dev), torch.zeros(n, dtype=F8, device=dev)
    ms, vs = torch.zeros(3, device=dev), torch.zeros(3, device=dev)
    rgc.rgc_adamw_batch([p], [torch.zeros(n, device=dev)], [m], [v], 0.1, 1, M_scales=[ms], V_scales=[vs], weight_decay=0.5)
    assert torch.allclose(p, old * 0.95, rtol=1e-6, atol=0)
    assert bool((m.float() == 0).all()) and bool((v.float() == 0).all())
    assert bool((ms == 2.0 ** -126).all()) and bool((vs == 2.0 ** -126).all())
    g = torch.full((n,), 1e-3, device=dev)
    g[5] = 0
    p2 = p.clone()
    rgc.rgc_adamw_batch([p], [g], [m], [v], 0.1, 1, M_scales=[ms], V_scales=[vs])
    # the first step's size is lr for every gradient that is not zero
    moved = p2 - p
    assert float(moved[5]) == 0 and float((moved[:5] - 0.1).abs().max()) < 1e-4
    assert bool((v.float()[:5] > 0).all()) and float(v.float()[5]) == 0


def test_infinities_and_nan_spoil_their_own_elements_only(dev):
    n = 256
    t = {k: v.to(dev) for k, v in _make(n, F32, F32, True, 4).items()}
    clean = {k: v.clone() for k, v in t.items()}
    t["G"][3], t["G"][200] = float("inf"), float("nan")
    clean["G"][3] = clean["G"][200] = 0.0
    for s in (t, clean):
        rgc.rgc_adamw_batch([s["P"]], [s["G"]], [s["M"]], [s["V"]], 0.1, 5, seed=9, M_scales=[s["Ms"]], V_scales=[s["Vs"]])
    keep = torch.ones(n, dtype=torch.bool, device=dev)
    keep[3] = keep[200] = False
    assert torch.equal(t["P"][keep], clean["P"][keep])
    for c, s in (("M", "Ms"), ("V", "Vs")):
        a = t[c].float() * t[s].repeat_interleave(B)
        b = clean[c].float() * clean[s].repeat_interleave(B)
        assert torch.isnan(a[~keep]).all()
        # the left-out elements may have been their block's largest: then the others keep finer steps
        same = t[s].repeat_interleave(B) == clean[s].repeat_interleave(B)
        assert torch.equal(a[keep & same], b[keep & same])
        assert torch.isfinite(a[keep]).all()


def test_small_second_moments_decay_in_expectation(dev):
    """sqrt(v) loses (1 - beta2) / 2 of itself a step, far below half a step of its code: over many steps without
    gradients its mean over many elements follows beta2^(t/2) all the same."""
    n, steps = 1 << 16, 200
    p, g = torch.zeros(n, device=dev), torch.zeros(n, device=dev)
    m, ms = torch.zeros(n, dtype=F8, device=dev), torch.zeros(n // B, device=dev)
    v, vs = torch.full((n,), 200.0, device=dev).to(F8), torch.full((n // B,), 2.0 ** -10, device=dev)
    start = float((v.float() * vs.repeat_interleave(B)).mean())
    for t in range(steps):
        rgc.rgc_adamw_batch([p], [g], [m], [v], 1e-3, t + 1, seed=t, M_scales=[ms], V_scales=[vs])
    ratio = float((v.float() * vs.repeat_interleave(B)).mean()) / start
    # a step's rounding is unbiased but for the 16-bit threshold (at most 2^-16 of a code's step, itself at most
    # 1/8 of the value, a step); the spread of the mean: steps * (value/8)^2 / 4 in variance an element
    tol = steps * 2.0 ** -19 + 6 * math.sqrt(steps / 4 / n) / 8
    assert abs(ratio - 0.999 ** (steps / 2)) < tol, (ratio, tol)


def test_bf16_parameters_move_in_expectation(dev):
    """A step of 2^-14 of a parameter, far below its last place, moves the mean of many by that much."""
    n, lr = 1 << 18, 2.0 ** -14
    p = torch.full((n,), 1.5, device=dev).bfloat16()
    rgc.rgc_adamw_batch([p], [torch.ones(n, device=dev)], [torch.zeros(n, device=dev)], [torch.zeros(n, device=dev)], lr, 1,
                        seed=77)
    moved = 1.5 - float(p.double().mean())
    spread = math.sqrt(lr * 2.0 ** -7 / n)  # a step of 2^-7 taken with probability lr / 2^-7
    assert abs(moved - lr) < 6 * spread + 2.0 ** -23


def test_the_same_seed_gives_the_same_bits_and_another_others(dev):
    out = []
    for seed in (5, 5, 6):
        t = {k: v.to(dev) for k, v in _make(5000, BF, BF, True, 2).items()}
        rgc.rgc_adamw_batch([t["P"]], [t["G"]], [t["M"]], [t["V"]], 1e-3, 3, seed=seed, M_scales=[t["Ms"]],
                            V_scales=[t["Vs"]])
        out.append(t)
    assert torch.equal(out[0]["P"], out[1]["P"]) and torch.equal(out[0]["V"].float(), out[1]["V"].float())
    assert not torch.equal(out[0]["P"], out[2]["P"]) and not torch.equal(out[0]["V"].float(), out[2]["V"].float())


def test_captured_and_replayed(dev):
    states = [[{k: v.to(dev) for k, v in _make(n, BF, F32, True, 20 + n).items()} for n in (3000, 77)] for _ in range(2)]

    def call(ts):
        rgc.rgc_adamw_batch([t["P"] for t in ts], [t["G"] for t in ts], [t["M"] for t in ts], [t["V"] for t in ts], 1e-2, 4,
                            seed=3, M_scales=[t["Ms"] for t in ts], V_scales=[t["Vs"] for t in ts])

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(states[0])
    for rep in range(3):
        for ts in states:
            for t in ts:
                t["G"].mul_(-1.5)
        graph.replay()
        call(states[1])
        torch.cuda.synchronize()
        for a, b in zip(*states):
            assert all(torch.equal(a[k].float(), b[k].float()) for k in a), rep
