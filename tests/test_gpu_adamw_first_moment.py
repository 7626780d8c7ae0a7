"""8-bit first moments of AdamW rounded stochastically: their codes against the
step in 64 bits and the documented random bits, and, over many steps, that they
follow the formula in the mean where rounding to nearest would hold them."""
import math

import numpy as np
import pytest
import torch

import oracle as orc
from rank_randomized_gradient_amd import AdamW, rgc
from test_gpu_adamw import BF, F32, F8, B, HP, _blocks, _e4m3, _make, _step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _m_bits(n, tensor, seed):
    """Element e's 16 bits: half e % 2 of word ((e % 8) / 2 + 1) % 4 of its group's Philox call."""
    group = np.arange((n + 7) // 8, dtype=np.uint64)
    words = orc.philox4x32_10(group & np.uint64(0xFFFFFFFF), group >> np.uint64(32), np.full_like(group, 4),
                              np.full_like(group, tensor), *orc.seed_to_key(seed))
    words = np.stack([np.asarray(w, dtype=np.uint64) for w in words], 1).astype(np.int64)
    e = np.arange(n)
    return torch.from_numpy(words[e // 8, (e % 8 // 2 + 1) % 4] >> (16 * (e % 2)) & 0xFFFF)


@pytest.mark.parametrize("pt", [BF, F32])
@pytest.mark.parametrize("gt", [BF, F32])
@pytest.mark.parametrize("beta1", [0.0, 0.9, 0.99])
def test_codes_against_64_bits(dev, pt, gt, beta1):
    """As the second moments' codes: the 64-bit value, its code's lower neighbour and the random threshold. Where the
    value lies within the fp32 error (and 2^-15 of a step, the threshold's own 16 bits) of the threshold either
    neighbour is right. All else, p and sqrt(v), has the bits of the call that rounds m to nearest."""
    sizes, seed, lr, t = [1, 9, 128, 129, 2049, 100003], 0x13579BDF02468, 1e-2, 7
    hp = dict(HP, beta1=beta1)
    ts = [_make(n, pt, gt, True, 40 + i) for i, n in enumerate(sizes)]
    runs = []
    for how in ("stochastic", "nearest") if beta1 <= 0.9 else ("stochastic",):
        on = [{k: v.to(dev) for k, v in s.items()} for s in ts]
        rgc.rgc_adamw_batch(*[[s[k] for s in on] for k in "PGMV"], lr, t, seed=seed, m_rounding=how,
                            M_scales=[s["Ms"] for s in on], V_scales=[s["Vs"] for s in on], **hp)
        runs.append(on)
    for i, (s, new) in enumerate(zip(ts, runs[0])):
        n = sizes[i]
        _, m, _, em, _ = _step(s, lr, t, 1.0, **hp)
        top = _blocks(m).abs().amax(1)
        got = new["Ms"].double().cpu()
        edge = ((torch.log2(top.clamp(min=2.0 ** -140)) + 0.5).remainder(1) - 0.5).abs() < 2.0 ** -20
        assert bool(((got == torch.exp2(torch.floor(torch.log2(top)) - 7)) | edge).all())
        unit = got.repeat_interleave(B)[:n]
        q, x = new["M"].double().cpu(), m / unit
        low, step = _e4m3(x.abs())
        reach = (x.abs() - low) / step + _m_bits(n, i, seed).double() / 65536
        want = torch.where(reach >= 1, low + step, low)
        tie = (reach - 1).abs() <= em / unit / step + 2.0 ** -15
        off = (q.abs() - want).abs()
        assert bool((off == 0)[~tie].all()), int((off != 0)[~tie].sum())
        assert bool((off[tie] <= step[tie] * 1.0001).all()) and int(tie.sum()) <= n / 16 + 2
        assert bool(((q == 0) | (torch.sign(q) == torch.sign(x))).all())
        for other in runs[1:]:
            for k in ("P", "V", "Ms", "Vs"):
                assert torch.equal(new[k].float(), other[i][k].float()), k


def _fresh(n, dev):
    return (torch.zeros(n, dtype=F8, device=dev), torch.zeros(n // B, device=dev),
            torch.zeros(n, dtype=F8, device=dev), torch.zeros(n // B, device=dev))


@pytest.mark.parametrize("beta1,steps", [(0.9, 22), (0.95, 45), (0.99, 230)])
def test_first_moments_decay_in_expectation(dev, beta1, steps):
    """Without gradients the mean of many follows beta1^t, to a tenth here, and goes on to nothing."""
    n = 1 << 16
    p, g = torch.zeros(n, device=dev), torch.zeros(n, device=dev)
    m, ms, v, vs = _fresh(n, dev)
    m.copy_(torch.full((n,), 200.0, device=dev))
    ms.fill_(2.0 ** -10)
    start = float((m.float() * ms.repeat_interleave(B)).mean())

    def step(t):
        rgc.rgc_adamw_batch([p], [g], [m], [v], 1e-3, t + 1, seed=t, beta1=beta1, M_scales=[ms], V_scales=[vs],
                            m_rounding="stochastic")

    for t in range(steps):
        step(t)
    ratio = float((m.float() * ms.repeat_interleave(B)).mean()) / start / beta1 ** steps
    # a step's rounding is off by at most 2^-16 of a code's step, itself at most 1/8 of the value; its variance is at
    # most (value/16)^2, so an element's relative variance grows by a factor of 1 + 1/256 a step
    tol = steps * 2.0 ** -19 + 6 * math.sqrt(math.expm1(steps / 256) / n)
    assert abs(ratio - 1) < tol, (ratio, tol)
    for t in range(steps, 12 * steps):  # a factor of 10^-12 and below: the blocks' scales follow
        step(t)
    assert float((m.float() * ms.repeat_interleave(B)).abs().max()) < 1e-6 * start


@pytest.mark.parametrize("beta1,steps", [(0.9, 150), (0.95, 300), (0.99, 1500)])
def test_first_moments_follow_a_steady_gradient(dev, beta1, steps):
    """The mean of m / g is 1 - beta1^t. Each step adds a variance of at most (m/16)^2 and keeps beta1^2 of the one
    before, with m^2 = 1 + variance: a steady state of (1/256) / (1 - beta1^2 - 1/256). The threshold's bias, 2^-19 of m
    a step, adds up to 1 / (1 - beta1) times that."""
    n = 1 << 16
    g = torch.rand(n, generator=torch.Generator().manual_seed(1)).add(0.5).to(dev)
    p = torch.zeros(n, device=dev)
    m, ms, v, vs = _fresh(n, dev)
    for t in range(steps):
        rgc.rgc_adamw_batch([p], [g], [m], [v], 1e-3, t + 1, seed=t, beta1=beta1, M_scales=[ms], V_scales=[vs],
                            m_rounding="stochastic")
    mean = float((m.float() * ms.repeat_interleave(B) / g).mean())
    tol = 6 * math.sqrt(1 / 256 / (1 - beta1 ** 2 - 1 / 256) / n) + 2.0 ** -19 / (1 - beta1)
    assert abs(mean - (1 - beta1 ** steps)) < tol, (mean, tol)


@pytest.mark.parametrize("beta1", [0.9, 0.95, 0.99])
def test_what_no_gradient_reaches_stands_still(dev, beta1):
    """Rows of an embedding that batches reach for 100 steps and then no more, beside rows that they go on reaching
    (each block half and half): once the momentum has run out they stay where they are, as with float32 moments. How
    far they go meanwhile: m's sum has its mean, and per element a variance below its square (a steady state's
    0.25 at beta1 = 0.99 and less below, and as much while it decays), 1/sqrt(v) is within a third in the mean (a
    relative variance of sqrt(v) of less than 0.1: at most (1/16)^2 in each of the about 25 steps that build it up), so
    twice the float32 run's root mean square is a wide bound."""
    n, live, dead = 1 << 14, 100, 1500
    moved = {}
    for bits in (8, 32):
        p = torch.nn.Parameter(torch.zeros(n, device=dev))
        opt = AdamW([p], lr=1e-3, betas=(beta1, 0.999), weight_decay=0.0, state_bits=bits, seed=3)
        gen = torch.Generator(device=dev).manual_seed(5)
        reached = (torch.arange(n, device=dev) % B) < B // 2
        for t in range(live + dead):
            g = torch.randn(n, generator=gen, device=dev) * 0.01
            p.grad = g if t < live else g * reached
            opt.step()
            if t == live - 1:
                at = p.detach().clone()
            if t == live + dead - 300:
                late = p.detach().clone()
        rest = ~reached
        moved[bits] = float((p.detach() - at)[rest].square().mean().sqrt())
        # Momentum that ran out: 1200 steps leave 6e-6 of it at beta1 = 0.99, nothing below. In 8 bits it ends in a few
        # subnormal steps of its block, 2^-16 of the block's largest m at most (of the live ones' spread, 0.01
        # sqrt((1 - beta1) / (1 + beta1)), five times). c such steps become beta1 c, between c - 1 and c, so they only
        # die, each with probability 1 - beta1: an element keeps at most 2^16 beta1^1200 of them in the mean, 0.38 at
        # 0.99 and none below; eight are beyond chance for 8192 elements (Poisson's tail above eight: 10^-10). Each
        # moves p by lr / sqrt(v) (half the mean's sqrt(v) at least) in each of the 300 steps.
        unit = 2.0 ** -16 * 5 * 0.01 * math.sqrt((1 - beta1) / (1 + beta1))
        root = 0.01 * math.sqrt((1 - 0.999 ** live) * 0.999 ** dead / (1 - 0.999 ** (live + dead)))
        steps = 8 if bits == 8 and 2 ** 16 * beta1 ** 1200 * n > 1e-3 else 0
        assert float((p.detach() - late)[rest].abs().max()) <= 1e-3 * moved[bits] + 1e-6 + steps * 300 * 1e-3 * unit / (root / 2)
    assert moved[8] < 2 * moved[32], moved
