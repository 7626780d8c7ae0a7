"""The head's loss, the norms and AdamW at their largest: offsets past 32 bits,
the most tokens, vocabularies of millions."""
import pytest
import torch

from rank_randomized_gradient_amd import rgc

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _fill(shape, std, seed, dev, dtype=BF):
    g = torch.Generator(device=dev).manual_seed(seed)
    out = torch.empty(shape, dtype=dtype, device=dev)
    rows = max(1, (1 << 26) // shape[-1])
    for i in range(0, shape[0], rows):
        out[i:i + rows] = (torch.randn(out[i:i + rows].shape, generator=g, device=dev) * std).to(dtype)
    return out


def _reference(x, w, y, grad):
    """loss and dX in 64 bits, a stretch of the vocabulary at a time."""
    x = x.double()
    step = max(1, (1 << 25) // w.shape[1])
    spans = [(i, w[i:i + step].double()) for i in range(0, w.shape[0], step)] if w.numel() < 1 << 28 else None
    pieces = (lambda: spans) if spans else (lambda: ((i, w[i:i + step].double()) for i in range(0, w.shape[0], step)))
    lse = torch.full((len(x),), -float("inf"), dtype=torch.float64, device=x.device)
    zt = torch.zeros_like(lse)
    for i, p in pieces():
        z = x @ p.T
        lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        here = (y >= i) & (y < i + len(p))
        zt = torch.where(here, z.gather(1, (y - i).clamp(0, len(p) - 1)[:, None])[:, 0], zt)
    dx = torch.zeros_like(x)
    for i, p in pieces():
        d = torch.exp(x @ p.T - lse[:, None])
        here = (y >= i) & (y < i + len(p))
        d[torch.arange(len(y), device=y.device)[here], (y - i)[here]] -= 1
        dx += (d * grad.double()[:, None]) @ p
    return lse - zt, dx


@pytest.mark.parametrize("T,V,k", [(3, 140001, 16384),  # W holds 4.6 GB
                                   (2, 3000001, 8),     # 46 pieces of the vocabulary
                                   (65536, 264, 64)])   # the most tokens
def test_cross_entropy(dev, T, V, k):
    print(T, V, k, flush=True)
    x, w = _fill((T, k), 1.0, 1, dev), _fill((V, k), k ** -0.5, 2, dev)
    y = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(3)).to(dev)
    y[0] = V - 1
    g = torch.ones(T, device=dev)
    loss, lse, _ = rgc.rgc_linear_cross_entropy_forward(x, w, y)
    dx = rgc.rgc_linear_cross_entropy_backward(x, w, y, lse, g)
    want, dwant = _reference(x, w, y, g)
    # logits of size about 1 with errors far below 2^-16; dX: its own rounding, 2^-8, and that of D's entries, which
    # are small beside the targets' (those are taken exactly)
    assert float((loss.double() - want).abs().max()) < 2.0 ** -16
    assert float((dx.double() - dwant).norm() / dwant.norm()) < 2.0 ** -8


def test_cross_entropy_sketch_of_many_tokens_and_entries(dev):
    T, V, k, r = 40000, 1000, 32, 8  # too many tokens for stacked terms
    x, w = _fill((T, k), 1.0, 4, dev), _fill((V, k), 0.2, 5, dev)
    y = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(6)).to(dev)
    g = torch.randn(T, generator=torch.Generator().manual_seed(7)).to(dev)
    xp, c = _fill((T, r), 1.0, 8, dev), torch.zeros(V, r, device=dev)
    _, lse, _ = rgc.rgc_linear_cross_entropy_forward(x, w, y)
    none = rgc.rgc_linear_cross_entropy_backward(x, w, y, lse, g, xp, c, input_grad=False)
    d = torch.softmax(x.double() @ w.double().T, 1)
    d[torch.arange(T, device=dev), y] -= 1
    want = (d * g.double()[:, None]).T @ xp.double()
    assert none is None and float((c.double() - want).norm() / want.norm()) < 2.0 ** -17


def test_norm_past_two_to_the_32_bytes(dev):
    rows, n = 33001, 65536
    x = _fill((rows, n), 1.0, 9, dev)
    w = torch.linspace(0.5, 1.5, n, device=dev)
    y, mean, rstd = rgc.rgc_layer_norm_forward(x, w)
    dx, dw, db = rgc.rgc_layer_norm_backward(y, x, w, mean, rstd)
    for at in (slice(0, 2), slice(rows - 3, rows)):
        xs = x[at].double()
        c = xs - xs.mean(1, keepdim=True)
        r = 1 / torch.sqrt(c.square().mean(1, keepdim=True) + 1e-5)
        h = y[at].double() * w.double()
        u = c * r
        want = (h - h.mean(1, keepdim=True) - u * (h * u).mean(1, keepdim=True)) * r
        # one rounding to bf16 each, 2^-8 of the value, and fp32 sums far below
        assert float((y[at].double() - u * w.double()).norm() / (u * w.double()).norm()) < 2.0 ** -8
        assert float((dx[at].double() - want).norm() / want.norm()) < 2.0 ** -8
    # a column of the sums, in 64 bits
    c = 65000
    assert abs(float(db[c]) - float(y[:, c].double().sum())) <= 2.0 ** -9 * float(y[:, c].double().abs().sum())


def test_adamw_past_two_to_the_32_bytes(dev):
    n = (1 << 31) + 1003
    p, g = torch.ones(n, dtype=BF, device=dev), torch.full((n,), 0.5, dtype=BF, device=dev)
    m, v = (torch.zeros(n, dtype=torch.float8_e4m3fn, device=dev) for _ in range(2))
    ms, vs = (torch.zeros((n + 127) // 128, device=dev) for _ in range(2))
    rgc.rgc_adamw_batch([p], [g], [m], [v], 2.0 ** -6, 1, seed=5, M_scales=[ms], V_scales=[vs])
    # the first step's size is lr, two steps of bf16 just below 1 and so exact; m = 0.05 and sqrt(v) = 0.5 sqrt(0.001)
    for at in (slice(0, 1000), slice(n - 1003, n), slice((1 << 31) - 500, (1 << 31) + 500)):
        assert bool((p[at].float() - (1 - 2.0 ** -6)).abs().max() <= 2.0 ** -8), at
        unit = ms[torch.arange(n, device=dev)[at] // 128]
        assert bool(((m[at].float() * unit - 0.05).abs() <= 0.05 * 2.0 ** -4).all()), at
        unit = vs[torch.arange(n, device=dev)[at] // 128]
        assert bool(((v[at].float() * unit - 0.5 * 0.001 ** 0.5).abs() <= 0.0159 * 2.0 ** -3).all()), at
