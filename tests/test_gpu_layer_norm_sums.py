"""The weights' gradients of the widest norm over rows whose offsets pass 2^32
bytes, every column against 64 bits."""
import pytest
import torch

from rank_randomized_gradient_amd import rgc

pytestmark = pytest.mark.gpu


def test_every_column_of_the_sums_past_two_to_the_32_bytes():
    """Rows from 32768 on lie past 2^32 bytes. A few rows, the last and the first past that border among them, have
    gradients of 64 beside others of size one, so that a row lost or taken twice moves db by 64.

    The sums: 64 slices of 516 rows in sequence and at most 32 joining additions, (rows/64 + 32) 2^-24 of the
    magnitudes. xhat for dw: mean and variance of 65536 elements in fp32 are off by 2^-17 of their magnitudes at most (64
    additions a thread and ten joining ones, below 2^-17.7), so xhat by 2^-17 mean|x| rstd + 2^-16 |xhat|."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda", 0)
    rows, n = 33001, 65536
    gen = torch.Generator(device=dev).manual_seed(1)
    x, dy = (torch.empty(rows, n, dtype=torch.bfloat16, device=dev) for _ in range(2))
    mean, rstd, size = (torch.empty(rows, dtype=torch.float64, device=dev) for _ in range(3))
    for i in range(0, rows, 1024):
        x[i:i + 1024] = torch.randn(x[i:i + 1024].shape, generator=gen, device=dev) + 0.5
        dy[i:i + 1024] = torch.randn(x[i:i + 1024].shape, generator=gen, device=dev)
        part = x[i:i + 1024].double()
        mean[i:i + 1024], size[i:i + 1024] = part.mean(1), part.abs().mean(1)
        rstd[i:i + 1024] = 1 / torch.sqrt((part - part.mean(1, keepdim=True)).square().mean(1) + 1e-5)
    dy[[0, 515, 516, 32767, 32768, 32999, 33000]] = 64.0
    w = torch.linspace(0.5, 1.5, n, device=dev)
    _, mu, rs = rgc.rgc_layer_norm_forward(x, w)
    _, dw, db = rgc.rgc_layer_norm_backward(dy, x, w, mu, rs)
    steps = (rows / 64 + 32) * 2.0 ** -24
    for c in range(0, n, 2048):
        at = slice(c, c + 2048)
        d = dy[:, at].double()
        xhat = (x[:, at].double() - mean[:, None]) * rstd[:, None]
        off = 2.0 ** -17 * (size * rstd)[:, None] + 2.0 ** -16 * xhat.abs()
        bound = steps * d.abs().sum(0)
        assert float(bound.max()) < 2  # far below a row of 64
        assert bool(((db[at].double() - d.sum(0)).abs() <= bound + 2.0 ** -24 * d.sum(0).abs()).all()), c
        want = (d * xhat).sum(0)
        bound = (d.abs() * off).sum(0) + steps * (d * xhat).abs().sum(0) + 2.0 ** -24 * want.abs()
        assert bool(((dw[at].double() - want).abs() <= bound).all()), c
