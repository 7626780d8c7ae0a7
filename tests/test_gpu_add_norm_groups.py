"""The residual norm's backward at rows and widths where its workgroups change: both sides of 16 rows to a compute unit, of 512 and
1024 (and 2048) elements, with a workspace of just the queried size. The gradient of X is row by row, so it has
the bits of the same rows called apart; the columns' sums are compared with 64 bits, off by an addition's half step
for each row at most (in sequence) and by the half step of rstd and mean."""
import pytest
import torch

from rank_randomized_gradient_amd import rgc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("n", [512, 513, 1000, 1024, 1025])
@pytest.mark.parametrize("more", [-5, 0, 1, 4100])
def test_either_side(n, xt, more):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda", 0)
    rows = 16 * torch.cuda.get_device_properties(dev).multi_processor_count + more
    print(rows, n, xt, flush=True)
    g = torch.Generator(device=dev).manual_seed(n)
    r = lambda: torch.randn(rows, n, generator=g, device=dev).to(xt)  # noqa: E731
    x, res, dy, ds = r(), r(), r(), r()
    w = 1 + 0.2 * torch.randn(n, generator=g, device=dev)
    s, y, mean, rstd = rgc.rgc_add_norm_forward(x, res, w, w)
    need = rgc.load_library().rgc_add_norm_backward_workspace_size(rows, n)
    ws = rgc.Workspace(dev)
    ws.get(need)
    for bias in (True, False):
        dx, dw, db = rgc.rgc_add_norm_backward(dy, ds, s, w, mean, rstd, bias=bias, workspace=ws)
        again = rgc.rgc_add_norm_backward(dy, ds, s, w, mean, rstd, bias=bias)
        assert all(p is None and q is None or torch.equal(p, q) for p, q in zip((dx, dw, db), again))
        for at in (0, rows // 2, rows - 7):
            part = rgc.rgc_add_norm_backward(dy[at:at + 7], ds[at:at + 7], s[at:at + 7], w, mean[at:at + 7], rstd[at:at + 7])[0]
            assert torch.equal(part, dx[at:at + 7])
        xhat = (s.double() - mean.double()[:, None]) * rstd.double()[:, None]
        step = (rows + 32) * 2.0 ** -24 + 2.0 ** -22
        terms = dy.double() * xhat
        # (x - mean is rounded, to half a step of itself)
        assert bool(((dw - terms.sum(0)).abs() <= step * terms.abs().sum(0) + 1e-30).all())
        if bias:
            assert bool(((db - dy.double().sum(0)).abs() <= step * dy.double().abs().sum(0) + 1e-30).all())
