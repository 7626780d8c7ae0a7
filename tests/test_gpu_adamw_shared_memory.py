"""An AdamW step whose tensors share memory would write what another workgroup
reads: it is refused."""
import pytest
import torch

from rank_randomized_gradient_amd import rgc

pytestmark = pytest.mark.gpu


def test_tensors_that_overlap_are_refused():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda", 0)
    t = lambda n=128, dtype=torch.float32: torch.zeros(n, dtype=dtype, device=dev)  # noqa: E731
    x, f8 = t(4096), torch.float8_e4m3fn
    for P, G, M, V in (([x[:128], x[64:192]], [t(), t()], [t(), t()], [t(), t()]),  # parameters that overlap
                       ([t()], [t()], [x[:128]], [x[:128]]),  # one tensor as both moments
                       ([x[:128]], [x[64:192]], [t()], [t()]),  # a gradient within what is written
                       ([x[:128]], [t()], [x[64:192]], [t()])):
        with pytest.raises(rgc.RgcError):
            rgc.rgc_adamw_batch(P, G, M, V, 1e-3, 1)
    s = t(1)
    with pytest.raises(rgc.RgcError):  # one scale for both moments
        rgc.rgc_adamw_batch([t()], [t()], [t(dtype=f8)], [t(dtype=f8)], 1e-3, 1, M_scales=[s], V_scales=[s])
    assert bool((x == 0).all())
    g = t().fill_(1.0)
    P = [x[:128], x[128:256]]  # side by side, one gradient for both
    rgc.rgc_adamw_batch(P, [g, g], [t(), t()], [t(), t()], 1e-3, 1)
    assert bool((x[:256] != 0).all()) and bool((x[256:] == 0).all()) and torch.equal(P[0], P[1])
