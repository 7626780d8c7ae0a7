"""Targets as text has them: a few of very many tokens, most of one or none. The
tokens of one target are added to its row of the sketch in batches, in token
order."""
import pytest
import torch

from rank_randomized_gradient_amd import rgc
from test_gpu_cross_entropy import _check, _inputs, _reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _targets(kind, T, V):
    if kind == "counts":  # entry v is the target of v tokens, spread over the call: every size of a batch up to a wave's
        y = torch.repeat_interleave(torch.arange(V), torch.arange(V))[:T]
        return y[torch.randperm(len(y), generator=torch.Generator().manual_seed(1))]
    if kind == "frequent":
        p = 1 / torch.arange(1, V + 1, dtype=torch.float64)
        return torch.multinomial(p, T, replacement=True, generator=torch.Generator().manual_seed(2))
    return torch.full((T,), V - 1)


@pytest.mark.parametrize("kind", ["counts", "frequent", "one"])
@pytest.mark.parametrize("T,V,k,r", [(2415, 72, 264, 256), (1000, 520, 64, 4), (600, 264, 136, 80)])
def test_sketch_of_frequent_targets(dev, kind, T, V, k, r):
    print(kind, T, V, k, r, flush=True)
    x, w, y, gr, xp, c = _inputs(T, V, k, r, 30, ignored=0.0)
    y[:] = torch.cat([_targets(kind, T, V), torch.full((T,), -100)])[:T]
    want, bound = _reference(x, w, y, gr, xp, c)
    cg = c.to(dev)
    _, lse, _ = rgc.rgc_linear_cross_entropy_forward(x.to(dev), w.to(dev), y.to(dev))
    rgc.rgc_linear_cross_entropy_backward(x.to(dev), w.to(dev), y.to(dev), lse, gr.to(dev), xp.to(dev), cg, input_grad=False)
    _check(cg, want["C"], bound["C"], "C")
    # the targets' entries are exact to fp32
    assert float((cg.double().cpu() - want["C"]).norm() / want["C"].norm()) < 2.0 ** -18
