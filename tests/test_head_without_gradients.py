"""Losses and log probabilities where no gradient is recorded need no projection: what scores a model that is not
trained, or not yet. The values are the training forward's."""
import pytest
import torch

from rank_randomized_gradient_amd import SketchedCrossEntropy, rgc, synth


@pytest.fixture
def seen(monkeypatch):
    """The projections that the library's calls are given."""
    given = []

    def loss(x, w, t, p=None):
        given.append(p)
        return x.float().sum(1), x.float().sum(1), None

    def log_prob(x, w, t, p=None):
        given.append(p)
        return x.float().sum(1), x.float().sum(1), x.float().sum(1), None

    monkeypatch.setattr(rgc, "rgc_linear_cross_entropy_forward", loss)
    monkeypatch.setattr(rgc, "rgc_linear_log_prob_forward", log_prob)
    return given


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_no_projection_is_asked_for(seen, off):
    head = SketchedCrossEntropy(8, 16, 4, device="cpu")
    x, y = torch.ones(2, 3, 8, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int64)
    with off():
        loss, (logp, entropy) = head(x, y), head.log_prob(x, y)
    assert loss.shape == logp.shape == entropy.shape == (2, 3) and seen == [None, None]
    for call in (head, head.log_prob):  # where a gradient is recorded it is
        with pytest.raises(rgc.RgcError, match="begin_update"):
            call(x, y)
    head.proj_seed = 1
    head(x, y), head.log_prob(x, y)
    assert seen[2] is head.proj and seen[3] is head.proj
    with off():
        head(x, y), head.log_prob(x, y)
    assert seen[4:] == [None, None]


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(5, 104), (200, 5000)])
def test_the_training_forwards_values(T, V):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w = synth.normal_bf16((V, 128), 0.2, seed=1)
    x, y = synth.normal_bf16((T, 128), 1.0, seed=2).cuda(), (torch.arange(T) % V).cuda()
    y[1] = -100
    trained, scored = (SketchedCrossEntropy(128, V, 16, device="cuda", weight=w) for _ in range(2))
    trained.begin_update(1)
    want = [trained(x, y), *trained.log_prob(x, y)]
    with torch.no_grad():
        got = [scored(x, y), *scored.log_prob(x, y)]
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and not any(t.requires_grad for t in got)
