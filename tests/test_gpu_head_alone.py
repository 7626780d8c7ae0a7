"""The head over inputs that require no gradient (features of a frozen body):
its sketch is trained all the same."""
import pytest
import torch

from rank_randomized_gradient_amd import SketchedCrossEntropy, rgc, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _job(dev, T, V, k, r):
    head = SketchedCrossEntropy(k, V, r, device=dev)
    head.begin_update(1)
    x = synth.normal_bf16((T, k), 1.0, seed=2).to(dev)
    y = (torch.arange(T) * 7 % V).to(dev)
    return head, x, y


@pytest.mark.parametrize("T,V,k,r", [(18, 104, 64, 16), (300, 1032, 136, 16), (200, 520, 64, 4)])
def test_the_sketch_is_added_to(dev, T, V, k, r):
    head, x, y = _job(dev, T, V, k, r)
    assert not x.requires_grad
    loss = head(x, y)
    (loss * torch.linspace(-1, 1, T, device=dev)).sum().backward()
    got = head.sketch.clone()
    head.sketch.zero_()
    xg = x.clone().requires_grad_(True)
    want = head(xg, y)
    (want * torch.linspace(-1, 1, T, device=dev)).sum().backward()
    assert torch.equal(loss, want) and torch.equal(got, head.sketch) and bool((got != 0).any())
    assert xg.grad is not None and x.grad is None


def test_beside_another_term_of_the_loss(dev):
    """Two microbatches; the other term of the objective has parameters of its own."""
    head, x, y = _job(dev, 40, 104, 64, 16)
    other = torch.nn.Parameter(torch.ones(3, device=dev))
    for _ in range(2):
        (head(x, y).mean() + other.sum()).backward()
    _, lse, xp = rgc.rgc_linear_cross_entropy_forward(x, head.weight, y, head.proj)
    c = torch.zeros_like(head.sketch)
    for _ in range(2):
        rgc.rgc_linear_cross_entropy_backward(x, head.weight, y, lse, torch.full((40,), 1 / 40, device=dev), xp, c,
                                              input_grad=False)
    assert torch.equal(head.sketch, c) and bool((other.grad == 2).all())


def test_without_grad_mode_there_is_no_graph(dev):
    head, x, y = _job(dev, 18, 104, 64, 16)
    with torch.no_grad():
        assert not head(x, y).requires_grad
    with torch.inference_mode():
        assert not head(x, y).requires_grad
    with pytest.raises(RuntimeError):
        with torch.no_grad():
            loss = head(x, y)
        loss.sum().backward()


def test_captured_and_replayed(dev):
    """A graph of loss and backward with no input gradient, replayed with new inputs."""
    head, x, y = _job(dev, 200, 520, 64, 16)
    head(x, y).mean().backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = head(x, y)
        loss.mean().backward()
    for rep in range(3):
        x.copy_(synth.normal_bf16(tuple(x.shape), 1.0, seed=20 + rep).to(dev))
        head.sketch.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = loss.detach().clone(), head.sketch.clone()
        head.sketch.zero_()
        want = head(x, y)
        want.mean().backward()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want.detach()) and torch.equal(got[1], head.sketch), rep
