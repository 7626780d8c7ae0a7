"""The binding's refusals of the log probabilities with GPU tensors (each raises
before anything is launched), a Workspace of the caller's, and modules at their edges."""
import pytest
import torch

from rank_randomized_gradient_amd import SketchedCrossEntropy, log_prob, rgc, synth

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _refused(*calls):
    for i, call in enumerate(calls):
        with pytest.raises(rgc.RgcError):
            call()
            pytest.fail(f"call {i} was not refused")


def test_head(dev):
    x, w = torch.zeros(9, 64, dtype=BF, device=dev), torch.zeros(104, 64, dtype=BF, device=dev)
    y, f = torch.zeros(9, dtype=torch.int64, device=dev), torch.zeros(9, device=dev)
    xp, c, p = torch.zeros(9, 16, dtype=BF, device=dev), torch.zeros(104, 16, device=dev), torch.zeros(64, 16, dtype=BF, device=dev)
    fwd, bwd = rgc.rgc_linear_log_prob_forward, rgc.rgc_linear_log_prob_backward
    _refused(lambda: fwd(x.float(), w, y), lambda: fwd(x, w.half(), y), lambda: fwd(x, w, y.int()), lambda: fwd(x, w, y[:8]),
             lambda: fwd(x, w[:, :56], y), lambda: fwd(x.t(), w, y), lambda: fwd(x, w, y.cpu()), lambda: fwd(x, w, y, p[:56]),
             lambda: fwd(x, w, y, p.float()), lambda: fwd(x[:, 1:57], w[:, 1:57], y), lambda: fwd(x[0], w, y),
             lambda: bwd(x, w, y, f[:8], f, f, f), lambda: bwd(x, w, y, f, f, f.double(), f), lambda: bwd(x, w, y, f, f, None, None),
             lambda: bwd(x, w, y, f, None, f, f), lambda: bwd(x, w, y, f, f[:5], f, f), lambda: bwd(x, w, y, f, f, f, f, xp),
             lambda: bwd(x, w, y, f, f, f, f, xp, c[:96]), lambda: bwd(x, w[:100], y, f, f, f, f, xp, c[:100]),
             lambda: bwd(x, w, y, f, f, f, f, dX=x[:8]), lambda: bwd(x, w, y, f, f, f, f, input_grad=False),
             lambda: bwd(x, w, y, f, f, f, f, xp, c, dX=x.clone(), input_grad=False))
    head = SketchedCrossEntropy(64, 104, 16, device=dev)
    _refused(lambda: head.log_prob(x, y))  # no projection yet
    head.begin_update(1)
    _refused(lambda: head.log_prob(x, y.int()), lambda: head.log_prob(x, y[:8]), lambda: head.alternatives(x, 0),
             lambda: head.alternatives(x, 65), lambda: head.alternatives(x.float(), 3), lambda: head.alternatives(x[:, :56], 3),
             lambda: head.alternatives(x.cpu(), 3))
    small = SketchedCrossEntropy(64, 8, 4, device=dev)
    _refused(lambda: small.alternatives(x, 9))  # more than there are


def test_logits(dev):
    z, y, f = torch.zeros(5, 40, device=dev), torch.zeros(5, dtype=torch.int64, device=dev), torch.zeros(5, device=dev)
    fwd, bwd = rgc.rgc_log_prob_forward, rgc.rgc_log_prob_backward
    _refused(lambda: fwd(z.half()), lambda: fwd(z.double()), lambda: fwd(z, y.int()), lambda: fwd(z, y[:4]), lambda: fwd(z, y.cpu()),
             lambda: fwd(z[0]), lambda: fwd(z.t()), lambda: fwd(z[:1].expand(5, 40)), lambda: fwd(z, y, 41), lambda: fwd(z, y, -1),
             lambda: fwd(torch.zeros(5, 100, device=dev), y, 65), lambda: fwd(torch.zeros(5, 0, device=dev), y),
             lambda: bwd(z, y, f, f, None, None), lambda: bwd(z, y, f, None, f, f), lambda: bwd(z, y, f[:4], f, f),
             lambda: bwd(z, y, f, f, f.double()), lambda: bwd(z, y, f, f, f, dZ=z.bfloat16()), lambda: bwd(z, y, f, f, f, dZ=z[:4]),
             lambda: log_prob(z, y.int()), lambda: log_prob(z[None], y))


def test_a_workspace_of_the_callers(dev):
    """One Workspace for all calls, grown on the way: the results of the calls' own."""
    ws = rgc.Workspace(dev)
    for T, V in ((3, 1000), (40, 20000), (5, 3000)):
        x, w = synth.normal_bf16((T, 64), 1.0, seed=T).to(dev), synth.normal_bf16((V, 64), 0.2, seed=V).to(dev)
        y, g = torch.arange(T, device=dev), torch.ones(T, device=dev)
        p, xp = synth.normal_bf16((64, 16), 1.0, seed=1).to(dev), synth.normal_bf16((T, 16), 1.0, seed=2).to(dev)
        runs = []
        for s in (None, ws):
            c = torch.zeros(V, 16, device=dev)
            logp, ent, lse, made = rgc.rgc_linear_log_prob_forward(x, w, y, p, workspace=s)
            dx = rgc.rgc_linear_log_prob_backward(x, w, y, lse, ent, g, g, xp, c, workspace=s)
            z, _ = rgc.rgc_linear_forward(x, w)
            runs.append([logp, ent, made, dx, c, *rgc.rgc_log_prob_forward(z, y, 7, workspace=s),
                         *rgc.rgc_grad_norm_batch([c, dx], 0.1, workspace=s),
                         *rgc.rgc_add_norm_backward(x, x, x, None, None, torch.ones(T, device=dev), bias=False, kind="rms",
                                                    workspace=s)[:2]])
        assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_alternatives_of_no_rows_and_of_one(dev):
    head = SketchedCrossEntropy(64, 104, 16, device=dev)
    logp, ids = head.alternatives(torch.zeros(2, 0, 64, dtype=BF, device=dev), 3)
    assert logp.shape == ids.shape == (2, 0, 3)
    logp, ids = head.alternatives(torch.zeros(64, dtype=BF, device=dev), 64)  # all logits equal
    assert ids.tolist() == list(range(64)) and float((logp + torch.log(torch.tensor(104.0))).abs().max()) < 1e-5


def test_a_module_under_no_grad(dev):
    head = SketchedCrossEntropy(64, 104, 16, device=dev)
    head.begin_update(1)
    x, y = synth.normal_bf16((5, 64), 1.0, seed=1).to(dev), torch.arange(5, device=dev)
    with torch.no_grad():
        logp, entropy = head.log_prob(x, y)
    assert not logp.requires_grad and not entropy.requires_grad and bool((head.sketch == 0).all())


@pytest.mark.parametrize("shape", [(6,), (2, 3)])
@pytest.mark.parametrize("which", ["head", "logits"])
def test_outputs_changed_in_place(dev, which, shape):
    """The log probabilities may be changed in place, with the gradient of what they became; the entropies, which the
    backward reads, are found changed by autograd."""
    x, y = synth.normal_bf16((*shape, 64), 1.0, seed=1).to(dev), torch.arange(6, device=dev).reshape(shape)
    head = SketchedCrossEntropy(64, 104, 16, device=dev)
    head.begin_update(1)
    call = head.log_prob if which == "head" else log_prob
    grads = []
    for change in (lambda t: t.mul_(3.0), lambda t: t * 3.0):
        leaf = x.clone().requires_grad_()
        logp, entropy = call(leaf, y)
        assert logp.shape == entropy.shape == shape
        (change(logp).sum() + entropy.sum()).backward()
        grads.append(leaf.grad)
    assert torch.equal(*grads)
    leaf = x.clone().requires_grad_()
    logp, entropy = call(leaf, y)
    with pytest.raises(RuntimeError, match="in-?place"):
        entropy.mul_(2.0).sum().backward()
