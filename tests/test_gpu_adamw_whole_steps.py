"""AdamW.step with parameters of several types, devices' calls and step counts:
it takes place as a whole or not at all."""
import pytest
import torch

from rank_randomized_gradient_amd import AdamW, rgc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _params(dev):
    g = torch.Generator().manual_seed(1)
    return [torch.nn.Parameter(torch.randn(n, generator=g).to(t).to(dev)) for n, t in ((300, F32), (500, BF), (77, F32))]


def _grads(params, seed):
    g = torch.Generator().manual_seed(seed)
    for p in params:
        p.grad = torch.randn(p.shape, generator=g).to(p.dtype).to(p.device)


def _bad_grads():
    def off_alignment(p):
        p.grad = torch.zeros(p.numel() + 1, dtype=p.dtype, device=p.device)[1:]

    def strided(p):
        p.grad = torch.zeros(2 * p.numel(), dtype=p.dtype, device=p.device)[::2]

    return [off_alignment, strided]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("spoil", _bad_grads())
def test_a_refused_step_changes_nothing(dev, bits, spoil):
    """The second of two calls is refused; the step made again with good gradients gives the bits of a run without
    the refusal."""
    a, b = AdamW(_params(dev), lr=1e-2, state_bits=bits, seed=3), AdamW(_params(dev), lr=1e-2, state_bits=bits, seed=3)
    for opt in (a, b):
        _grads(opt.params, 5)
        opt.step()
    before = [p.detach().clone() for p in a.params]
    moments = [{k: v.clone() for k, v in s.items() if torch.is_tensor(v)} for s in a.state]
    _grads(a.params, 6)
    spoil(a.params[1])
    with pytest.raises(rgc.RgcError):
        a.step()
    assert a.steps == 1 and all(s["step"] == 1 for s in a.state)
    assert all(torch.equal(p, q) for p, q in zip(a.params, before))
    assert all(torch.equal(s[k].float(), m[k].float()) for s, m in zip(a.state, moments) for k in m)
    for opt in (a, b):
        _grads(opt.params, 7)
        opt.step()
    assert all(torch.equal(p, q) for p, q in zip(a.params, b.params))
    assert all(torch.equal(s[k].float(), t[k].float()) for s, t in zip(a.state, b.state) for k in s if torch.is_tensor(s[k]))


def test_a_scalar_that_is_refused_changes_nothing(dev):
    opt = AdamW(_params(dev), lr=float("nan"))
    before = [p.detach().clone() for p in opt.params]
    _grads(opt.params, 5)
    with pytest.raises(rgc.RgcError):
        opt.step()
    assert opt.steps == 0 and all(torch.equal(p, q) for p, q in zip(opt.params, before))
