"""The binding's refusals of the head's loss, the norms and AdamW with GPU
tensors (each raises before anything is launched), and a Workspace of the
caller's that grows from call to call."""
import pytest
import torch

from rank_randomized_gradient_amd import LayerNorm, SketchedCrossEntropy, rgc, synth

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rgc.load_library()
    return torch.device("cuda", 0)


def _refused(call):
    with pytest.raises(rgc.RgcError):
        call()


def test_cross_entropy(dev):
    x, w = torch.zeros(9, 64, dtype=BF, device=dev), torch.zeros(104, 64, dtype=BF, device=dev)
    y, f = torch.zeros(9, dtype=torch.int64, device=dev), torch.zeros(9, device=dev)
    xp, c, p = torch.zeros(9, 16, dtype=BF, device=dev), torch.zeros(104, 16, device=dev), torch.zeros(64, 16, dtype=BF, device=dev)
    fwd, bwd = rgc.rgc_linear_cross_entropy_forward, rgc.rgc_linear_cross_entropy_backward
    for call in (lambda: fwd(x.float(), w, y), lambda: fwd(x, w.half(), y), lambda: fwd(x, w, y.int()), lambda: fwd(x, w, y[:8]),
                 lambda: fwd(x, w[:, :56], y), lambda: fwd(x.t(), w, y), lambda: fwd(x, w, y.cpu()), lambda: fwd(x, w, y, p[:56]),
                 lambda: fwd(x, w, y, p.float()), lambda: fwd(x[:, 1:57], w[:, 1:57], y),  # rows off 16-byte alignment
                 lambda: fwd(x[:, :60], w[:, :60], y), lambda: fwd(x[0], w, y),
                 lambda: bwd(x, w, y, f[:8], f), lambda: bwd(x, w, y, f, f.double()), lambda: bwd(x, w, y, f, f, xp),
                 lambda: bwd(x, w, y, f, f, xp, c[:96]), lambda: bwd(x, w, y, f, f, xp[:8], c), lambda: bwd(x, w, y, f, f, xp, c.bfloat16()),
                 lambda: bwd(x, w[:100], y, f, f, xp, c[:100]), lambda: bwd(x, w, y, f, f, dX=x[:8]),
                 lambda: bwd(x, w, y, f, f, dX=torch.zeros(9, 64, device=dev)),
                 lambda: bwd(x, w, y, f, f, xp, c, dX=x.clone(), input_grad=False)):
        _refused(call)
    head = SketchedCrossEntropy(64, 104, 16, device=dev)
    _refused(lambda: head(x, y))  # no projection yet
    head.begin_update(1)
    _refused(lambda: head(x, y.int()))
    _refused(lambda: head(x, y[:8]))


def test_norms(dev):
    x, w = torch.zeros(5, 40, dtype=BF, device=dev), torch.ones(40, device=dev)
    s = torch.ones(5, device=dev)
    fwd, bwd = rgc.rgc_layer_norm_forward, rgc.rgc_layer_norm_backward
    for call in (lambda: fwd(x.half()), lambda: fwd(x, w[:39]), lambda: fwd(x, w.half()), lambda: fwd(x, w, w.bfloat16()),
                 lambda: fwd(x, w, kind="batch"), lambda: fwd(x, w, eps=-1.0), lambda: fwd(x, w, eps=float("nan")),
                 lambda: fwd(x.t(), w[:5]), lambda: fwd(x[0], w), lambda: fwd(x, w, Y=x.float()), lambda: fwd(x, w.cpu()),
                 lambda: fwd(x[:1].expand(5, 40)), lambda: fwd(torch.zeros(2, 65537, dtype=BF, device=dev)),
                 lambda: fwd(torch.zeros(2, 0, dtype=BF, device=dev)),
                 lambda: bwd(x.float(), x, w, s, s), lambda: bwd(x[:4], x, w, s, s), lambda: bwd(x, x, w, None, s),
                 lambda: bwd(x, x, w, s, s[:4]), lambda: bwd(x, x, w, s.double(), s), lambda: bwd(x, x, w, s, s, dX=x[:4])):
        _refused(call)
    _refused(lambda: LayerNorm(40, device=dev)(x[:, :39]))
    _refused(lambda: LayerNorm(40, kind="max", device=dev))


def test_adamw(dev):
    def t(n=64, dtype=F32):
        return torch.zeros(n, dtype=dtype, device=dev)

    step = lambda P, G, M, V, **kw: rgc.rgc_adamw_batch(P, G, M, V, 1e-3, 1, **kw)  # noqa: E731
    for call in (lambda: step([t()], [t(63)], [t()], [t()]), lambda: step([t()], [t()], [t(dtype=BF)], [t()]),
                 lambda: step([t(dtype=torch.float16)], [t()], [t()], [t()]),
                 lambda: step([t(), t(dtype=BF)], [t(), t()], [t(), t()], [t(), t()]),
                 lambda: step([t()], [t().cpu()], [t()], [t()]), lambda: step([t(128)[::2]], [t()], [t()], [t()]),
                 lambda: step([t(65)[1:]], [t()], [t()], [t()]),  # off 16-byte alignment
                 lambda: step([t()], [t()], [t(dtype=F8)], [t(dtype=F8)]),
                 lambda: step([t()], [t()], [t(dtype=F8)], [t(dtype=F8)], M_scales=[t(1)], V_scales=[t(2)]),
                 lambda: step([t()], [t()], [t()], [t()], M_scales=[t(1)], V_scales=[t(1)]),
                 lambda: step([t()], [t()], [t()], [t()], grad_scale=t(2)), lambda: step([t()], [t()], [t()], [t()], beta1=1.0),
                 lambda: step([t()], [t()], [t()], [t()], eps=0.0), lambda: step([1.0], [t()], [t()], [t()]),
                 lambda: rgc.rgc_adamw_batch([t()], [t()], [t()], [t()], 1e-3, 0)):
        with pytest.raises((rgc.RgcError, AttributeError)):
            call()


def test_a_workspace_of_the_callers(dev):
    ws = rgc.Workspace(dev)
    for T, V, k, r in ((40, 200, 64, 16), (300, 3000, 264, 16), (10, 96, 64, 0)):
        x, w = synth.normal_bf16((T, k), 1.0, seed=T).to(dev), synth.normal_bf16((V, k), 0.1, seed=V).to(dev)
        y = (torch.arange(T) % V).to(dev)
        g = torch.ones(T, device=dev)
        xp = synth.normal_bf16((T, r), 1.0, seed=1).to(dev) if r else None
        c = [torch.zeros(V, r, device=dev) if r else None for _ in range(2)]
        a, la, _ = rgc.rgc_linear_cross_entropy_forward(x, w, y)
        b, lb, _ = rgc.rgc_linear_cross_entropy_forward(x, w, y, workspace=ws)
        assert torch.equal(a, b) and torch.equal(la, lb)
        assert torch.equal(rgc.rgc_linear_cross_entropy_backward(x, w, y, la, g, xp, c[0]),
                           rgc.rgc_linear_cross_entropy_backward(x, w, y, la, g, xp, c[1], workspace=ws))
        assert not r or torch.equal(*c)
        n, mu, rs = rgc.rgc_layer_norm_forward(x)
        for p, q in zip(rgc.rgc_layer_norm_backward(n, x, None, mu, rs),
                        rgc.rgc_layer_norm_backward(n, x, None, mu, rs, workspace=ws)):
            assert torch.equal(p, q)
