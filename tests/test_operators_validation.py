"""Refusals of the head's loss, the norms and AdamW (CPU only: every call here
is rejected on the host, or has nothing to do, before any launch)."""
import ctypes

import pytest
import torch

from rank_randomized_gradient_amd import rgc
from rank_randomized_gradient_amd.adamw import AdamW

OK, NULL, SHAPE, UNSUP, ALIGN, WS, VALUE = 0, 1, 2, 3, 4, 5, 7
FAKE = 0x10000  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    return rgc.load_library()


def _call(fn, defaults, **kw):
    assert set(kw) <= set(defaults), set(kw) - set(defaults)
    return fn(*{**defaults, **kw}.values())


FWD = dict(X=FAKE, ldx=64, W=FAKE, ldw=64, P=FAKE, targets=FAKE, loss=FAKE, lse=FAKE, XP=FAKE, T=16, V=100, k=64, r=16,
           ws=FAKE, n=1 << 30, s=None)
BWD = dict(X=FAKE, ldx=64, W=FAKE, ldw=64, targets=FAKE, lse=FAKE, grad=FAKE, XP=FAKE, C=FAKE, dX=FAKE, lddx=64, T=16,
           V=104, k=64, r=16, ws=FAKE, n=1 << 40, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, X=None, W=None, targets=None, loss=None, lse=None, ws=None), OK),
    (dict(T=-1), SHAPE), (dict(V=0), SHAPE), (dict(k=0), SHAPE), (dict(r=-1), SHAPE), (dict(r=128), SHAPE),
    (dict(ldx=56), SHAPE), (dict(ldw=56), SHAPE),
    (dict(r=24), UNSUP), (dict(k=60, ldx=64, ldw=64), UNSUP), (dict(T=65537), UNSUP), (dict(V=(1 << 24) + 1), UNSUP),
    (dict(k=65544, ldx=65544, ldw=65544), UNSUP), (dict(ldx=(1 << 23) + 8), UNSUP),
    (dict(X=None), NULL), (dict(W=None), NULL), (dict(targets=None), NULL), (dict(loss=None), NULL), (dict(lse=None), NULL),
    (dict(P=None), NULL), (dict(XP=None), NULL),
    (dict(X=FAKE + 2), ALIGN), (dict(ldx=68), ALIGN), (dict(targets=FAKE + 4), ALIGN), (dict(loss=FAKE + 2), ALIGN),
    (dict(P=FAKE + 8), ALIGN), (dict(ws=FAKE + 128), ALIGN),
    (dict(ws=None), WS), (dict(n=100), WS),
])
def test_cross_entropy_forward(lib, kw, want):
    assert _call(lib.rgc_linear_cross_entropy_forward, FWD, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, X=None, W=None, dX=None, ws=None), OK),
    (dict(T=-1), SHAPE), (dict(V=0), SHAPE), (dict(r=128), SHAPE), (dict(lddx=56), SHAPE),
    (dict(V=100), UNSUP),  # a sketched head's V is a multiple of 8
    (dict(r=24), UNSUP), (dict(T=65537), UNSUP), (dict(lddx=(1 << 23) + 8), UNSUP),
    (dict(dX=None, r=0, XP=None, C=None), NULL), (dict(lse=None), NULL), (dict(grad=None), NULL), (dict(XP=None), NULL), (dict(C=None), NULL),
    (dict(dX=FAKE + 8), ALIGN), (dict(lddx=68), ALIGN), (dict(C=FAKE + 4), ALIGN), (dict(grad=FAKE + 1), ALIGN),
    (dict(ws=FAKE + 64), ALIGN), (dict(ws=None), WS), (dict(n=1000), WS),
])
def test_cross_entropy_backward(lib, kw, want):
    assert _call(lib.rgc_linear_cross_entropy_backward, BWD, **kw) == want


def test_cross_entropy_workspaces(lib):
    f, b = lib.rgc_linear_cross_entropy_forward_workspace_size, lib.rgc_linear_cross_entropy_backward_workspace_size
    assert f(0, 100, 64, 16) == b(0, 104, 64, 16) == 0
    assert f(16, 100, 60, 0) == 0 and b(16, 100, 64, 24) == 0  # unsupported
    # never the logits, nor all of D: far below 2 bytes a logit for a large vocabulary
    assert 0 < f(4096, 131072, 4096, 128) < 4096 * 131072 * 2 / 16
    assert 0 < b(4096, 131072, 4096, 128) < 4096 * 131072 * 2 / 2
    need = b(16, 104, 64, 16)
    assert _call(lib.rgc_linear_cross_entropy_backward, BWD, n=need - 1) == WS


NF = dict(kind=0, xt=0, wt=1, X=FAKE, ldx=100, w=FAKE, b=FAKE, eps=1e-5, Y=FAKE, ldy=100, mean=FAKE, rstd=FAKE, rows=4,
          n=100, s=None)
NB = dict(kind=0, xt=0, wt=1, dY=FAKE, lddy=100, X=FAKE, ldx=100, w=FAKE, mean=FAKE, rstd=FAKE, dX=FAKE, lddx=100, dw=FAKE,
          db=FAKE, rows=4, n=100, ws=FAKE, nb=1 << 30, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0, X=None, Y=None), OK),
    (dict(kind=2), UNSUP), (dict(xt=2), UNSUP), (dict(wt=-1), UNSUP), (dict(n=65537, ldx=65537, ldy=65537), UNSUP),
    (dict(rows=(1 << 31) + 1), UNSUP), (dict(ldx=(1 << 31) + 1), UNSUP),
    (dict(rows=-1), SHAPE), (dict(n=0), SHAPE), (dict(ldx=99), SHAPE), (dict(ldy=99), SHAPE),
    (dict(X=None), NULL), (dict(Y=None), NULL),
    (dict(X=FAKE + 1), ALIGN), (dict(xt=1, Y=FAKE + 2), ALIGN), (dict(w=FAKE + 2), ALIGN), (dict(b=FAKE + 2), ALIGN),
    (dict(mean=FAKE + 2), ALIGN), (dict(rstd=FAKE + 1), ALIGN),
    (dict(eps=-1e-9), VALUE), (dict(eps=float("nan")), VALUE), (dict(eps=float("inf")), VALUE), (dict(eps=1e300), VALUE),
])
def test_norm_forward(lib, kw, want):
    assert _call(lib.rgc_layer_norm_forward, NF, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(kind=5), UNSUP), (dict(n=65537), UNSUP), (dict(rows=-1), SHAPE), (dict(lddy=99), SHAPE), (dict(lddx=99), SHAPE),
    (dict(dw=None), NULL), (dict(dY=None), NULL), (dict(dX=None), NULL), (dict(rstd=None), NULL), (dict(mean=None), NULL),
    (dict(dw=FAKE + 2), ALIGN), (dict(db=FAKE + 2), ALIGN), (dict(ws=FAKE + 16), ALIGN), (dict(ws=None), WS),
    (dict(nb=100), WS),
])
def test_norm_backward(lib, kw, want):
    assert _call(lib.rgc_layer_norm_backward, NB, **kw) == want


def test_norm_workspace_covers_both_paths(lib):
    size = lib.rgc_layer_norm_backward_workspace_size
    assert size(0, 100) == size(10, 0) == size(10, 65537) == 0
    for rows in (1, 3, 100, 5000, 1 << 20):
        for n in (1, 8, 128, 1003, 4096, 16384, 16385, 65536):
            assert size(rows, n) % (8 * n) == 0 and 0 < size(rows, n) <= min(rows, 4096) * 8 * n


def _adam(lib, n=1, numels=(100,), **kw):
    arr = lambda p, m=n: (ctypes.c_void_p * max(m, 1))(*([p] * m)) if p != "none" else None  # noqa: E731
    d = dict(pt=0, gt=0, bits=8, P=FAKE, G=FAKE, M=FAKE, V=FAKE, Ms=FAKE, Vs=FAKE, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8,
             wd=0.0, step=1, scale=None)
    d.update(kw)
    return lib.rgc_adamw_batch(n, d["pt"], d["gt"], d["bits"], arr(d["P"]), arr(d["G"]), arr(d["M"]), arr(d["V"]),
                               arr(d["Ms"]), arr(d["Vs"]), (ctypes.c_int64 * max(n, 1))(*numels[:n]), d["lr"], d["b1"],
                               d["b2"], d["eps"], d["wd"], d["step"], d["scale"], 1, None)


def test_adamw(lib):
    inf, nan = float("inf"), float("nan")
    assert _adam(lib, n=0) == OK
    assert _adam(lib, numels=(0,), P=None, G=None) == OK  # nothing to do
    assert lib.rgc_adamw_batch(-1, 0, 0, 8, None, None, None, None, None, None, None, 1e-3, .9, .999, 1e-8, 0., 1, None, 0,
                               None) == SHAPE
    for kw in (dict(pt=2), dict(gt=7), dict(bits=16), dict(numels=((1 << 34) + 1,))):
        assert _adam(lib, **kw) == UNSUP, kw
    assert _adam(lib, numels=(-1,)) == SHAPE
    for kw in (dict(lr=nan), dict(lr=inf), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=nan), dict(eps=0.0),
               dict(eps=-1e-8), dict(eps=1e-60), dict(eps=1e-39), dict(eps=inf), dict(wd=nan), dict(step=0)):
        assert _adam(lib, **kw) == VALUE, kw
    for kw in (dict(P=None), dict(G=None), dict(M=None), dict(V=None), dict(Ms=None), dict(Vs=None), dict(P="none"),
               dict(Ms="none")):
        assert _adam(lib, **kw) == NULL, kw
    for kw in (dict(P=FAKE + 2), dict(G=FAKE + 8), dict(M=FAKE + 4), dict(V=FAKE + 1), dict(Ms=FAKE + 2), dict(scale=FAKE + 2)):
        assert _adam(lib, **kw) == ALIGN, kw


def test_the_binding_refuses_cpu_tensors_and_mismatched_lists():
    x = torch.zeros(16, 64, dtype=torch.bfloat16)
    y = torch.zeros(16, dtype=torch.int64)
    f = torch.zeros(16)
    for call in (lambda: rgc.rgc_linear_cross_entropy_forward(x, x, y),
                 lambda: rgc.rgc_linear_cross_entropy_backward(x, x, y, f, f),
                 lambda: rgc.rgc_layer_norm_forward(x),
                 lambda: rgc.rgc_layer_norm_backward(x, x, None, f, f),
                 lambda: rgc.rgc_adamw_batch([f], [f], [f], [f], 1e-3, 1),
                 lambda: rgc.rgc_adamw_batch([f], [], [f], [f], 1e-3, 1),
                 lambda: rgc.rgc_adamw_batch([f], [f], [f], [f], 1e-3, 1, M_scales=[f])):
        with pytest.raises(rgc.RgcError):
            call()
    assert rgc.rgc_adamw_batch([], [], [], [], 1e-3, 1) == []


def test_a_refused_step_is_not_counted():
    """A parameter's step count sets its bias corrections: it counts the updates made, not the calls refused."""
    p = torch.nn.Parameter(torch.ones(8))
    p.grad = torch.ones(8)
    opt = AdamW([p])
    for _ in range(2):
        with pytest.raises(rgc.RgcError):
            opt.step()  # a CPU tensor
    assert opt.state[0] is None or opt.state[0]["step"] == 0
