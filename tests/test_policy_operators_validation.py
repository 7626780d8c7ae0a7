"""Refusals of the log probabilities, the clipping and the residual norm (CPU
only: every call here is rejected on the host, or has nothing to do, before any
launch)."""
import ctypes

import pytest
import torch

from rank_randomized_gradient_amd import AdamW, clip_grad_norm, log_prob, rgc

OK, NULL, SHAPE, UNSUP, ALIGN, WS, VALUE = 0, 1, 2, 3, 4, 5, 7
FAKE = 0x10000  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    return rgc.load_library()


def _call(fn, defaults, **kw):
    assert set(kw) <= set(defaults), set(kw) - set(defaults)
    return fn(*{**defaults, **kw}.values())


HF = dict(X=FAKE, ldx=64, W=FAKE, ldw=64, P=FAKE, tokens=FAKE, logp=FAKE, entropy=FAKE, lse=FAKE, XP=FAKE, T=16, V=100, k=64,
          r=16, ws=FAKE, n=1 << 30, s=None)
HB = dict(X=FAKE, ldx=64, W=FAKE, ldw=64, tokens=FAKE, lse=FAKE, entropy=FAKE, gl=FAKE, ge=FAKE, XP=FAKE, C=FAKE, dX=FAKE,
          lddx=64, T=16, V=104, k=64, r=16, ws=FAKE, n=1 << 40, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, X=None, W=None, tokens=None, logp=None, entropy=None, ws=None), OK),
    (dict(T=-1), SHAPE), (dict(V=0), SHAPE), (dict(r=128), SHAPE), (dict(ldx=56), SHAPE), (dict(ldw=56), SHAPE),
    (dict(r=24), UNSUP), (dict(k=60, ldx=64, ldw=64), UNSUP), (dict(T=65537), UNSUP), (dict(V=(1 << 24) + 1), UNSUP),
    (dict(T=65536, V=1 << 24), UNSUP),  # too many tiles
    (dict(X=None), NULL), (dict(tokens=None), NULL), (dict(logp=None), NULL), (dict(entropy=None), NULL),
    (dict(lse=None), NULL), (dict(P=None), NULL), (dict(XP=None), NULL),
    (dict(X=FAKE + 2), ALIGN), (dict(tokens=FAKE + 4), ALIGN), (dict(logp=FAKE + 2), ALIGN), (dict(entropy=FAKE + 1), ALIGN),
    (dict(ws=FAKE + 128), ALIGN), (dict(ws=None), WS), (dict(n=100), WS),
])
def test_linear_log_prob_forward(lib, kw, want):
    assert _call(lib.rgc_linear_log_prob_forward, HF, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, X=None, W=None, dX=None, ws=None), OK),
    (dict(T=-1), SHAPE), (dict(V=0), SHAPE), (dict(r=128), SHAPE), (dict(lddx=56), SHAPE),
    (dict(V=100), UNSUP), (dict(r=24), UNSUP), (dict(T=65537), UNSUP),
    (dict(gl=None, ge=None), NULL), (dict(entropy=None), NULL), (dict(lse=None), NULL), (dict(XP=None), NULL),
    (dict(C=None), NULL), (dict(dX=None, r=0, XP=None, C=None), NULL),
    (dict(gl=FAKE + 2), ALIGN), (dict(ge=FAKE + 1), ALIGN), (dict(entropy=FAKE + 2), ALIGN), (dict(dX=FAKE + 8), ALIGN),
    (dict(gl=None, ws=None), WS), (dict(ge=None, entropy=None, ws=None), WS), (dict(n=1000), WS),
])
def test_linear_log_prob_backward(lib, kw, want):
    assert _call(lib.rgc_linear_log_prob_backward, HB, **kw) == want


def test_linear_log_prob_workspaces(lib):
    f, b = lib.rgc_linear_log_prob_forward_workspace_size, lib.rgc_linear_log_prob_backward_workspace_size
    assert f(0, 100, 64, 16) == b(0, 104, 64, 16) == f(65536, 1 << 24, 64, 0) == 0
    assert 0 < f(4096, 131072, 4096, 128) < 4096 * 131072 * 2 / 16
    assert b(4096, 131072, 4096, 128) == lib.rgc_linear_cross_entropy_backward_workspace_size(4096, 131072, 4096, 128)
    need = f(16, 100, 64, 16)
    assert need > lib.rgc_linear_cross_entropy_forward_workspace_size(16, 100, 64, 16)
    assert _call(lib.rgc_linear_log_prob_forward, HF, n=need - 1) == WS


LF = dict(zt=0, Z=FAKE, ldz=1000, tokens=FAKE, logp=FAKE, entropy=FAKE, lse=FAKE, top=5, top_logp=FAKE, top_ids=FAKE, rows=4,
          V=1000, ws=FAKE, n=1 << 30, s=None)
LB = dict(zt=0, Z=FAKE, ldz=1000, tokens=FAKE, lse=FAKE, entropy=FAKE, gl=FAKE, ge=FAKE, dZ=FAKE, lddz=1000, rows=4, V=1000,
          s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0, Z=None, entropy=None, ws=None), OK),
    (dict(zt=2), UNSUP), (dict(V=(1 << 24) + 1, ldz=1 << 25), UNSUP), (dict(rows=(1 << 31) + 1), UNSUP), (dict(top=65), UNSUP),
    (dict(ldz=(1 << 31) + 1), UNSUP),
    (dict(rows=-1), SHAPE), (dict(V=0), SHAPE), (dict(ldz=999), SHAPE), (dict(top=-1), SHAPE), (dict(V=4, ldz=4), SHAPE),
    (dict(Z=None), NULL), (dict(logp=None), NULL), (dict(entropy=None), NULL), (dict(lse=None), NULL),
    (dict(top_logp=None), NULL), (dict(top_ids=None), NULL),
    (dict(Z=FAKE + 1), ALIGN), (dict(zt=1, Z=FAKE + 2), ALIGN), (dict(tokens=FAKE + 4), ALIGN), (dict(lse=FAKE + 2), ALIGN),
    (dict(top_ids=FAKE + 4), ALIGN), (dict(top_logp=FAKE + 2), ALIGN),
    (dict(V=100000, ldz=100000, ws=None), WS), (dict(V=100000, ldz=100000, n=64), WS),
    (dict(V=100000, ldz=100000, ws=FAKE + 64), ALIGN),
])
def test_log_prob_forward(lib, kw, want):
    assert _call(lib.rgc_log_prob_forward, LF, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0, Z=None, dZ=None), OK),
    (dict(zt=7), UNSUP), (dict(V=(1 << 24) + 1, ldz=1 << 25, lddz=1 << 25), UNSUP), (dict(lddz=(1 << 31) + 1), UNSUP),
    (dict(rows=-1), SHAPE), (dict(V=-3), SHAPE), (dict(ldz=999), SHAPE), (dict(lddz=999), SHAPE),
    (dict(Z=None), NULL), (dict(dZ=None), NULL), (dict(tokens=None), NULL), (dict(lse=None), NULL), (dict(gl=None, ge=None), NULL),
    (dict(entropy=None), NULL),
    (dict(Z=FAKE + 1), ALIGN), (dict(dZ=FAKE + 1), ALIGN), (dict(gl=FAKE + 2), ALIGN), (dict(ge=FAKE + 2), ALIGN),
    (dict(entropy=FAKE + 2), ALIGN), (dict(tokens=FAKE + 4), ALIGN),
])
def test_log_prob_backward(lib, kw, want):
    assert _call(lib.rgc_log_prob_backward, LB, **kw) == want


def test_log_prob_workspaces(lib):
    size = lib.rgc_log_prob_forward_workspace_size
    assert size(0, 1000, 5) == size(4, 0, 5) == size(4, 1000, 65) == size(4, 3, 4) == 0
    assert size(1 << 20, 131072, 20) == 0  # a workgroup to a row
    for rows in (1, 3, 100, 2047):
        for V in (1, 4096, 4097, 131072, 1 << 24):
            assert size(rows, V, 1) <= 64 * rows * 24 + 256


ARR = dict(n=1, gts=(0,), Gs=(FAKE,), numels=(100,))


def _arrays(d):
    n = max(len(d["numels"] or ()), 1)
    fill = lambda t, v: None if v is None else (t * n)(*v)  # noqa: E731
    return d["n"], fill(ctypes.c_int, d["gts"]), fill(ctypes.c_void_p, d["Gs"]), fill(ctypes.c_int64, d["numels"])


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), SHAPE), (dict(numels=(-1,)), SHAPE), (dict(n=(1 << 24) + 1), UNSUP), (dict(gts=(2,)), UNSUP),
    (dict(numels=((1 << 34) + 1,)), UNSUP), (dict(Gs=(None,)), NULL), (dict(Gs=None), NULL), (dict(gts=None), NULL),
    (dict(numels=None), NULL), (dict(Gs=(FAKE + 1,)), ALIGN), (dict(gts=(1,), Gs=(FAKE + 2,)), ALIGN),
    (dict(max_norm=-1.0), VALUE), (dict(max_norm=float("nan")), VALUE), (dict(norm=None), NULL), (dict(norm=FAKE + 2), ALIGN),
    (dict(out=None), NULL), (dict(out=FAKE + 2), ALIGN), (dict(scale=FAKE + 2), ALIGN), (dict(ws=None), WS), (dict(nb=7), WS), (dict(ws=FAKE + 64), ALIGN),
])
def test_grad_norm(lib, kw, want):
    d = {**ARR, "max_norm": 1.0, "scale": None, "norm": FAKE, "out": FAKE, "ws": FAKE, "nb": 1 << 20, **kw}
    assert lib.rgc_grad_norm_batch(*_arrays(d), d["max_norm"], d["scale"], d["norm"], d["out"], d["ws"], d["nb"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(n=0, gts=None, Gs=None, numels=None, scale=None), OK), (dict(n=1, numels=(0,), Gs=(None,)), OK),
    (dict(n=-1), SHAPE), (dict(gts=(2,)), UNSUP), (dict(Gs=(None,)), NULL), (dict(scale=None), NULL),
    (dict(scale=FAKE + 1), ALIGN), (dict(Gs=(FAKE + 1,)), ALIGN),
])
def test_scale(lib, kw, want):
    d = {**ARR, "scale": FAKE, **kw}
    assert lib.rgc_scale_batch(*_arrays(d), d["scale"], None) == want


def test_grad_norm_workspace(lib):
    size = lambda *n: lib.rgc_grad_norm_batch_workspace_size(len(n), (ctypes.c_int64 * max(len(n), 1))(*n))  # noqa: E731
    assert size() == size(0) == size(-1) == size((1 << 34) + 1) == 0
    assert size(1) == size(8192) == 8 and size(8193) == size(1, 0, 1) == 16
    assert size(1 << 34) <= 8 * 8192  # few partial sums, whatever the sizes


AF = dict(kind=0, xt=0, wt=1, X=FAKE, ldx=100, R=FAKE, ldr=100, w=FAKE, b=FAKE, eps=1e-5, S=FAKE, lds=100, Y=FAKE, ldy=100,
          mean=FAKE, rstd=FAKE, rows=4, n=100, s=None)
AB = dict(kind=0, xt=0, wt=1, dY=FAKE, lddy=100, dS=FAKE, ldds=100, S=FAKE, lds=100, w=FAKE, mean=FAKE, rstd=FAKE, dX=FAKE,
          lddx=100, dw=FAKE, db=FAKE, rows=4, n=100, ws=FAKE, nb=1 << 30, s=None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0, X=None, R=None, S=None, Y=None), OK),
    (dict(kind=2), UNSUP), (dict(xt=2), UNSUP), (dict(n=65537, ldx=65537, ldr=65537, lds=65537, ldy=65537), UNSUP),
    (dict(ldr=(1 << 31) + 1), UNSUP), (dict(rows=-1), SHAPE), (dict(ldr=99), SHAPE), (dict(lds=99), SHAPE), (dict(ldy=99), SHAPE),
    (dict(X=None), NULL), (dict(R=None), NULL), (dict(S=None), NULL), (dict(Y=None), NULL),
    (dict(R=FAKE + 1), ALIGN), (dict(xt=1, S=FAKE + 2), ALIGN), (dict(w=FAKE + 2), ALIGN), (dict(eps=-1.0), VALUE),
])
def test_add_norm_forward(lib, kw, want):
    assert _call(lib.rgc_add_norm_forward, AF, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(kind=5), UNSUP), (dict(rows=-1), SHAPE), (dict(ldds=99), SHAPE), (dict(lds=99), SHAPE), (dict(dw=None), NULL),
    (dict(dY=None), NULL), (dict(S=None), NULL), (dict(dX=None), NULL), (dict(mean=None), NULL), (dict(rstd=None), NULL),
    (dict(dS=FAKE + 1), ALIGN), (dict(dS=None, ldds=0, ws=None), WS), (dict(nb=100), WS), (dict(ws=FAKE + 16), ALIGN),
])
def test_add_norm_backward(lib, kw, want):
    assert _call(lib.rgc_add_norm_backward, AB, **kw) == want


def test_the_binding_refuses_cpu_tensors():
    x = torch.zeros(16, 64, dtype=torch.bfloat16)
    y, f = torch.zeros(16, dtype=torch.int64), torch.zeros(16)
    p = torch.nn.Parameter(torch.ones(8))
    p.grad = torch.ones(8)
    for call in (lambda: rgc.rgc_linear_log_prob_forward(x, x, y), lambda: rgc.rgc_linear_log_prob_backward(x, x, y, f, f, f, f),
                 lambda: rgc.rgc_log_prob_forward(x, y), lambda: rgc.rgc_log_prob_backward(x, y, f, f, f), lambda: log_prob(x, y),
                 lambda: log_prob(x, y[:3]), lambda: log_prob(x, y.int()), lambda: rgc.rgc_grad_norm_batch([f]),
                 lambda: rgc.rgc_scale_batch([f], f[:1]), lambda: clip_grad_norm([p], 1.0), lambda: AdamW([p]).step(max_norm=1.0),
                 lambda: rgc.rgc_add_norm_forward(x, x), lambda: rgc.rgc_add_norm_backward(x, x, x, None, f, f)):
        with pytest.raises(rgc.RgcError):
            call()
    assert float(clip_grad_norm([torch.nn.Parameter(torch.ones(3))], 1.0)) == 0
    assert AdamW([torch.nn.Parameter(torch.ones(3))]).step(max_norm=1.0) is None  # no gradients, no norm


def test_lists_of_gradients():
    """The compiled module's addresses, sizes, types and bytes; lists that are none."""
    pack = rgc._lists().pack_gradients
    a, b = torch.zeros(5), torch.zeros(2, 3, dtype=torch.bfloat16)
    pointers, sizes, types, lengths, device = pack((a, b))
    read = lambda x, t: list((t * 2).from_buffer_copy(x))  # noqa: E731
    assert read(pointers, ctypes.c_uint64) == [a.data_ptr(), b.data_ptr()] and read(sizes, ctypes.c_int64) == [5, 6]
    assert read(types, ctypes.c_int32) == [1, 0] and read(lengths, ctypes.c_int64) == [20, 12] and device == -1
    for bad in ([], [a, None], [a, 3], [a.half()], [a.double()], [a[::2]], [a.to_sparse()], [b.t()]):
        assert pack(bad) is None
    with pytest.raises(TypeError):
        pack(3)


def test_fresh_tensors():
    fresh = rgc._lists().fresh
    x = torch.zeros(3)
    a, none, b, c = fresh(x, torch.bfloat16, (2, 5), torch.int64, None, torch.uint8, (0,), torch.float32, ())
    assert a.dtype == torch.bfloat16 and a.shape == (2, 5) and none is None and b.shape == (0,) and c.dim() == 0
    assert a.is_contiguous() and a.device == x.device and fresh(x) == ()
    for bad in ((), (x, torch.float32), (3, torch.float32, (1,)), (x, 5, (1,)), (x, torch.float32, [1]),
                (x, torch.float32, (1.5,)), (x, torch.float32, (1, 1, 1, 1, 1))):
        with pytest.raises(TypeError):
            fresh(*bad)
    with pytest.raises(RuntimeError):
        fresh(x, torch.float32, (-1,))
