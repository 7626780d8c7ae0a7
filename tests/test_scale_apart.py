"""A factor on the device that lies in a tensor which the call changes would be read by one
workgroup after another wrote it: the binding refuses it. On the CPU, with the library's calls
recorded in the place of launches; on the GPU, a factor beside the tensors in one buffer."""
import contextlib
import types

import pytest
import torch

from rank_randomized_gradient_amd import rgc

F32, BF = torch.float32, torch.bfloat16


class Recorder:
    """A library whose calls succeed and do nothing."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def lib(monkeypatch):
    """The binding on host tensors: it checks what it is given and calls a Recorder."""
    made = Recorder()
    monkeypatch.setattr(rgc, "load_library", lambda: made)
    monkeypatch.setattr(rgc, "_need_gpu", lambda *ts: types.SimpleNamespace(index=-1))
    monkeypatch.setattr(rgc, "_on", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(rgc, "_stream", lambda dev: None)
    return made


def test_scale_batch(lib):
    flat = torch.ones(64)
    half = flat[40:48].view(BF)
    for Gs, scale in (([flat], flat[:1]), ([flat], flat[63:]), ([flat[:8], flat[8:16]], flat[15:16]),
                      ([flat[20:], flat[:4]], flat[3]), ([half], flat[40:41]), ([half[1:5]], flat[42:43])):
        with pytest.raises(rgc.RgcError):
            rgc.rgc_scale_batch(Gs, scale)
    assert lib.calls == []
    for Gs, scale in (([flat[1:]], flat[:1]), ([flat[:8], flat[9:]], flat[8:9]), ([half[2:]], flat[40:41]), ([half[:4]], flat[42:43]),
                      ([flat[5:5], flat[:5]], flat[5])):
        assert rgc.rgc_scale_batch(Gs, scale) is Gs
    assert lib.calls == ["rgc_scale_batch"] * 5


def test_adamw(lib):
    """Not in a parameter, a moment or a moment's scale; in a gradient, which is only read, it may lie."""
    z = torch.zeros
    for gt in (BF, F32):
        for eight in (False, True):
            state = torch.float8_e4m3fn if eight else F32
            P, G, M, V = z(256), z(256, dtype=gt), z(256, dtype=state), z(256, dtype=state)
            scales = dict(M_scales=[z(2)], V_scales=[z(2)]) if eight else {}
            step = lambda s: rgc.rgc_adamw_batch([P], [G], [M], [V], 1e-3, 1, grad_scale=s, **scales)  # noqa: E731, B023
            written = [P, M, V] + [t for ts in scales.values() for t in ts]
            for t in written:
                words = t.view(F32) if t.dtype != F32 else t
                for at in (0, len(words) - 1):
                    with pytest.raises(rgc.RgcError):
                        step(words[at:at + 1])
            assert lib.calls == []
            step(z(1))
            step(z(()))
            step(G.view(F32)[-1])
            assert lib.calls == ["rgc_adamw_batch_with"] * 3
            lib.calls.clear()


@pytest.mark.gpu
def test_a_factor_beside_the_tensors():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    flat = torch.ones(100001, device="cuda")
    flat[777] = 0.25
    rgc.rgc_scale_batch([flat[:777], flat[778:]], flat[777:778])
    assert bool((flat == 0.25).all())
    with pytest.raises(rgc.RgcError):
        rgc.rgc_scale_batch([flat], flat[777])
