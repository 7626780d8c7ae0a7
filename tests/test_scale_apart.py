"""A factor on the device that lies in a tensor which the call changes would be read by one
workgroup after another wrote it: the binding refuses it. On the CPU, with the library's calls
recorded in the place of launches; on the GPU, a factor beside the tensors in one buffer."""
import contextlib

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
    monkeypatch.setattr(rgc, "_need_gpu", lambda *ts: torch.device("cpu"))
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
