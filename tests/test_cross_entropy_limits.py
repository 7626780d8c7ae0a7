"""The joint limit of tokens and vocabulary of the head's loss (CPU only: every
call is refused on the host)."""
import pytest

from rank_randomized_gradient_amd import rgc

UNSUP, WS = 3, 5
FAKE = 0x10000  # an aligned address that is never dereferenced


def _forward(lib, T, V, ws_bytes):
    return lib.rgc_linear_cross_entropy_forward(FAKE, 64, FAKE, 64, None, FAKE, FAKE, FAKE, None, T, V, 64, 0, FAKE, ws_bytes,
                                                None)


@pytest.mark.parametrize("T,V", [(65536, 1 << 22), (65536, 1 << 24), (65535, 1 << 24), (20000, 1 << 24)])
def test_too_many_tiles_are_refused_before_a_workspace_is_asked_for(T, V):
    lib = rgc.load_library()
    assert lib.rgc_linear_cross_entropy_forward_workspace_size(T, V, 64, 0) == 0
    assert _forward(lib, T, V, 0) == _forward(lib, T, V, 1 << 62) == UNSUP


@pytest.mark.parametrize("T,V", [(65536, (1 << 22) - 65536), (16000, 1 << 24), (64, 1 << 24), (128, 1 << 24)])
def test_the_largest_that_fit(T, V):
    lib = rgc.load_library()
    assert lib.rgc_linear_cross_entropy_forward_workspace_size(T, V, 64, 0) > 0
    assert _forward(lib, T, V, 0) == WS
