"""Refusals of the AdamW step's forms (CPU only: rejected on the host, or
nothing to do, before any launch)."""
import ctypes

import pytest
import torch

from rank_randomized_gradient_amd import rgc

OK, UNSUP, VALUE = 0, 3, 7


@pytest.fixture(scope="module")
def lib():
    return rgc.load_library()


def _with(lib, flags=0, bits=8, beta1=0.9, **kw):
    a = dict(lr=1e-3, beta2=0.999, eps=1e-8, wd=0.0, step=1)
    a.update(kw)
    none = (ctypes.c_void_p * 1)(None)
    return lib.rgc_adamw_batch_with(flags, 1, 0, 0, bits, none, none, none, none, none, none, (ctypes.c_int64 * 1)(0),
                                    a["lr"], beta1, a["beta2"], a["eps"], a["wd"], a["step"], None, 1, None)


def test_rounding_m_to_nearest_ends_at_a_beta1_that_decays(lib):
    assert _with(lib, beta1=0.9) == OK and _with(lib, beta1=0.0) == OK
    assert _with(lib, beta1=0.9001) == _with(lib, beta1=0.95) == _with(lib, beta1=0.99) == VALUE
    stochastic = rgc.RGC_ADAMW_STOCHASTIC_M
    assert _with(lib, flags=stochastic, beta1=0.99) == OK and _with(lib, bits=32, beta1=0.99) == OK
    assert _with(lib, flags=stochastic, beta1=1.0) == VALUE


def test_flags(lib):
    assert _with(lib, flags=1 << 20) == UNSUP
    with pytest.raises(rgc.RgcError):
        rgc.rgc_adamw_batch([], [], [], [], 1e-3, 1, m_rounding="down")


def test_scalars_that_would_make_infinities_of_finite_inputs(lib):
    assert _with(lib, bits=32, lr=1e20, wd=1e20) == VALUE  # lr wd
    assert _with(lib, bits=32, lr=1e29, beta1=0.999999) == VALUE  # lr / (1 - beta1)
    assert _with(lib, bits=32, lr=1e29, beta1=0.999999, step=10 ** 9) == OK
    # a beta that fp32 holds as 1 would never forget
    assert _with(lib, bits=32, beta1=1 - 1e-9) == _with(lib, bits=32, beta2=1 - 1e-9) == VALUE
    assert _with(lib, bits=32, beta1=1 - 2.0 ** -24, beta2=1 - 2.0 ** -24) == OK


def test_check_only(lib):
    """The refusals of the call, and nothing launched: addresses that are never read."""
    fake = (ctypes.c_void_p * 1)(0x10000)
    n = (ctypes.c_int64 * 1)(100)

    def call(p=fake, lr=1e-3):
        return lib.rgc_adamw_batch_with(rgc.RGC_ADAMW_CHECK_ONLY, 1, 0, 0, 32, p, fake, fake, fake, None, None, n, lr, 0.9,
                                        0.999, 1e-8, 0.0, 1, None, 1, None)

    assert call() == OK and call((ctypes.c_void_p * 1)(0x10008)) == 4 and call((ctypes.c_void_p * 1)(None)) == 1
    assert call(lr=float("nan")) == VALUE
