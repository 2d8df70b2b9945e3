"""Refusals of the serving entry points that tokens and outputs in one place need (on the host, no GPU needed)."""

import ctypes

import pytest

from test_serving_cpu import INVALID, P, _L, _qgemv, _wq


@pytest.mark.parametrize("dt,esz", [(1, 2), (0, 4)])
def test_outputs_over_the_tokens_are_refused(dt, esz):
    """The products store outputs while tokens are still read: neither the same buffer nor a part of it."""
    L = _L()
    h = L.lib()
    T, d_in, d_out, n = 3, 256, 64, 1 << 20
    x, ws = 1 << 20, P(1 << 28)
    x_end = x + T * d_in * esz
    z_apart = P(1 << 24)
    a = L.QwhaAdapter(d_in, d_out, 256, 0, 10, 4096, 4096, 4096)

    def decode(y, z):
        return h.qwha_adapter_decode(ctypes.byref(a), None, dt, P(x), T, ctypes.c_float(1.0), z, P(y), ws, n, None)

    for y in (x, x_end - 16, x - T * d_out * esz + 16):
        assert _qgemv(L, _wq(L), d_out=d_out, d_in=d_in, dt=dt, x=P(x), T=T, y=P(y), ws=ws, nbytes=n) == INVALID
        assert h.qwha_last_error() == b"X and Y overlap"
        assert decode(y, None) == INVALID
        assert decode(y, z_apart) == INVALID
    assert decode(x_end, P(x)) == INVALID and h.qwha_last_error() == b"X and Z_out overlap"
    assert decode(x_end, P(x_end + 16)) == INVALID and h.qwha_last_error() == b"Y and Z_out overlap"
