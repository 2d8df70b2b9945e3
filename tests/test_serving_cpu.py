"""Refusals of the serving entry points: all on the host, before any CUDA call (no GPU needed)."""

import ctypes

import numpy as np
import pytest

from _serving import butterflies, quantize, values, pack
from test_abi import _ensure_built
from workloads import rng_for

P = ctypes.c_void_p
OK, INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
BUF = P(4096)


def _L():
    _ensure_built()
    import walsh_hadamard_sparse_b200._lib as L

    return L


def _wq(L, bits=4, group=64, **kw):
    f = dict(qweight=4096, scales=4096, zeros=4096)
    f.update(kw)
    return L.QwhaQweight(bits, group, f["qweight"], f["scales"], f["zeros"])


def _qgemv(L, wq, d_out=64, d_in=256, dt=1, x=BUF, T=1, y=BUF, ws=None, nbytes=0):
    return L.lib().qwha_qgemv(ctypes.byref(wq) if wq is not None else None, d_out, d_in, dt, x, T, y, ws, nbytes, None)


def test_qgemv_refusals():
    L = _L()
    assert _qgemv(L, None) == INVALID
    assert _qgemv(L, _wq(L, bits=5)) == INVALID
    assert _qgemv(L, _wq(L, group=12)) == INVALID  # not a multiple of 8
    assert _qgemv(L, _wq(L, group=0)) == INVALID
    assert _qgemv(L, _wq(L), d_in=96) == INVALID  # 64 does not divide 96
    assert _qgemv(L, _wq(L), d_out=0) == INVALID
    assert _qgemv(L, _wq(L), dt=2) == INVALID
    assert _qgemv(L, _wq(L), T=-1) == INVALID
    assert _qgemv(L, _wq(L), T=65) == UNSUPPORTED
    assert b"qwha_adapter_fwd" in L.lib().qwha_last_error()
    assert _qgemv(L, _wq(L), x=None) == INVALID
    assert _qgemv(L, _wq(L), x=P(8)) == MISALIGNED
    assert _qgemv(L, _wq(L), y=P(4100)) == MISALIGNED
    assert _qgemv(L, _wq(L, scales=4)) == MISALIGNED
    assert _qgemv(L, _wq(L, zeros=None)) == INVALID
    assert _qgemv(L, _wq(L), T=0, x=None, y=None) == OK  # nothing to do
    for dt, base, pieces in ((1, 1, 1), (0, 2, 3)):  # two bytes a value and piece, and the sums
        need = L.lib().qwha_workspace_size(12, 64, 256, 0, 3, base)
        assert need > 3 * 256 * 2 * pieces
        assert _qgemv(L, _wq(L), dt=dt, T=3) == WORKSPACE
        assert _qgemv(L, _wq(L), dt=dt, T=3, ws=BUF, nbytes=need - 1) == WORKSPACE
        assert _qgemv(L, _wq(L), dt=dt, T=3, ws=P(4096 + 16), nbytes=need) == MISALIGNED


def test_decode_refusals():
    L = _L()
    h = L.lib()

    def call(T=1, ws=BUF, nbytes=1 << 20, z=None, wq=None, dt=1, alpha=1.0, **kw):
        f = dict(d_in=256, d_out=64, had_block=256, algo=0, p=10, row_ptr=4096, col_idx=4096, coef=4096)
        f.update(kw)
        a = L.QwhaAdapter(**f)
        return h.qwha_adapter_decode(ctypes.byref(a), ctypes.byref(wq) if wq is not None else None, dt, BUF, T,
                                     ctypes.c_float(alpha), z, BUF, ws, nbytes, None)

    assert call(had_block=48) == INVALID
    assert call(d_out=60) == INVALID  # not a multiple of 8
    assert call(p=-1) == INVALID
    assert call(T=65) == UNSUPPORTED
    assert call(T=-1) == INVALID
    assert call(z_given=1) == UNSUPPORTED
    assert call(dt=3) == INVALID
    assert call(wq=_wq(L, bits=8)) == INVALID
    assert call(z=P(8)) == MISALIGNED
    assert call(row_ptr=None) == INVALID
    need = h.qwha_workspace_size(10, 64, 256, 10, 3, 0)
    assert need >= 4 * 256 * 4  # tokens padded to a power of two
    assert call(T=3, nbytes=need - 1) == WORKSPACE
    assert call(T=3, ws=None, nbytes=0) == WORKSPACE
    assert call(T=3, ws=P(4096 + 16), nbytes=need) == MISALIGNED
    assert call(T=0) == OK
    assert h.qwha_workspace_size(10, 64, 256, 0, 3, 0) == 0  # no entries: no transform to hold
    for base in (1, 2):  # with a base weight, its operands too
        assert h.qwha_workspace_size(10, 64, 256, 10, 3, base) == need + h.qwha_workspace_size(12, 64, 256, 0, 3, base)


def _cache(L, **kw):
    f = dict(bits=4, group=64, had_block=64, heads=2, head_dim=128, page_size=16, n_pages=4, codes=4096, scales=4096,
             zeros=4096)
    f.update(kw)
    return L.QwhaCache(**f)


@pytest.mark.parametrize("kw,want", [
    (dict(bits=5), INVALID), (dict(bits=1), INVALID), (dict(heads=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(head_dim=100), INVALID), (dict(head_dim=264, group=8, had_block=0), UNSUPPORTED), (dict(group=48), INVALID),
    (dict(group=4), INVALID), (dict(group=0), INVALID), (dict(had_block=3), INVALID), (dict(had_block=256), INVALID),
    (dict(had_block=1), INVALID), (dict(had_block=-2), INVALID), (dict(page_size=0), INVALID),
    (dict(n_pages=-1), INVALID), (dict(n_pages=1 << 31), INVALID), (dict(codes=None), INVALID),
    (dict(scales=4104), MISALIGNED)])
def test_cache_refusals(kw, want):
    L = _L()
    h = L.lib()
    c = (L.QwhaCache * 2)(_cache(L), _cache(L, **kw))  # the second of a pair is checked too
    rows = (P * 2)(4096, 4096)
    assert h.qwha_cache_write(c, 2, 1, rows, BUF, 3, None) == want
    assert h.qwha_cache_read(c, 2, 1, BUF, 2, BUF, None, 2, rows, 3, None) == want
    assert h.qwha_validate_slots(ctypes.byref(c[1]), BUF, 3, BUF, 1 << 20, None) == want


def test_cache_call_refusals():
    L = _L()
    h = L.lib()
    c = (L.QwhaCache * 1)(_cache(L))
    rows = (P * 1)(4096)
    assert h.qwha_cache_write(c, 0, 1, rows, BUF, 3, None) == INVALID
    assert h.qwha_cache_write(c, 3, 1, rows, BUF, 3, None) == INVALID
    assert h.qwha_cache_write(c, 1, 2, rows, BUF, 3, None) == INVALID
    assert h.qwha_cache_write(None, 1, 1, rows, BUF, 3, None) == INVALID
    assert h.qwha_cache_write(c, 1, 1, rows, BUF, -1, None) == INVALID
    assert h.qwha_cache_write(c, 1, 1, rows, None, 3, None) == INVALID
    assert h.qwha_cache_write(c, 1, 1, (P * 1)(4104), BUF, 3, None) == MISALIGNED
    assert h.qwha_cache_write(c, 1, 1, rows, None, 0, None) == OK
    assert h.qwha_cache_read(c, 1, 1, BUF, -1, BUF, None, 2, rows, 3, None) == INVALID
    assert h.qwha_cache_read(c, 1, 1, BUF, 2, None, None, 2, rows, 3, None) == INVALID
    assert h.qwha_cache_read(c, 1, 1, None, 2, BUF, None, 2, rows, 3, None) == INVALID
    assert h.qwha_cache_read(c, 1, 1, BUF, 2, BUF, P(4), 2, rows, 3, None) == MISALIGNED
    assert h.qwha_cache_read(c, 1, 1, BUF, 2, BUF, None, 0, rows, 3, None) == OK
    assert h.qwha_cache_read(c, 1, 1, BUF, 2, BUF, None, 2, rows, 0, None) == OK
    need = h.qwha_workspace_size(11, 1, 1, 64, 0, 0)
    assert need >= 8 + 64 // 8
    assert h.qwha_validate_slots(ctypes.byref(c[0]), BUF, 3, BUF, need - 1, None) == WORKSPACE


def test_the_quantizer_statement():
    """The plain statement the GPU tests compare with: within a step of the value for every width (half a step and
    2^-12 of one, or at the clamped end one step), zero exact, a constant row exact at its ends."""
    g = rng_for(90, "quantizer")
    for bits in (2, 3, 4, 8):
        rows = g.standard_normal((50, 64)).astype(np.float32) * 3
        rows[0] = 0.0
        rows[1] = 2.5
        q, s, z = quantize(rows, bits, 32, 0, "f32")
        back = values(pack(q, bits), s, z, bits, 32)
        step = np.repeat(s.astype(np.float64), 32, axis=1)
        assert np.all(np.abs(back - rows) <= step * 1.001)
        assert np.mean(np.abs(back - rows) <= step * 0.501) > 0.95
        assert np.all(back[0] == 0) and np.allclose(back[1], 2.5, rtol=1e-6)
    x = g.standard_normal((3, 64))
    assert np.allclose(butterflies(butterflies(x, 16), 16), x, atol=1e-12)
