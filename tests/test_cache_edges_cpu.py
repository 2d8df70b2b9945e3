"""Refusals on the host of what the operators around the cache have at their borders."""

import ctypes

from test_serving_cpu import BUF, INVALID, MISALIGNED, OK, WORKSPACE, P, _cache, _L


def test_resize_with_copies_refusals():
    L = _L()
    h = L.lib()

    def call(want=BUF, origin=P(1 << 20), fresh=P(1 << 21), ws=BUF, less=0, **kw):
        f = dict(page_size=16, max_pages=8, n_seqs=4, n_pages=32, refs=4096, pages=4096, held=4096)
        f.update(kw)
        need = h.qwha_workspace_size(14, 4, 1, 32, 0, 0)
        return h.qwha_pages_resize_copies(ctypes.byref(L.QwhaPageTable(**f)), want, origin, fresh, ws, need - less, None)

    for kw in (dict(page_size=0), dict(max_pages=-1), dict(n_seqs=-1), dict(n_pages=-1), dict(refs=None), dict(held=None)):
        assert call(**kw) == INVALID, kw
    assert call(want=None) == INVALID and call(origin=None) == INVALID and call(fresh=None) == INVALID
    assert call(origin=P(6)) == MISALIGNED and call(fresh=P(6)) == MISALIGNED
    assert call(origin=P(1 << 20), fresh=P((1 << 20) + 12)) == INVALID  # the last of the one is the first of the other
    assert call(less=1) == WORKSPACE and call(ws=None) != OK
    assert call(n_seqs=0, want=None, origin=None, fresh=None) == OK
    assert h.qwha_pages_resize_copies(None, BUF, BUF, BUF, BUF, 1 << 20, None) == INVALID


def test_attention_upto_refusals():
    """A negative length is refused; all else as without one (the same checks, in the same order)."""
    L = _L()
    h, c = L.lib(), _cache(L)

    def call(longest, n=4, q=P(1 << 20), q_heads=4):
        k = ctypes.byref(c)
        return h.qwha_cache_attention_upto(k, k, 1, q, n, q_heads, 512, BUF, 2, BUF, BUF, 2, None, ctypes.c_float(0.1), longest, P(1 << 22), None,
                                           BUF, 1 << 30, None)

    assert call(-1) == INVALID and b"longest" in h.qwha_last_error()
    for longest in (0, 1, 2**63 - 1):
        assert call(longest, n=0) == OK and call(longest, n=-1) == INVALID and call(longest, q=None) == INVALID
        assert call(longest, q_heads=3) == INVALID and b"q_heads" in h.qwha_last_error()
