"""Refusals on the host of what the operators around the cache have at their borders."""

import ctypes

from test_serving_cpu import BUF, INVALID, MISALIGNED, OK, WORKSPACE, P, _L


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
