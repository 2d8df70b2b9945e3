"""Refusals of the operators around the cache, all on the host before any CUDA call, and their plain statements."""

import ctypes

import numpy as np
import pytest

from _cache_ops import Table, rotary
from test_serving_cpu import BUF, INVALID, MISALIGNED, OK, UNSUPPORTED, WORKSPACE, P, _cache, _L

I64x2, I32x2 = ctypes.c_int64 * 2, ctypes.c_int32 * 2


def test_rotary_refusals():
    h = _L().lib()

    def call(dt=1, n_x=2, x=(1 << 20, 1 << 21), xs=(256, 256), y=(1 << 22, 1 << 23), ys=(256, 256), heads=(4, 2), D=64,
             n=8, pos=BUF, freq=BUF, rot=64, layout=0, factor=1.0):
        return h.qwha_rotary(dt, n_x, (P * 2)(*x), I64x2(*xs), (P * 2)(*y), I64x2(*ys), I32x2(*heads), D, n, pos, freq, rot,
                             layout, ctypes.c_float(factor), 0, None)

    assert call(dt=2) == INVALID and call(n_x=0) == INVALID and call(n_x=3) == INVALID
    assert call(D=60) == INVALID and call(D=0) == INVALID and call(D=264) == UNSUPPORTED
    assert call(rot=63) == INVALID and call(rot=66) == INVALID and call(rot=-2) == INVALID
    assert call(layout=2) == INVALID and call(n=-1) == INVALID and call(factor=float("inf")) == INVALID
    assert call(heads=(0, 2)) == INVALID
    assert call(xs=(248, 256)) == INVALID  # tokens overlap
    assert call(xs=(260, 256)) == MISALIGNED
    assert call(x=(None, 1 << 21)) == INVALID and call(x=((1 << 20) + 8, 1 << 21)) == MISALIGNED
    assert call(pos=None) == INVALID and call(freq=None) == INVALID and call(freq=P(4)) == MISALIGNED and call(pos=P(4)) == MISALIGNED
    # overlaps: shifted, the other's input, two outputs; slices side by side and in place pass the check (n = 0 launches
    # nothing, so they are tried with the overlap of the next argument instead)
    assert call(y=((1 << 20) + 512, 1 << 23)) == INVALID
    assert call(y=(1 << 21, 1 << 23)) == INVALID
    assert call(y=(1 << 22, 1 << 22)) == INVALID and b"outputs" in h.qwha_last_error()
    base = 1 << 20
    assert call(x=(base, base + 512), xs=(384, 384), y=(base, base + 512), ys=(384, 384), heads=(4, 4)) == INVALID
    assert call(x=(base, base + 512), xs=(384, 384), y=(base, base + 512), ys=(384, 384), pos=None) == INVALID
    assert b"positions" in h.qwha_last_error()
    assert call(n=0, x=(None, None)) == OK


def _attend(h, k, v, dt=1, q=P(1 << 20), n=4, q_heads=4, stride=512, pages=BUF, max_pages=2, q_start=BUF, past=BUF, n_seqs=2,
            tree=None, scale=0.1, out=P(1 << 22), lse=None, ws=BUF, nbytes=1 << 30):
    ref = lambda c: None if c is None else ctypes.byref(c)  # noqa: E731
    return h.qwha_cache_attention(ref(k), ref(v), dt, q, n, q_heads, stride, pages, max_pages, q_start, past, n_seqs, tree,
                                  ctypes.c_float(scale), out, lse, ws, nbytes, None)


def test_attention_refusals():
    L = _L()
    h, c = L.lib(), _cache(L)
    call = lambda **kw: _attend(h, c, c, **kw)  # noqa: E731
    assert _attend(h, None, c) == INVALID and _attend(h, c, None) == INVALID
    for kw in (dict(heads=4), dict(head_dim=64), dict(page_size=8), dict(n_pages=5)):
        assert _attend(h, c, _cache(L, **kw)) == INVALID and b"differ" in h.qwha_last_error()
    for kw in (dict(bits=5), dict(group=48), dict(had_block=3), dict(codes=None)):
        assert _attend(h, c, _cache(L, **kw)) == INVALID and _attend(h, _cache(L, **kw), c) == INVALID
    assert call(dt=2) == INVALID
    assert call(q_heads=3) == INVALID and call(q_heads=0) == INVALID
    assert call(n=-1) == INVALID and call(n=1 << 31) == INVALID
    assert call(n_seqs=-1) == INVALID and call(max_pages=-1) == INVALID
    assert call(scale=float("nan")) == INVALID and call(scale=float("inf")) == INVALID
    assert call(stride=504) == INVALID and call(stride=516) == MISALIGNED
    for name in ("q", "out", "pages", "q_start", "past", "ws"):
        assert call(**{name: None}) == (WORKSPACE if name == "ws" else INVALID), name
        assert call(**{name: P(4098)}) == MISALIGNED, name  # index arrays: not aligned to their elements
    assert call(tree=P(4)) == MISALIGNED and call(lse=P(8)) == MISALIGNED
    need = h.qwha_workspace_size(13, 4, 128, 2, 4, 1)
    assert need > 0 and call(nbytes=need - 1) == WORKSPACE
    assert call(out=P((1 << 20) + 1024)) == INVALID  # q and out overlap
    assert call(lse=P(1 << 20)) == INVALID and call(lse=P(1 << 22)) == INVALID
    assert call(n=0, q=None, out=None) == OK and call(n_seqs=0, q=None) == OK


def test_page_refusals():
    L = _L()
    h = L.lib()

    def table(**kw):
        f = dict(page_size=16, max_pages=8, n_seqs=4, n_pages=32, refs=4096, pages=4096, held=4096)
        f.update(kw)
        return ctypes.byref(L.QwhaPageTable(**f))

    need = h.qwha_workspace_size(14, 4, 1, 32, 0, 0)
    more = h.qwha_workspace_size(14, 4, 1, 32, 3, 0)
    assert more > need >= 4 * 32
    for kw, want in ((dict(page_size=0), INVALID), (dict(max_pages=-1), INVALID), (dict(n_seqs=-1), INVALID),
                     (dict(n_pages=-1), INVALID), (dict(refs=None), INVALID), (dict(pages=4098), MISALIGNED),
                     (dict(held=None), INVALID)):
        assert h.qwha_pages_resize(table(**kw), BUF, BUF, need, None) == want, kw
        assert h.qwha_pages_fork(table(**kw), BUF, BUF, 3, BUF, BUF, BUF, more, None) == want, kw
    assert h.qwha_pages_resize(None, BUF, BUF, need, None) == INVALID
    assert h.qwha_pages_resize(table(), None, BUF, need, None) == INVALID
    assert h.qwha_pages_resize(table(), BUF, BUF, need - 1, None) == WORKSPACE
    assert h.qwha_pages_resize(table(n_seqs=0), None, None, 0, None) == OK
    assert h.qwha_pages_fork(table(), BUF, BUF, -1, BUF, BUF, BUF, more, None) == INVALID
    assert h.qwha_pages_fork(table(), BUF, None, 3, BUF, BUF, BUF, more, None) == INVALID
    assert h.qwha_pages_fork(table(), BUF, BUF, 3, BUF, P(6), BUF, more, None) == MISALIGNED
    assert h.qwha_pages_fork(table(), BUF, BUF, 3, BUF, BUF, BUF, more - 1, None) == WORKSPACE
    assert h.qwha_pages_fork(table(), None, None, 0, None, None, None, 0, None) == OK


@pytest.mark.parametrize("kw,want", [(dict(bits=5), INVALID), (dict(heads=0), INVALID), (dict(group=48), INVALID),
                                     (dict(scales=4104), MISALIGNED), (dict(n_pages=-1), INVALID)])
def test_move_refusals_of_the_caches(kw, want):
    L = _L()
    h = L.lib()
    c = (L.QwhaCache * 2)(_cache(L), _cache(L, **kw))
    assert h.qwha_cache_copy_pages(c, 2, BUF, BUF, 3, None) == want
    assert h.qwha_cache_compact(c, 2, BUF, 2, BUF, BUF, 4, 2, None) == want


def test_move_refusals():
    L = _L()
    h = L.lib()
    c = (L.QwhaCache * 1)(_cache(L))
    assert h.qwha_cache_copy_pages(c, 0, BUF, BUF, 3, None) == INVALID
    assert h.qwha_cache_copy_pages(None, 1, BUF, BUF, 3, None) == INVALID
    assert h.qwha_cache_copy_pages(c, 1, BUF, BUF, -1, None) == INVALID
    assert h.qwha_cache_copy_pages(c, 1, None, BUF, 3, None) == INVALID
    assert h.qwha_cache_copy_pages(c, 1, BUF, P(6), 3, None) == MISALIGNED
    assert h.qwha_cache_copy_pages(c, 1, None, None, 0, None) == OK
    assert h.qwha_cache_compact(c, 3, BUF, 2, BUF, BUF, 4, 2, None) == INVALID
    assert h.qwha_cache_compact(c, 1, BUF, -1, BUF, BUF, 4, 2, None) == INVALID
    assert h.qwha_cache_compact(c, 1, BUF, 2, BUF, BUF, -1, 2, None) == INVALID
    assert h.qwha_cache_compact(c, 1, None, 2, BUF, BUF, 4, 2, None) == INVALID
    assert h.qwha_cache_compact(c, 1, BUF, 2, P(4), BUF, 4, 2, None) == MISALIGNED
    assert h.qwha_cache_compact(c, 1, BUF, 2, BUF, None, 4, 2, None) == INVALID
    assert h.qwha_cache_compact(c, 1, BUF, 2, BUF, BUF, 0, 2, None) == OK
    assert h.qwha_cache_compact(c, 1, BUF, 2, BUF, BUF, 4, 0, None) == OK


def test_rotary_frequencies():
    _L()
    from walsh_hadamard_sparse_b200 import rotary_frequencies as rf

    f, m = rf(8, 10000.0, device="cpu")
    assert m == 1.0 and np.allclose(f.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-15)
    assert np.allclose(rf(8, scaling="linear", factor=4.0, device="cpu")[0].numpy(), f.numpy() / 4, rtol=1e-15)
    g = rf(64, scaling="base", factor=4.0, device="cpu")[0].numpy()
    plain = rf(64, device="cpu")[0].numpy()
    assert g[0] == 1.0 and np.isclose(g[-1], plain[-1] / 4, rtol=1e-12) and np.all(g <= plain)
    for how in ("ramp", "bands"):
        g, m = rf(64, scaling=how, factor=4.0, trained=4096, low=1.0, high=32.0, device="cpu")
        r = plain / g.numpy()
        turns = 4096 * plain / (2 * np.pi)
        assert np.all(r >= 1 - 1e-12) and np.all(r <= 4 + 1e-12) and np.all(np.diff(r) >= -1e-12)
        assert r[0] == 1.0 and np.isclose(r[-1], 4.0)
        assert np.allclose(r[turns > 34], 1.0, atol=1e-12) or how == "ramp"
        assert m == (0.1 * np.log(4.0) + 1.0 if how == "ramp" else 1.0)
    assert rf(0, device="cpu")[0].shape == (0,)
    for bad in (dict(rot=7), dict(rot=8, scaling="x"), dict(rot=8, base=1.0), dict(rot=8, factor=0.0), dict(rot=8, low=4, high=2)):
        with pytest.raises(ValueError):
            rf(**bad, device="cpu")


def test_the_plain_rotary_is_a_rotation_and_its_inverse():
    g = np.random.default_rng(1)
    x, pos, freq = g.standard_normal((5, 2, 24)), g.integers(0, 1000, 5), g.uniform(0, 1, 8)
    for pairs in (False, True):
        y = rotary(x, pos, freq, pairs, 1.0, False)
        assert np.allclose((y**2).sum(-1), (x**2).sum(-1))
        assert np.allclose(rotary(y, pos, freq, pairs, 1.0, True), x)
        dy = g.standard_normal(x.shape)  # the inverse is the gradient: <dy, R x> = <R^T dy, x>
        assert np.isclose((dy * y).sum(), (rotary(dy, pos, freq, pairs, 1.0, True) * x).sum())


def test_the_plain_table():
    t = Table(np.zeros(6, np.int32), np.full((3, 4), -1, np.int32), np.zeros(3, np.int64), 4)
    t.resize([6, 4, 0])
    assert t.pages[0, :2].tolist() == [0, 1] and t.pages[1, 0] == 2 and t.held.tolist() == [6, 4, 0]
    origin, fresh, bad = t.fork([0], [2])
    assert not bad and origin.tolist() == [1] and fresh.tolist() == [3] and t.pages[2].tolist() == [0, 3, -1, -1]
    assert t.refs.tolist() == [2, 1, 1, 1, 0, 0]
    t.resize([16, 8, -1])  # two more pages for row 0 and one for row 1: only two are free
    assert t.held.tolist() == [16, 4, 6] and t.pages[0].tolist() == [0, 1, 4, 5]
    t.resize([0, 8, -1])
    assert t.refs.tolist() == [1, 1, 1, 1, 0, 0] and t.pages[1, :2].tolist() == [2, 1]
