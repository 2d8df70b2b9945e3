"""The operators around the cache where calls that their documentation allows lie at a border: blocks of cached heads that are
not full, pages that two sequences name, groups without values, scales far apart, long moves."""

import functools

import numpy as np
import pytest

import _cache_ops as R
from _serving import half_step, pack, unpack
from _util import host, to_dev
from test_cache_ops_gpu import Setup, _W, _ints, poison, random_trees
from workloads import rng_for

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- blocks of heads


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,D,bits,group", [(9, 128, 4, 128), (11, 64, 8, 64), (13, 128, 4, 32), (20, 64, 4, 64), (9, 80, 3, 40),
                                                (11, 24, 8, 8), (5, 256, 8, 64), (7, 256, 8, 256)])
def test_attention_blocks_of_heads_that_are_not_full(heads, D, bits, group, dtype, monkeypatch):
    """Numbers of cached heads whose last block has fewer than the others, in a pool whose every slot is used: the last block
    takes nothing from behind the last token."""
    monkeypatch.setattr(R, "shuffled_table", functools.partial(R.shuffled_table, spare=0))
    key = f"{heads}-{D}-{bits}-{group}-{dtype}"
    for new, grp in ((1, 1), (3, 2)):
        s = Setup(f"blocks{key}{new}", [15, 160, 33, 0], [new] * 4, heads=heads, grp=grp, D=D, bits=bits, group=group, dtype=dtype, room=1 << 20,
                  page_size=1, tree=random_trees if new > 1 else None)
        assert s.kv[0].n_slots == sum(s.past) + 4 * new  # no page is left over
        s.check()


# ---------------------------------------------------------------- pages that two sequences name


class GuardedTable(R.Table):
    """The page table whose sequences do not grow inside a page with other users: they claim one (copies) or stay."""

    def resize(self, want, copies=False):
        n, ps = len(want), self.ps
        origin, fresh, bad = np.full(n, -1, np.int32), np.full(n, -1, np.int32), False
        grow = []
        for b, w in enumerate(want):
            if w == -1:
                continue
            if w < -1 or w > self.pages.shape[1] * ps:
                bad = True
            elif w <= self.held[b]:
                for j in range(self.count(w), self.count(self.held[b])):
                    self.refs[self.pages[b, j]] -= 1
                    self.pages[b, j] = -1
                self.held[b] = w
            else:
                grow.append(b)
        free, at, refs = self.free(), 0, self.refs.copy()
        for b in grow:
            have, to = self.count(self.held[b]), self.count(want[b])
            claim = int(self.held[b] % ps > 0 and refs[self.pages[b, have - 1]] > 1)
            if claim and not copies:
                bad = True
                continue
            at += to - have + claim
            if at > len(free) and to - have + claim:
                continue
            got = free[at - (to - have + claim):at]
            if claim:
                origin[b], fresh[b] = self.pages[b, have - 1], got[0]
                self.refs[origin[b]] -= 1
                self.pages[b, have - 1] = got[0]
            self.pages[b, have:to] = got[claim:]
            self.refs[got] = 1
            self.held[b] = want[b]
        return origin, fresh, bad


def _same(t, d):
    assert np.array_equal(_ints(d.refs), t.refs) and np.array_equal(_ints(d.pages), t.pages) and np.array_equal(_ints(d.held), t.held)


@pytest.mark.parametrize("copies", [False, True])
@pytest.mark.parametrize("n_seqs,n_pages,max_pages,page_size", [(3, 10, 4, 16), (40, 200, 12, 5), (600, 3000, 9, 16), (600, 1100, 9, 16),
                                                                (2100, 9000, 7, 16), (33, 4097, 64, 3), (20, 70000, 400, 3)])
def test_a_guarded_page_table(n_seqs, n_pages, max_pages, page_size, copies):
    """Random growth, cuts and forks: no sequence grows inside a page that another one names, pages running out among them."""
    import torch

    W, g = _W(), rng_for(350, str(n_seqs), str(n_pages))
    t = GuardedTable(np.zeros(n_pages, np.int32), np.full((n_seqs, max_pages), -1, np.int32), np.zeros(n_seqs, np.int64), page_size)
    d = W.PageTable(page_size, to_dev(t.refs), to_dev(t.pages), to_dev(t.held), guard=not copies)
    room, share, claims, refused = max_pages * page_size, max(1, n_pages * page_size // n_seqs), 0, 0
    for step in range(10):
        want = g.integers(0, min(room, 2 * share) + 1, n_seqs)
        want[g.random(n_seqs) < 0.3] = -1
        want[g.random(n_seqs) < 0.1] = 0
        out = (torch.full((n_seqs,), 7, dtype=torch.int32, device="cuda"), torch.full((n_seqs,), 7, dtype=torch.int32, device="cuda"))
        W.pages_resize(d, to_dev(want), copies=out if copies else None)
        origin, fresh, bad = t.resize(want, copies)
        _same(t, d)
        if copies:
            assert np.array_equal(_ints(out[0]), origin) and np.array_equal(_ints(out[1]), fresh) and not bad
            claims += int((origin >= 0).sum())
            assert not set(origin[origin >= 0]) & set(fresh[fresh >= 0])  # as cache_copy_pages wants them
        refused += bad
        if bad:
            with pytest.raises(W.QwhaError, match="shared page"):
                W.check_stream_status()
        dst = g.permutation(np.flatnonzero(t.held == 0))[:max(1, n_seqs // 3)]
        src = g.integers(-1, n_seqs, len(dst))
        if len(dst):
            t.fork(src, dst)
            W.pages_fork(d, to_dev(src), to_dev(dst))
            _same(t, d)
    W.check_stream_status()
    assert n_seqs < 10 or (claims if copies else refused)


def test_a_sequence_cut_back_to_a_shared_prefix_writes_to_its_own_page():
    """A's 32 tokens in two pages, B a fork of it that is cut back to 20 tokens and goes on: A keeps its tokens, B has A's first
    20; and A cut back itself, with B reading."""
    import torch

    W, g = _W(), rng_for(351)
    ps, heads, D = 16, 2, 64
    for which in (0, 1):  # who is cut back and grows
        t = W.page_table(12, ps, 2, 4)
        caches = tuple(W.cache_alloc(12, ps, heads, D, bits=4, group=64, had_block=0) for _ in range(2))

        def write(b, lo, hi):
            rows = [torch.randn(hi - lo, heads, D, generator=torch.Generator(device="cuda").manual_seed(int(g.integers(1 << 30))),
                                device="cuda") for _ in range(2)]
            table = _ints(t.pages)
            slots = np.array([table[b, i // ps] * ps + i % ps for i in range(lo, hi)], np.int64)
            W.cache_write(caches, tuple(rows), to_dev(slots))

        def read(b, n):
            return [x.clone() for x in W.cache_read(caches, t.pages[b:b + 1].contiguous(), to_dev(np.array([0, n], np.int64)), n,
                                                    dtype=torch.float32)]

        W.pages_resize(t, to_dev(np.array([32, 0])))
        write(0, 0, 32)
        copies = W.pages_fork(t, to_dev(np.array([0])), to_dev(np.array([1])))
        W.cache_copy_pages(caches, *copies)
        assert int(t.refs.max()) == 2
        both = [read(b, 32) for b in (0, 1)]
        cut, other = which, 1 - which
        want = np.array([-1, -1])
        want[cut] = 20
        W.pages_resize(t, to_dev(want))
        assert t.held.tolist()[cut] == 20
        want[cut] = 21
        W.pages_resize(t, to_dev(want))  # without copies: it stays, and is reported
        assert t.held.tolist()[cut] == 20 and int(t.refs.sum()) == 4
        with pytest.raises(W.QwhaError, match="shared page"):
            W.check_stream_status()
        out = (torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"))
        W.pages_resize(t, to_dev(want), copies=out)
        assert t.held.tolist()[cut] == 21 and int(t.refs.max()) == 2 and int(t.refs.sum()) == 4
        assert out[0].tolist()[cut] == int(t.pages[other, 1]) and out[1].tolist()[cut] == int(t.pages[cut, 1])
        W.cache_copy_pages(caches, *out)
        write(cut, 20, 21)
        for x, y in zip(read(other, 32), both[other]):
            assert torch.equal(x, y)
        for x, y in zip(read(cut, 21), both[cut]):
            assert torch.equal(x[:20], y[:20]) and not torch.equal(x[20], y[20])
        W.pages_resize(t, to_dev(want + 3 * (want >= 0)))  # its own page now: nothing more to ask
        assert t.held.tolist()[cut] == 24
        W.check_stream_status()


def test_a_guarded_page_table_in_a_graph():
    import torch

    W = _W()
    d = W.page_table(64, 16, 4, 8)
    W.pages_resize(d, torch.tensor([32, 0, 0, 16], device="cuda"))
    W.pages_fork(d, torch.tensor([0, 0], device="cuda"), torch.tensor([1, 2], device="cuda"))
    cut, want = torch.tensor([20, 20, 32, 16], device="cuda"), torch.tensor([40, 21, 33, 17], device="cuda")
    out = tuple(torch.empty(4, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(W.workspace_size(W.api.OP_PAGES, 4, 1, 64, 0, 0), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        W.pages_resize(d, cut, ws=ws)
        W.pages_resize(d, want, ws=ws, copies=out)
    g.replay()
    first = [x.tolist() for x in (d.pages, d.held, *out)]
    assert first[1] == [40, 21, 33, 17] and first[2][:2] == [1, 1] and first[2][2:] == [-1, -1] and first[0][2][1] == 1
    g.replay()  # the pages are their own now
    assert out[0].tolist() == [-1] * 4 and d.held.tolist() == first[1]
    assert int((d.refs > 0).sum()) == d.pages[d.pages >= 0].unique().numel()
    W.check_stream_status()


def test_rows_that_contradict_the_table_are_left():
    """Entries outside the cache, counts of no users: the rows and pairs that hold them change nothing, the others are served."""
    import torch

    W = _W()
    pages = np.full((8, 4), -1, np.int32)
    pages[0], pages[1, :2], pages[2, :2], pages[3, :3] = [0, 1, 2, 3], [4, 77], [-5, 5], [6, 7, 8]
    refs = np.zeros(20, np.int32)
    refs[[0, 1, 2, 3, 4, 5, 6, 8]] = 1  # page 7 is named by row 3 and counts no users
    held = np.array([16, 8, 7, 10, 0, 0, 0, 0], np.int64)

    def table(guard):
        return W.PageTable(4, to_dev(refs), to_dev(pages), to_dev(held), guard)

    for guard in (False, True):
        d = table(guard)
        W.pages_resize(d, to_dev(np.array([5, 0, 0, -1, 6, -1, -1, -1])))
        with pytest.raises(W.QwhaError, match="page table"):
            W.check_stream_status()
        assert d.held.tolist() == [5, 8, 7, 10, 6, 0, 0, 0]
        assert d.pages.tolist() == [[0, 1, -1, -1], *pages[1:4].tolist(), [2, 3, -1, -1], *pages[5:].tolist()]
        assert d.refs[:9].tolist() == [1, 1, 1, 1, 1, 1, 1, 0, 1] and int(d.refs.sum()) == 8
        # the page without users: given back, its count stays 0
        W.pages_resize(d, to_dev(np.array([-1, -1, -1, 4, -1, -1, -1, -1])))
        with pytest.raises(W.QwhaError, match="page table"):
            W.check_stream_status()
        assert d.held.tolist()[3] == 4 and d.refs[6:9].tolist() == [1, 0, 0]
    d = table(False)
    a, b = W.pages_fork(d, to_dev(np.array([1, 2, 3, 0])), to_dev(np.array([4, 5, 6, 7])))
    with pytest.raises(W.QwhaError, match="page table"):
        W.check_stream_status()
    assert a.tolist() == b.tolist() == [-1] * 4
    assert d.held.tolist() == [16, 8, 7, 10, 0, 0, 0, 16] and torch.equal(d.pages[:7], to_dev(pages)[:7])
    assert d.pages[7].tolist() == [0, 1, 2, 3] and d.refs[:9].tolist() == [2, 2, 2, 2, 1, 1, 1, 0, 1] and int(d.refs[9:].max()) == 0


# ---------------------------------------------------------------- groups without values


def put_idle(s, g, share=0.15):
    """Groups of a Setup's pools whose codes become their zero points, in every pool: [pools] of masks like the scales."""
    masks = []
    for (codes, sc, z), bits, group in zip((s.pk, s.pv), s.fmt[:2], (s.fmt[2], s.group_v)):
        m = g.random(sc.shape) < share
        q = unpack(codes, bits)
        codes[...] = pack(np.where(np.repeat(m, group, -1), np.repeat(z, group, -1), q).astype(np.uint8), bits)
        masks.append(m)
    return masks


def to_caches(s):
    for pool, cache in zip((s.pk, s.pv), s.kv):
        for t, d in zip(pool, (cache.codes, cache.scales, cache.zeros)):
            d.copy_(to_dev(t))


@pytest.mark.parametrize("dtype,grp,new", [("bf16", 2, 4), ("f32", 3, 5), ("bf16", 3, 8), ("bf16", 4, 40), ("f32", 2, 30), ("bf16", 1, 2)])
@pytest.mark.parametrize("D,bits,group", [(128, 4, 128), (64, 2, 32), (128, 3, 64), (96, 8, 32), (40, 4, 8), (256, 3, 128), (24, 3, 8),
                                          (80, 2, 16)])
def test_attention_groups_without_values_have_no_say(D, bits, group, dtype, grp, new):
    """A group whose codes all equal its zero point is zeros, whatever its scale: tiny, the 1 that cache_write stores for a row
    of zeros, or far above all others, the results of trees and chunks have the same bits; one that is a NaN stays one."""
    for tree in (None, random_trees):
        s = Setup(f"idle{D}{bits}{group}{dtype}{grp}{new}", [70, 300], [new, new], heads=3, grp=grp, D=D, bits=bits, group=group, dtype=dtype,
                  tree=tree, had_v=8)
        masks = put_idle(s, s.g)
        s.pv[1][...] *= np.float32(2.0**-12)
        results = []
        for scale in (2.0**-40, 1.0, -(2.0**60)):
            for m, pool in zip(masks, (s.pk, s.pv)):
                pool[1][m] = scale
            to_caches(s)
            results.append((host(s.run()), host(s.lse)))
        for out, lse in results[1:]:
            assert np.array_equal(out, results[0][0]) and np.array_equal(lse, results[0][1])
        for m, pool in zip(masks, (s.pk, s.pv)):
            pool[1][m] = 2.0**-40
        s.check(to_dev(results[2][0]))  # the bounds of tiny scales hold for the others
        # a token of the past of sequence 1, which all its rows see (but those that see nothing of a tree see the past too)
        slot = int(s.table[1, 200 // 16]) * 16 + 200 % 16
        for pool in (s.pk, s.pv):
            keep = pool[1].copy()
            pool[1].reshape(-1, *pool[1].shape[2:])[slot, 1] = np.nan
            to_caches(s)
            got = host(s.run())
            assert np.isnan(got[new:, grp:2 * grp]).any(-1).all() and not np.isnan(got[:new]).any() and not np.isnan(got[:, 2 * grp:]).any()
            pool[1][...] = keep
        _W().check_stream_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,bits,group", [(128, 4, 128), (128, 8, 64), (40, 4, 8)])
def test_attention_of_one_token_with_groups_without_values(D, bits, group, dtype):
    """The same with the scale 1 that cache_write stores and one token to a sequence: within the bounds."""
    s = Setup(f"idleone{D}{bits}{group}{dtype}", [70, 300], [1, 1], heads=3, grp=2, D=D, bits=bits, group=group, dtype=dtype)
    for m, pool in zip(put_idle(s, s.g), (s.pk, s.pv)):
        pool[1][...] *= np.float32(2.0**-9)
        pool[1][m] = 1.0
    to_caches(s)
    s.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("past,new,heads,grp,D,bits,group,page_size", [
    ([700], [64], 2, 4, 128, 4, 128, 16), ([33, 0, 500], [64, 5, 33], 9, 2, 64, 8, 32, 3), ([300, 64], [7, 3], 3, 40, 128, 3, 64, 16),
    ([100, 31], [9, 40], 2, 3, 256, 4, 128, 16), ([90] * 20, [6] * 20, 5, 1, 40, 4, 8, 16), ([0, 50], [130, 60], 1, 5, 96, 2, 96, 100)])
def test_attention_of_tiles_done_again(past, new, heads, grp, D, bits, group, page_size, dtype):
    """Tokens of far larger scales in the middle and at the end of the new ones: rows that do not see them, in every part of a
    group and block of heads, one sequence to all CTAs and many; what they hold may be no number; the same bits again."""
    for tree in (None, random_trees)[:1 + (max(new) <= 64)]:
        s = Setup(f"again{past[0]}{D}{dtype}", past, new, heads=heads, grp=grp, D=D, bits=bits, group=group, page_size=page_size, dtype=dtype,
                  tree=tree, had_v=8, size=0.5)
        for b, m in enumerate(new):
            for u in {m // 2, m - 1}:
                poison(s, (b, past[b] + u), 2.0**22, (0, 1))
        got = s.check()
        for _ in range(2):
            assert np.array_equal(host(s.run()), got)
        if tree is None:  # the last token of the first sequence is seen by the last row alone
            slot = int(s.table[0, (past[0] + new[0] - 1) // page_size]) * page_size + (past[0] + new[0] - 1) % page_size
            for c in s.kv:
                c.scales.view(s.kv[0].n_slots, heads, -1)[slot] = float("nan")
            out = host(s.run())
            assert np.isnan(out[new[0] - 1]).any(-1).all()
            # (not the same bits: where the tile is not done again its other rows' weights are rounded to the largest scale met)
            want, _, tol, _ = s.ref()
            others = np.arange(len(out)) != new[0] - 1
            assert np.all((np.abs(out - want) <= tol + half_step(dtype) * np.abs(want))[others])


def lift(s, b, t, which, factor, channel):
    """Token t of sequence b: scales of pool `which` times factor, its codes zero points but for one channel."""
    slot, bits, group = int(s.table[b, t // s.page_size]) * s.page_size + t % s.page_size, s.fmt[which], (s.fmt[2], s.group_v)[which]
    codes, sc, z = (s.pk, s.pv)[which]
    codes, sc, z = (x.reshape(-1, *x.shape[2:])[slot] for x in (codes, sc, z))
    q, zz = unpack(codes, bits), np.repeat(z, group, -1)
    idle = zz.copy()
    idle[:, channel] = np.where(q[:, channel] == zz[:, channel], zz[:, channel] ^ 1, q[:, channel])
    codes[...] = pack(idle.astype(np.uint8), bits)
    sc *= np.float32(factor)
    return slot


@pytest.mark.parametrize("past,new,grp,heads", [([300, 40], [40, 64], 4, 2), ([2000], [130], 2, 2), ([700, 100], [1, 1], 60, 1)])
@pytest.mark.parametrize("D,bits,group", [(128, 4, 128), (64, 8, 32), (96, 3, 32), (128, 2, 64)])
@pytest.mark.parametrize("factor", [2.0**11, 2.0**16, 2.0**20, 2.0**24, 2.0**30])
def test_attention_of_many_rows_keeps_tokens_beside_one_of_a_far_larger_scale(factor, D, bits, group, past, new, grp, heads):
    """A token that all rows see, whose key or value is large in one channel alone: the query has nothing there, or the output is
    looked at in the others. What is left of it there is nothing, and the other tokens keep all their bits."""
    for which in (0, 1):
        for at in (0, past[0] - 1):
            s = Setup(f"beside{D}{bits}{factor}{past[0]}{which}", past, new, heads=heads, grp=grp, D=D, bits=bits, group=group)
            assert s.cached
            channel = D - 3
            slot = lift(s, 0, at, which, factor, channel)
            to_caches(s)
            if which == 0:
                s.qv[..., channel] = 0.0
                s.q[..., channel] = 0.0
            got = host(s.run())
            kd, vd = (R.dense_pool(p, bits, group) for p in (s.pk, s.pv))
            step = R.largest_steps(s.pv, bits, group)
            step[slot] = np.abs(vd[slot]) if which else step[slot]
            want, lse, tol, lse_tol = R.attention(s.qv, kd, vd, step, 0, 0, s.table, 16, s.past, s.new, None, s.scale, 2.0**-11, s.cached)
            keep = np.arange(D) != channel
            err = np.abs(got - want)[..., keep] - half_step("bf16") * np.abs(want)[..., keep]
            assert np.all(err <= tol[..., keep])
            if which == 0:
                assert np.all(np.abs(host(s.lse) - lse) <= lse_tol)
            _W().check_stream_status()


# ---------------------------------------------------------------- the choice of the kernel


@pytest.mark.parametrize("D,bits,group", [(128, 4, 128), (64, 8, 32), (96, 3, 32)])
@pytest.mark.parametrize("new,grp", [(3, 4), (8, 5), (20, 2)])
def test_attention_told_of_the_longest_sequence(D, bits, group, new, grp):
    """A wide table with the longest length is answered as a narrow one is, by the same kernel; a wide one without by the one
    that keeps cached values exact; whatever is told, the answer is right."""
    key = dict(heads=2, grp=grp, D=D, bits=bits, group=group, tree=random_trees, had_v=8)
    narrow = Setup(f"upto{D}{new}", [300, 70, 0], [new] * 3, **key)
    wide = Setup(f"upto{D}{new}", [300, 70, 0], [new] * 3, room=1 << 20, **key)
    want = host(narrow.run())
    assert np.array_equal(host(wide.run(longest=300 + new)), want) and np.array_equal(host(wide.lse), host(narrow.lse))
    for longest in (0, 5, 1 << 40):
        wide.check(wide.run(longest=longest))
    wide.cached = 0.0
    wide.check()
    wide.check(wide.run(longest=1 << 20))


@pytest.mark.parametrize("D,bits,bits_v,group", [(128, 4, 4, 128), (64, 3, 8, 32), (96, 8, 2, 96), (128, 2, 3, 64), (32, 4, 4, 32)])
@pytest.mark.parametrize("new,grp", [(3, 3), (4, 4), (11, 4), (22, 2), (44, 1)])
def test_attention_of_9_to_44_rows_keeps_cached_values_exact(D, bits, bits_v, group, new, grp):
    """In a table of much room, bounds without a rounding of what is cached: chunks and trees, scales over powers of two."""
    for tree in (None, random_trees):
        s = Setup(f"exact{D}{bits}{new}", [150, 33], [new, new], heads=3, grp=grp, D=D, bits=bits, bits_v=bits_v, group=group, tree=tree,
                  room=1 << 20, had_k=8)
        assert s.cached
        s.cached = 0.0
        s.check()
        s.pk[1][...] *= (2.0 ** s.g.integers(-6, 1, s.pk[1].shape)).astype(np.float32)
        s.pv[1][...] *= (2.0 ** s.g.integers(-3, 3, s.pv[1].shape)).astype(np.float32)
        to_caches(s)
        s.check()


# ---------------------------------------------------------------- long moves


@pytest.mark.parametrize("heads,D,bits,group,page_size,past,kept", [(2, 128, 4, 128, 64, [20000], [9000]), (1, 24, 3, 8, 7, [3000, 700, 129, 128], [2999, 129, 128, 128]),
                                                                  (8, 64, 8, 32, 16, [4096, 1, 4095, 0], [257, 1, 4095, 0])])
def test_compact_of_a_long_context(heads, D, bits, group, page_size, past, kept):
    """Thousands of kept tokens, in pages that are not in order; sequences that keep all, one or none; a row that breaks off
    behind the first 128 and one behind the second."""
    W, g = _W(), rng_for(360, str(heads), str(D))
    first = np.array([11 if n > 2000 else 0 for n in past], np.int64)
    table, n_pages = R.shuffled_table(g, [n + int(f) for n, f in zip(past, first)], page_size)
    pools = [R.random_pool(g, n_pages, page_size, heads, D, b, group) for b in (bits, 4)]
    caches = tuple(W.QCache(b, group, 0, *(to_dev(t) for t in p)) for b, p in zip((bits, 4), pools))
    keep = np.full((len(past), max(kept) + 1), -1, np.int32)
    for b, (n, m) in enumerate(zip(past, kept)):
        keep[b, :m] = np.sort(g.choice(n, m, replace=False))

    def move(keep):
        for p in pools:
            for t in p:
                flat = t.reshape(-1, *t.shape[2:])
                old = flat.copy()
                for b, row in enumerate(keep):
                    stop = np.flatnonzero(np.diff(row, prepend=-1) <= 0)
                    u = row[:stop[0] if len(stop) else len(row)].astype(np.int64)
                    at = [first[b] + u, first[b] + np.arange(len(u))]
                    src, dst = (table[b, x // page_size] * np.int64(page_size) + x % page_size for x in at)
                    flat[dst] = old[src]

    W.cache_compact(caches, to_dev(table), to_dev(first), to_dev(keep))
    W.check_stream_status()
    move(keep)
    broken = keep.copy()
    for b, at in enumerate((128, 129, 127, 256)[:len(past)]):
        if kept[b] > at:
            broken[b, at] = broken[b, at - 1]
    W.cache_compact(caches, to_dev(table), to_dev(first), to_dev(broken))
    with pytest.raises(W.QwhaError, match="ascend"):
        W.check_stream_status()
    move(broken)
    for p, c in zip(pools, caches):
        for want, got in zip(p, (c.codes, c.scales, c.zeros)):
            assert np.array_equal(_ints(got), want)
