"""The operators around the cache on the GPU against their plain statements in 64 bits: rotary positions, attention over
the cache, the page table, moves of cached rows, and a step of speculative answering that uses them together."""

import numpy as np
import pytest

import _cache_ops as R
from _serving import half_step, quantize, values, pack
from _util import bf16_dev, host, to_dev
from workloads import f32_to_bf16_bits, rng_for

pytestmark = pytest.mark.gpu

F32 = 2.0**-24


def _rows(g, shape, dtype, size=1.0):
    """(device tensor, its values in fp64)"""
    import torch

    x = (g.standard_normal(shape) * size).astype(np.float32)
    t = to_dev(x) if dtype == "f32" else bf16_dev(f32_to_bf16_bits(x).reshape(shape))
    assert t.dtype == (torch.float32 if dtype == "f32" else torch.bfloat16)
    return t, host(t)


def _W():
    import walsh_hadamard_sparse_b200 as W

    return W


def _ints(t):
    return t.cpu().numpy()


# ---------------------------------------------------------------- rotary


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,rot,n,hq,hk", [(64, 64, 1, 1, 1), (128, 128, 5, 32, 8), (80, 40, 3, 3, 1), (80, 32, 700, 2, 2),
                                           (256, 256, 2, 7, 1), (96, 0, 4, 2, 1), (8, 2, 3, 5, 5), (64, 6, 9, 4, 2)])
def test_rotary(dtype, pairs, D, rot, n, hq, hk):
    import torch

    W, g = _W(), rng_for(301, dtype, str(pairs), str(D), str(rot))
    wide, x = _rows(g, (n, hq + 2 * hk, D), dtype)
    pos = np.concatenate([[0], g.integers(0, 1 << 20, n)])[-n:] if n > 1 else np.array([131071])
    freq = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    dp, df = to_dev(pos.astype(np.int64)), to_dev(freq)
    for factor, inverse in ((1.0, False), (1.25, True)):
        q, k = W.rotary((wide[:, :hq], wide[:, hq:hq + hk]), dp, df, interleaved=pairs, factor=factor, inverse=inverse)
        assert q.shape == (n, hq, D) and q.is_contiguous() and k.shape == (n, hk, D)
        ref = R.rotary(x, pos, freq, pairs, factor, inverse)
        # sine and cosine: 4 roundings of fp32 (the turned rest, the function to 2 ulp, the factor), two products and a sum
        size = np.abs(ref[..., :0].sum(-1, keepdims=True)) + np.sqrt((x[..., :rot] ** 2).max(-1, keepdims=True, initial=0) * 2) * factor
        for got, part in ((q, slice(0, hq)), (k, slice(hq, hq + hk))):
            tol = half_step(dtype) * np.abs(ref[:, part]) + 10 * F32 * size[:, part]
            assert np.all(np.abs(host(got) - ref[:, part]) <= tol)
            assert np.array_equal(host(got)[..., rot:], x[:, part, rot:])  # copied, not computed
    one = W.rotary(wide[:, :hq], dp, df, interleaved=pairs)
    both = W.rotary((wide[:, :hq], wide[:, hq:hq + hk]), dp, df, interleaved=pairs)
    assert torch.equal(one, both[0])
    held = wide.clone()  # in place, within the projection: the values' heads stay
    out = W.rotary((held[:, :hq], held[:, hq:hq + hk]), dp, df, interleaved=pairs, out=(held[:, :hq], held[:, hq:hq + hk]))
    assert torch.equal(held[:, :hq], both[0]) and torch.equal(held[:, hq:hq + hk], both[1])
    assert torch.equal(held[:, hq + hk:], wide[:, hq + hk:]) and out[0].data_ptr() == held.data_ptr()


def test_rotary_far_positions_and_its_gradient():
    W, g = _W(), rng_for(302, "far")
    freq = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    pos = np.array([0, 1, -1, 4095, 10**6 + 7, 2**31 - 1, -(2**31), 10**9])
    x, xv = _rows(g, (len(pos), 2, 64), "f32")
    y = host(W.rotary(x, to_dev(pos), to_dev(freq)))
    # 10^9 radians: fp64 keeps 2^-53 of them, 1e-7; the rest as above
    assert np.abs(y - R.rotary(xv, pos, freq, False, 1.0, False)).max() <= (10 * F32 + 2.0**31 * 2.0**-52) * 2 * np.abs(xv).max()
    # the gradient by differences of the formula, along random directions
    dy, dyv = _rows(g, xv.shape, "f32")
    dx = host(W.rotary(dy, to_dev(pos), to_dev(freq), factor=1.5, inverse=True))
    for _ in range(3):
        v, h = g.standard_normal(xv.shape), 1e-3
        num = ((R.rotary(xv + h * v, pos, freq, False, 1.5, False) - R.rotary(xv - h * v, pos, freq, False, 1.5, False)) * dyv).sum() / (2 * h)
        assert abs((dx * v).sum() - num) <= 1e-5 * np.abs(dx * v).sum()


def test_rotary_refusals_in_python():
    import torch

    W = _W()
    x, pos, f = torch.randn(4, 2, 64, device="cuda"), torch.arange(4, device="cuda"), torch.ones(32, device="cuda", dtype=torch.float64)
    for args in ((x, pos[:3], f), (x, pos.int(), f), (x, pos, f.float()), (x.half(), pos, f), (x.transpose(0, 1), pos, f),
                 (x[..., ::2], pos, f), (x.cpu(), pos, f), (x[0], pos, f), ((x, x, x), pos, f)):
        with pytest.raises((ValueError, TypeError)):
            W.rotary(*args)
    with pytest.raises(W.QwhaError):
        W.rotary(x, pos, torch.ones(33, device="cuda", dtype=torch.float64))  # rot 66 of 64
    with pytest.raises(W.QwhaError):
        W.rotary(x[1:], pos[1:], f, out=x[:3])
    assert W.rotary(x[:0], pos[:0], f).shape == (0, 2, 64)


# ---------------------------------------------------------------- attention


class Setup:
    """A pool, a table and queries of an attention call, on both sides."""

    def __init__(self, key, past, new, heads=2, grp=2, D=64, bits=4, bits_v=None, group=64, had_k=0, had_v=0, page_size=16,
                 dtype="bf16", tree=None, zero_top=None, size=1.0, room=0, group_v=None):
        W, g = _W(), rng_for(310, key)
        self.past, self.new, self.dtype, self.g = past, new, dtype, g
        bits_v, group_v = bits_v or bits, group_v or group
        self.table, n_pages = R.shuffled_table(g, [a + b for a, b in zip(past, new)], page_size)
        # a table of more room than is used: calls that are not known to be small have other kernels
        self.table = np.pad(self.table, ((0, 0), (0, max(0, room // page_size - self.table.shape[1]))), constant_values=-1)
        self.pk = R.random_pool(g, n_pages, page_size, heads, D, bits, group, zero_top)
        self.pv = R.random_pool(g, n_pages, page_size, heads, D, bits_v, group_v, zero_top)
        self.fmt, self.page_size, self.group_v = (bits, bits_v, group, had_k, had_v), page_size, group_v
        self.kv = (W.QCache(bits, group, had_k, *(to_dev(t) for t in self.pk)),
                   W.QCache(bits_v, group_v, had_v, *(to_dev(t) for t in self.pv)))
        self.q, self.qv = _rows(g, (sum(new), heads * grp, D), dtype, size)
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.tree = tree(g, new) if callable(tree) else tree
        self.scale = D**-0.5
        # calls of more than 8 rows to a cached head may round cached values (R.attention)
        rows = -(-sum(new) // len(new)) * grp
        self.cached = 2.0**-11 + 2.0**-21 if dtype == "bf16" and D % 32 == 0 and D <= 128 and group % 32 == group_v % 32 == 0 and rows > 8 else 0.0

    def run(self, **kw):
        import torch

        W = _W()
        self.lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        tree = None if self.tree is None else to_dev(self.tree)
        args = dict(tree=tree, lse=self.lse, scale=self.scale)
        args.update(kw)
        return W.cache_attention(self.kv, self.q, to_dev(self.table), to_dev(self.starts), to_dev(np.array(self.past, np.int64)),
                                 **args)

    def ref(self):
        bits, bits_v, group, had_k, had_v = self.fmt
        eps = 2.0**-11 if self.dtype == "bf16" else 2.0**-21
        return R.attention(self.qv, R.dense_pool(self.pk, bits, group), R.dense_pool(self.pv, bits_v, self.group_v),
                           R.largest_steps(self.pv, bits_v, self.group_v), had_k, had_v, self.table, self.page_size, self.past, self.new, self.tree, self.scale, eps, self.cached)

    def check(self, out=None):
        got = host(self.run() if out is None else out)
        out, lse, tol, lse_tol = self.ref()
        err = np.abs(got - out) - half_step(self.dtype) * np.abs(out)
        worst = np.unravel_index(np.argmax(err - tol), err.shape) if err.size else ()
        assert np.all(err <= tol), (worst, got[worst], out[worst], tol[worst])
        l = host(self.lse)
        assert np.array_equal(np.isneginf(l), np.isneginf(lse))
        ok = np.isfinite(lse)
        assert np.all(np.abs(l[ok] - lse[ok]) <= lse_tol[ok])
        _W().check_stream_status()
        return got


def random_trees(g, new):
    """Masks of random trees (ancestors and itself), some nodes with no mask at all."""
    out = []
    for m in new:
        mask = []
        for j in range(m):
            p = int(g.integers(-1, j)) if j else -1
            mask.append((mask[p] if p >= 0 else 0) | 1 << j)
        out += [0 if g.random() < 0.15 else v for v in mask]
    return np.array([v - 2**64 if v >= 2**63 else v for v in out], np.int64)


FORMATS = [(64, 4, 64, 0), (64, 2, 32, 64), (80, 3, 40, 16), (96, 4, 96, 32), (128, 4, 128, 128), (128, 8, 64, 128),
           (128, 3, 128, 0), (128, 2, 32, 64), (256, 4, 64, 256), (256, 8, 256, 0), (8, 4, 8, 8), (40, 4, 8, 0), (128, 4, 8, 2),
           (128, 4, 16, 64), (256, 2, 128, 128), (24, 8, 24, 8), (128, 3, 32, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,bits,group,had", FORMATS)
def test_attention_formats(D, bits, group, had, dtype):
    """Every format, one token each and small trees, over lengths around the borders of tiles."""
    key = f"{D}-{bits}-{group}-{had}-{dtype}"
    Setup("one" + key, [0, 1, 15, 16, 63, 64, 65, 200], [1] * 8, D=D, bits=bits, group=group, had_k=had, had_v=had,
          dtype=dtype).check()
    for room in (0, 1 << 20):
        Setup("tree" + key, [0, 33, 128], [3, 7, 1], D=D, bits=bits, group=group, had_k=0, had_v=had, dtype=dtype,
              tree=random_trees, grp=3, room=room).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,grp,new", [(1, 1, 1), (1, 9, 1), (3, 1, 5), (2, 7, 3), (8, 4, 2), (1, 40, 2), (5, 4, 9),
                                           (2, 4, 33), (1, 16, 17), (2, 3, 64), (9, 2, 1), (12, 5, 4)])
def test_attention_heads_and_rows(heads, grp, new, dtype):
    for tree in (None, random_trees):
        for room in (0, 1 << 20):
            Setup(f"{heads}-{grp}-{new}-{dtype}-{tree is None}", [17, 0, 90], [new, max(1, new - 2), new], heads=heads, grp=grp,
                  D=128, group=128, had_k=128, had_v=128, dtype=dtype, tree=tree, room=room).check()


@pytest.mark.parametrize("page_size", [1, 3, 16, 100])
@pytest.mark.parametrize("D,group", [(128, 128), (64, 32), (40, 8)])
def test_attention_chunks_of_prompts(page_size, D, group):
    """Causal chunks longer than a tile of rows, ragged, with and without a past, and a sequence without tokens."""
    for dtype in ("bf16", "f32"):
        s = Setup(f"chunk{page_size}-{D}-{dtype}", [0, 5, 131, 7], [70, 150, 33, 0], D=D, group=group, had_k=8, had_v=0,
                  page_size=page_size, dtype=dtype)
        s.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,group,group_v,bits,bits_v", [(128, 64, 128, 4, 4), (128, 128, 32, 4, 2), (128, 8, 64, 3, 8), (64, 64, 16, 2, 4),
                                                         (256, 256, 32, 4, 4), (80, 40, 80, 4, 3), (24, 24, 8, 8, 4), (96, 32, 96, 4, 4)])
def test_attention_groups_of_different_sizes(D, group, group_v, bits, bits_v, dtype):
    """Keys and values in groups of their own, one token each, small trees, chunks; one cached head and several."""
    fmt = dict(D=D, group=group, group_v=group_v, bits=bits, bits_v=bits_v, dtype=dtype, had_v=8)
    key = f"groups{D}-{group}-{group_v}-{dtype}"
    Setup("one" + key, [0, 15, 64, 200], [1] * 4, heads=1, **fmt).check()
    Setup("three" + key, [700, 3], [1, 1], heads=3, grp=5, **fmt).check()
    for room in (0, 1 << 20):
        Setup("tree" + key, [0, 33, 128], [3, 7, 1], heads=5, grp=3, tree=random_trees, room=room, **fmt).check()
    Setup("chunk" + key, [0, 131], [70, 33], heads=2, grp=2, **fmt).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,bits,bits_v,group", [(80, 4, 4, 40), (80, 2, 8, 40), (64, 3, 3, 64), (64, 3, 2, 32), (96, 2, 2, 96), (96, 3, 3, 96),
                                                 (80, 3, 2, 40), (24, 4, 8, 24), (8, 8, 8, 8), (32, 2, 2, 32), (16, 4, 2, 16)])
def test_attention_heads_that_share_pieces_of_16_bytes(D, bits, bits_v, group, dtype):
    """All heads' codes of a token are whole 16-byte pieces, one head's are not."""
    for heads in (1, 2, 3, 4, 8, 16):
        Setup(f"pieces{heads}-{D}-{bits}-{bits_v}-{dtype}", [33, 0, 400], [1, 2, 1], heads=heads, D=D, bits=bits, bits_v=bits_v, group=group,
              dtype=dtype, room=1 << 20).check()


def test_attention_many_and_long_sequences():
    """More sequences than a CTA has threads; one long context cut between all CTAs beside short ones."""
    g = rng_for(311, "many")
    past = [int(v) for v in g.integers(0, 40, 700)]
    Setup("many", past, [1] * 700, heads=1, grp=4, D=64).check()
    Setup("long", [30000, 3, 9000], [1, 2, 1], heads=1, grp=2, D=64, page_size=64).check()
    Setup("longtree", [9000, 0, 40], [64, 3, 1], heads=1, grp=2, D=128, group=128, tree=random_trees).check()


def test_attention_peaked_and_flat_scores():
    """Scores of several hundred, where one token takes all; all scores alike; the largest score at either end."""
    s = Setup("peaked", [300], [2], D=64, size=60.0, dtype="f32")
    s.check()
    s = Setup("flat", [500], [2], D=64, dtype="bf16")
    s.scale = 0.0
    s.check()
    s = Setup("negative", [100, 3], [1, 1], D=128, group=64, dtype="f32", size=8.0)
    s.scale = -0.3
    s.check()
    for at in (0, 77, 200):
        s = Setup(f"end{at}", [200], [1], D=64, dtype="bf16", size=4.0)
        codes, sc, z = s.pk
        slot = s.table[0, at // 16] * 16 + at % 16
        sc.reshape(-1, *sc.shape[2:])[slot] *= 20.0
        s.kv[0].scales.copy_(to_dev(sc))
        s.check()


def test_attention_zero_points_of_a_whole_byte_and_large_scales():
    for bits in (2, 4, 8):
        Setup(f"zeros{bits}", [50, 3], [1, 4], D=64, bits=bits, group=32, zero_top=255).check()
    s = Setup("scales", [60], [3], D=128, group=64, dtype="bf16")
    for pool, cache in zip((s.pk, s.pv), s.kv):  # scales over many powers of two in the values, small ones in the keys
        pool[1][...] *= (2.0 ** s.g.integers(-60, 50, pool[1].shape)).astype(np.float32) if cache is s.kv[1] else 2.0**-20
        cache.scales.copy_(to_dev(pool[1]))
    s.check()


def test_attention_large_values_on_zero_weights():
    """A query channel a thousand times the others meets codes equal to their zero point: nothing is left of it."""
    s = Setup("spike", [100], [1], D=64, bits=4, group=64, dtype="f32")
    s.qv[..., 5] = 3000.0
    s.q.copy_(to_dev(s.qv.astype(np.float32)))
    codes, sc, z = s.pk
    flat = codes.reshape(-1, codes.shape[-1])
    zz = z.reshape(-1)
    flat[:, 2] = (flat[:, 2] & 0x0F) | ((zz & 15) << 4)  # code 5 = zero point
    s.kv[0].codes.copy_(to_dev(codes))
    # the bound of R.attention, which takes |k q| and is not widened by the spike: k is 0 there
    s.check()


def test_attention_bad_groups_in_masked_places():
    """NaN groups in tokens that are not seen (behind the end, on other pages, outside a node's tree) have no effect; one
    that is seen makes its rows NaN and no others."""
    import torch

    for D, group in ((128, 64), (40, 8)):
        s = Setup(f"nan{D}", [20, 37, 0], [4, 3, 2], D=D, group=group, tree=np.array([1, 2, 5, 8, 1, 3, 7, 0, 0], np.int64))
        clean = s.check()
        assert np.all(clean[7:] == 0)  # rows that see nothing
        seen = set()
        for b, (p, m) in enumerate(zip(s.past, s.new)):
            for t in range(p + m):
                u = t - p
                at = s.starts[b]
                if u < 0 or any(int(s.tree[at + j]) >> u & 1 for j in range(m)):
                    seen.add(int(s.table[b, t // 16]) * 16 + t % 16)
        n_slots = s.kv[0].n_slots
        for c in s.kv:
            flat = c.scales.view(n_slots, -1)
            for slot in range(n_slots):
                if slot not in seen:
                    flat[slot] = float("nan")
        assert np.array_equal(host(s.run()), clean)
        # node 2 of sequence 0 (mask 5) and nobody else sees node 2
        slot = int(s.table[0, 22 // 16]) * 16 + 22 % 16
        for c in s.kv:
            keep = c.scales.view(n_slots, -1)[slot].clone()
            c.scales.view(n_slots, -1)[slot] = float("nan")
            got = host(s.run())
            assert np.all(np.isnan(got[2])) and np.array_equal(np.delete(got, 2, 0), np.delete(clean, 2, 0))
            c.scales.view(n_slots, -1)[slot] = keep
        torch.cuda.synchronize()


# Calls of many rows to a cached head, whose cached values are rounded to f16 with their scales.
MANY = [(32, 4, 4, 32, 0, 0), (64, 2, 3, 64, 64, 0), (64, 3, 2, 32, 0, 64), (96, 4, 8, 32, 32, 32), (96, 8, 4, 96, 0, 2),
        (128, 4, 4, 128, 128, 128), (128, 4, 4, 64, 64, 0), (128, 8, 8, 32, 8, 128), (128, 3, 3, 64, 128, 64), (128, 2, 2, 128, 0, 32)]


def many_rows(*args, **kw):
    s = Setup(*args, **kw)
    assert s.cached
    return s


@pytest.mark.parametrize("D,bits,bits_v,group,had_k,had_v", MANY)
def test_attention_of_many_rows(D, bits, bits_v, group, had_k, had_v):
    """Chunks and trees of more than 32 rows to a cached head: every width, and other widths for the values; pasts around
    the borders of tiles of tokens; sequences of one row or none beside them; 200 rows to a token."""
    fmt = dict(D=D, bits=bits, bits_v=bits_v, group=group, had_k=had_k, had_v=had_v)
    key = "-".join(map(str, fmt.values()))
    many_rows("a" + key, [0, 127, 128, 129, 300, 1], [64, 1, 40, 33, 64, 0], grp=4, tree=random_trees, **fmt).check()
    many_rows("b" + key, [0, 1000, 64], [300, 130, 1], grp=3, heads=1, page_size=100, **fmt).check()
    many_rows("c" + key, [5, 140], [3, 1], grp=200, heads=1, **fmt).check()


@pytest.mark.parametrize("past,new,heads,grp", [([100] * 60, [17] * 60, 8, 2), ([0] * 30, [130] * 30, 3, 5), ([3000, 0, 10], [50, 1, 300], 2, 4),
                                                ([5000], [64], 1, 4)])
def test_attention_of_many_rows_cut_between_ctas(past, new, heads, grp):
    """Several tiles to a CTA, and a tile to all of them; again with the same bits."""
    s = many_rows(f"cut{past[0]}-{grp}", past, new, heads=heads, grp=grp, D=128, group=128, had_k=128, had_v=128)
    got = s.check()
    for _ in range(3):
        assert np.array_equal(host(s.run()), got)


@pytest.mark.parametrize("past,new,heads,grp,tree", [([13000, 9000], [126, 117], 8, 3, False), ([3000] * 18, [46, 43, 40] * 6, 4, 7, True),
                                                     ([900, 300, 800] * 5, [161, 90, 33] * 5, 2, 8, False), ([7000, 5000], [513, 200], 2, 8, False)])
def test_attention_of_many_rows_whose_last_tiles_are_short(past, new, heads, grp, tree):
    """Segments with rows in one of the two tiles between segments with rows in both, over many tokens; the same bits again
    and again, from the first run on."""
    s = many_rows(f"short{past[0]}-{grp}", past, new, heads=heads, grp=grp, D=64, group=64, had_k=64, had_v=64, page_size=64,
                  tree=random_trees if tree else None)
    got = s.check()
    for _ in range(8):
        assert np.array_equal(host(s.run()), got)


def test_attention_of_many_rows_scores_and_scales():
    """Peaked and flat scores, queries of zeros, scales over many powers of two, the largest key or value last."""
    s = many_rows("peaked", [300], [40], D=64, size=60.0)
    s.check()
    s = many_rows("flat", [500], [40], D=64)
    s.scale = 0.0
    s.check()
    s = many_rows("negative", [100, 3], [40, 40], D=128, group=64, size=8.0)
    s.scale = -0.3
    s.check()
    s = many_rows("nothing", [100], [64], D=128, group=128)
    s.qv[...] = 0.0
    s.q.zero_()
    s.check()
    for which in (0, 1):
        for at in (0, 150, 299):
            s = many_rows(f"end{which}{at}", [300], [40], D=64, size=2.0)
            slot = int(s.table[0, at // 16]) * 16 + at % 16
            sc = (s.pk, s.pv)[which][1]
            sc.reshape(-1, *sc.shape[2:])[slot] *= 20.0
            s.kv[which].scales.copy_(to_dev(sc))
            s.check()


@pytest.mark.parametrize("D,group", [(64, 32), (128, 32), (128, 64), (128, 128)])
def test_attention_of_many_rows_scales_of_many_powers_of_two(D, group):
    """Values whose groups and tokens lie many powers of two apart, each group to its own measure."""
    s = many_rows(f"powers{D}{group}", [260, 60], [40, 30], D=D, group=group)
    for pool, cache in zip((s.pk, s.pv), s.kv):
        if cache is s.kv[1]:
            pool[1][...] *= (2.0 ** s.g.integers(-50, 40, (1, 1, 1, D // group))).astype(np.float32)
            pool[1][...] *= (2.0 ** s.g.integers(-5, 5, pool[1].shape)).astype(np.float32)
        else:
            pool[1][...] *= 2.0**-20
        cache.scales.copy_(to_dev(pool[1]))
    s.check()


def poison(s, where, factor, which):
    """Scales of token `where` (sequence, token) times factor."""
    b, t = where
    slot = int(s.table[b, t // s.page_size]) * s.page_size + t % s.page_size
    for i, pool in enumerate((s.pk, s.pv)):
        if i in which:
            sc = pool[1].reshape(-1, *pool[1].shape[2:])
            sc[slot] *= np.float32(factor)
            s.kv[i].scales.copy_(to_dev(pool[1]))


@pytest.mark.parametrize("dtype,grp,new", [("bf16", 4, 40), ("bf16", 2, 8), ("f32", 2, 8), ("bf16", 2, 2), ("f32", 1, 3), ("f32", 4, 40)])
@pytest.mark.parametrize("factor", [2.0**9, 2.0**13, 2.0**20, 1e30])
@pytest.mark.parametrize("which", [(0,), (1,), (0, 1)])
def test_attention_scales_that_only_some_rows_see(dtype, grp, new, factor, which):
    """A token of far larger scales than the others takes nothing from the rows that do not see it: behind them in a chunk,
    or on another branch of a tree; with and without tokens that all rows see."""
    for past, room in ((200, 0), (0, 0), (200, 1 << 20), (0, 1 << 20)):
        for tree in (None, random_trees):
            for D, group in ((128, 64), (64, 64), (40, 8)):
                s = Setup(f"wide{dtype}{grp}{new}{factor}{which}{past}{D}", [past, 30], [new, new], heads=2, grp=grp, D=D, group=group, dtype=dtype,
                          room=room, tree=tree, size=0.5 if 0 in which else 1.0)
                poison(s, (0, past + new - 1), factor, which)
                s.check()


def test_attention_of_many_rows_scales_that_only_some_rows_see_in_whole_tiles():
    """The same where CTAs have several tiles each, none cut; lse too (checked with the outputs)."""
    s = many_rows("whole", [100] * 200, [24] * 200, heads=4, grp=2, D=128, group=128, had_v=128)
    for b in (0, 77, 199):
        poison(s, (b, 110), 1e25, (0, 1))
    s.check()


def test_attention_of_many_rows_bad_groups_in_masked_places():
    """NaN and infinite groups in tokens that no row sees, or that some rows see."""
    for D, group in ((128, 64), (64, 64), (128, 32)):
        tree = np.zeros(64, np.int64)
        for j in range(64):
            tree[j] = 0 if j in (7, 50) else np.int64((1 << (j // 8 * 8)) | (1 << j) if j < 63 else -2**63)
        s = many_rows(f"nan{D}{group}", [150], [64], D=D, group=group, tree=tree, grp=4)
        clean = s.check()
        n_slots = s.kv[0].n_slots
        for value in (float("nan"), float("inf"), -float("inf")):
            keep = [c.scales.clone() for c in s.kv]
            seen = set()
            for t in range(214):
                if t < 150 or any(int(m) >> (t - 150) & 1 for m in tree):
                    seen.add(int(s.table[0, t // 16]) * 16 + t % 16)
            for c in s.kv:
                flat = c.scales.view(n_slots, -1)
                for slot in range(n_slots):
                    if slot not in seen:
                        flat[slot] = value
            assert np.array_equal(host(s.run()), clean)
            for at, rows in ((150 + 13, [13]), (150 + 16, [j for j in range(16, 24)])):  # a leaf; the root of a branch
                slot = int(s.table[0, at // 16]) * 16 + at % 16
                rows = [j for j in rows if j not in (7, 50)]
                for c in s.kv:
                    old = c.scales.view(n_slots, -1)[slot].clone()
                    c.scales.view(n_slots, -1)[slot] = value
                    got = host(s.run())
                    assert np.array_equal(np.delete(got, rows, 0), np.delete(clean, rows, 0))
                    if value != value:
                        assert np.all(np.isnan(got[rows]))
                    elif c is s.kv[1]:
                        assert not np.any(np.isfinite(got[rows]))
                    c.scales.view(n_slots, -1)[slot] = old
            for c, k in zip(s.kv, keep):
                c.scales.copy_(k)


def test_attention_of_many_rows_pages_and_rows_behind():
    """Pages that are none, rows behind the last sequence, and keys and values in groups of different sizes."""
    import torch

    W = _W()
    s = many_rows("bad", [200, 40], [40, 40], D=128, group=128, grp=2)
    q = torch.cat((s.q, s.q[:2]))
    out = torch.full_like(q, 3.0)
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    W.cache_attention(s.kv, q, to_dev(s.table), to_dev(s.starts), to_dev(np.array(s.past)), out=out, lse=lse)
    assert torch.all(out[80:] == 3.0) and torch.all(lse[80:] == 5.0)
    for bad in (-1, int(s.kv[0].scales.shape[0])):
        keep = s.table.copy()
        s.table[0, 3] = bad
        got = s.run()
        with pytest.raises(W.QwhaError, match="page"):
            W.check_stream_status()
        s.table[0, 3] = -1
        s.check(got)
        s.table = keep
    other = R.random_pool(s.g, s.kv[0].scales.shape[0], 16, 2, 128, 4, 64)
    kv = (s.kv[0], W.QCache(4, 64, 0, *(to_dev(t) for t in other)))
    got = host(W.cache_attention(kv, s.q, to_dev(s.table), to_dev(s.starts), to_dev(np.array(s.past)), scale=s.scale))
    want, _, tol, _ = R.attention(s.qv, R.dense_pool(s.pk, 4, 128), R.dense_pool(other, 4, 64), R.largest_steps(other, 4, 64), 0, 0, s.table,
                                  16, s.past, s.new, None, s.scale, 2.0**-11, 2.0**-11 + 2.0**-21)
    assert np.all(np.abs(got - want) <= tol + half_step("bf16") * np.abs(want))


def test_attention_rows_behind_the_last_sequence_and_bad_pages():
    import torch

    W = _W()
    for D, group in ((128, 128), (40, 8)):
        s = Setup(f"bad{D}", [20, 40], [2, 1], D=D, group=group)
        q = torch.cat((s.q, s.q[:2]))
        out = torch.full_like(q, 3.0)
        lse = torch.full(q.shape[:2], 5.0, device="cuda")
        W.cache_attention(s.kv, q, to_dev(s.table), to_dev(s.starts), to_dev(np.array(s.past)), out=out, lse=lse)
        assert torch.all(out[3:] == 3.0) and torch.all(lse[3:] == 5.0)
        assert torch.equal(out[:3], s.run())
        W.check_stream_status()
        for bad in (-1, int(s.kv[0].scales.shape[0])):
            keep = s.table.copy()
            s.table[1, 1] = bad  # tokens 16..31 of sequence 1
            got = s.run()
            with pytest.raises(W.QwhaError, match="page"):
                W.check_stream_status()
            s.table[1, 1] = -1
            s.lse = s.lse
            s.check(got)
            s.table = keep
        with pytest.raises(W.QwhaError):  # the table ends before the sequence does
            W.cache_attention(s.kv, s.q, to_dev(np.ascontiguousarray(s.table[:, :2])), to_dev(s.starts), to_dev(np.array(s.past)))
            W.check_stream_status()
        # lengths that make no sense are cut, not followed
        for past, starts in (([-5, 1 << 40], [0, 2, 3]), ([20, 40], [0, 1 << 40, 3]), ([20, 40], [-3, 2, -7])):
            W.cache_attention(s.kv, s.q, to_dev(s.table), to_dev(np.array(starts)), to_dev(np.array(past)))
        try:
            W.check_stream_status()
        except W.QwhaError as e:
            assert e.status == 1


def test_attention_strided_queries_streams_graphs_and_repeats():
    """Queries within a fused projection; another stream; two captured graphs that share a workspace; repeated bits."""
    import torch

    W = _W()
    s = Setup("graph", [700, 30, 9], [3, 1, 2], heads=2, grp=4, D=128, group=128, had_k=128, had_v=128)
    want = s.run()
    for _ in range(3):
        assert torch.equal(s.run(), want)
    wide = torch.zeros(s.q.shape[0], 12, 128, device="cuda", dtype=s.q.dtype)
    wide[:, 2:10] = s.q
    table, starts, past = to_dev(s.table), to_dev(s.starts), to_dev(np.array(s.past))
    assert torch.equal(W.cache_attention(s.kv, wide[:, 2:10], table, starts, past, scale=s.scale), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = W.cache_attention(s.kv, s.q, table, starts, past, scale=s.scale)
    side.synchronize()
    assert torch.equal(other, want)
    ws = torch.empty(W.workspace_size(W.api.OP_ATTENTION, 8, 128, 2, 6, 1), dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(want) for _ in range(2)], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            W.cache_attention(s.kv, s.q, table, starts, past, scale=s.scale, out=o, ws=ws)
        graphs.append(g)
    ws.fill_(255)
    for _ in range(3):
        for g in graphs:
            g.replay()
    assert all(torch.equal(o, want) for o in outs)
    past.copy_(to_dev(np.array([90, 2, 9])))  # a captured call follows the lengths on the device
    graphs[0].replay()
    s.past = [90, 2, 9]
    assert torch.equal(outs[0], s.run())
    W.check_stream_status()


def test_attention_refusals_in_python():
    import torch

    W = _W()
    s = Setup("refuse", [20], [2])
    table, starts, past = to_dev(s.table), to_dev(s.starts), to_dev(np.array(s.past))
    for args in ((s.kv, s.q[:, :3], table, starts, past), (s.kv, s.q[..., :32], table, starts, past),
                 (s.kv, s.q, table.long(), starts, past), (s.kv, s.q, table, starts[:1], past),
                 (s.kv, s.q, table, starts, past.int()), (s.kv, s.q.half(), table, starts, past),
                 (s.kv, s.q.cpu(), table, starts, past)):
        with pytest.raises((ValueError, TypeError, W.QwhaError)):
            W.cache_attention(*args)
    with pytest.raises(ValueError):
        W.cache_attention(s.kv, s.q, table, starts, past, tree=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(W.QwhaError):
        W.cache_attention(s.kv, s.q, table, starts, past, out=s.q)
    assert W.cache_attention(s.kv, s.q[:0], table, starts, past).shape[0] == 0
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    W.cache_attention(s.kv, s.q, table[:0], starts[:1], none)


# ---------------------------------------------------------------- page table


def _table(t):
    W = _W()
    return W.PageTable(t.ps, to_dev(t.refs), to_dev(t.pages), to_dev(t.held))


def _same(t, d):
    assert np.array_equal(_ints(d.refs), t.refs) and np.array_equal(_ints(d.pages), t.pages) and np.array_equal(_ints(d.held), t.held)


@pytest.mark.parametrize("n_seqs,n_pages,max_pages,page_size", [(1, 1, 1, 1), (3, 10, 4, 16), (40, 200, 12, 5), (600, 3000, 9, 16),
                                                                (2100, 9000, 7, 16), (2, 70000, 40000, 1), (33, 4097, 64, 3)])
def test_page_table_against_the_plain_one(n_seqs, n_pages, max_pages, page_size):
    """Random growth, shrinking and forks, pages running out among them."""
    import torch

    W, g = _W(), rng_for(320, str(n_seqs), str(n_pages))
    t = R.Table(np.zeros(n_pages, np.int32), np.full((n_seqs, max_pages), -1, np.int32), np.zeros(n_seqs, np.int64), page_size)
    d = _table(t)
    room = max_pages * page_size
    share = max(1, n_pages * page_size // n_seqs)
    for step in range(8):
        want = g.integers(0, min(room, 2 * share) + 1, n_seqs)
        want[g.random(n_seqs) < 0.3] = -1
        want[g.random(n_seqs) < 0.2] = 0
        assert not t.resize(want)
        held = W.pages_resize(d, to_dev(want))
        assert held is d.held
        _same(t, d)
        m = max(1, n_seqs // 3)
        empty = np.flatnonzero(t.held == 0)
        dst = g.permutation(empty)[:m]
        src = g.integers(-1, n_seqs, len(dst))
        if len(dst):
            origin, fresh, bad = t.fork(src, dst)
            a, b = W.pages_fork(d, to_dev(src), to_dev(dst))
            assert np.array_equal(_ints(a), origin) and np.array_equal(_ints(b), fresh)
            _same(t, d)
            assert not bad
    W.check_stream_status()
    t.resize(np.zeros(n_seqs, np.int64))
    W.pages_resize(d, torch.zeros(n_seqs, dtype=torch.int64, device="cuda"))
    _same(t, d)
    assert not t.refs.any()


def test_page_table_refused_rows():
    W = _W()
    t = R.Table(np.zeros(20, np.int32), np.full((6, 3), -1, np.int32), np.zeros(6, np.int64), 4)
    d = _table(t)
    want = np.array([5, 13, -2, 1, 0, 12])  # 13 is above 3 pages of 4
    assert t.resize(want)
    W.pages_resize(d, to_dev(want))
    _same(t, d)
    with pytest.raises(W.QwhaError, match="page table"):
        W.check_stream_status()
    src, dst = np.array([0, 0, 9, 0, 3, 0, 5, -1]), np.array([1, 1, 2, 5, 7, -1, 4, 99])
    origin, fresh, bad = t.fork(src, dst)
    a, b = W.pages_fork(d, to_dev(src), to_dev(dst))
    assert bad and np.array_equal(_ints(a), origin) and np.array_equal(_ints(b), fresh)
    _same(t, d)
    with pytest.raises(W.QwhaError, match="page table"):
        W.check_stream_status()
    # rows that contradict the table: reported, nothing outside is touched
    d.held[0], d.held[3] = 1000, -4
    d.pages[5, 0] = 77
    W.pages_resize(d, to_dev(np.array([0, -1, -1, 8, -1, 0])))
    with pytest.raises(W.QwhaError, match="page table"):
        W.check_stream_status()
    assert int(d.held[0]) == 1000 and int(d.held[3]) == -4 and int(d.refs.min()) >= 0


def test_page_table_in_a_graph():
    import torch

    W = _W()
    d = W.page_table(64, 16, 4, 8)
    want, back = torch.tensor([20, 1, 0, 128], device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    ws = torch.empty(W.workspace_size(W.api.OP_PAGES, 4, 1, 64, 0, 0), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        W.pages_resize(d, want, ws=ws)
    for _ in range(2):
        g.replay()
        assert d.held.tolist() == [20, 1, 0, 128] and d.pages[0, :3].tolist() == [0, 1, -1] and int(d.refs.sum()) == 11
        W.pages_resize(d, back)
        assert int(d.refs.sum()) == 0 and int(d.pages.max()) == -1
    W.check_stream_status()


# ---------------------------------------------------------------- moves


@pytest.mark.parametrize("heads,D,bits,group,page_size", [(2, 64, 4, 64, 16), (1, 8, 3, 8, 1), (3, 24, 3, 8, 5), (8, 128, 8, 32, 64),
                                                          (1, 80, 2, 40, 7), (5, 256, 4, 256, 16)])
def test_copy_pages_and_compact(heads, D, bits, group, page_size):
    import torch

    W, g = _W(), rng_for(330, str(heads), str(D), str(bits))
    lens = [page_size * 3 + 2, 1, 40, 300]
    table, n_pages = R.shuffled_table(g, lens, page_size, spare=9)
    pools = [R.random_pool(g, n_pages, page_size, heads, D, b, group) for b in (bits, 4)]
    caches = tuple(W.QCache(b, group, 0, *(to_dev(t) for t in p)) for b, p in zip((bits, 4), pools))
    order = g.permutation(n_pages).astype(np.int32)
    k = n_pages // 2
    src, dst = order[:k].copy(), order[k:2 * k].copy()
    src[0] = -1
    if k > 2:
        dst[1] = -1
    W.cache_copy_pages(caches, to_dev(src), to_dev(dst))
    for p in pools:
        for a, b in zip(src, dst):
            if a >= 0 and b >= 0:
                for t in p:
                    t[b] = t[a]
    first = np.array([3, 0, 0, 11], np.int64)
    keep = np.full((4, 250), -1, np.int32)
    for b, n in enumerate((2, 1, 25, 200)):
        keep[b, :n] = np.sort(g.choice(lens[b] - first[b], n, replace=False))
    keep[2, 30] = 5  # behind the -1 that ends the row: not read
    W.cache_compact(caches, to_dev(table), to_dev(first), to_dev(keep))
    for p in pools:
        for t in p:
            flat = t.reshape(-1, *t.shape[2:])
            old = flat.copy()
            for b in range(4):
                for i, u in enumerate(keep[b]):
                    if u < 0:
                        break
                    a, c = first[b] + u, first[b] + i
                    flat[table[b, c // page_size] * page_size + c % page_size] = old[table[b, a // page_size] * page_size + a % page_size]
    for p, c in zip(pools, caches):
        for want, got in zip(p, (c.codes, c.scales, c.zeros)):
            assert np.array_equal(_ints(got), want)
    W.check_stream_status()
    before = [t.clone() for c in caches for t in (c.codes, c.scales, c.zeros)]
    # pages outside: reported, nothing moves; a row that stops ascending moves up to there
    W.cache_copy_pages(caches, to_dev(np.array([n_pages, 0], np.int32)), to_dev(np.array([0, -2], np.int32)))
    with pytest.raises(W.QwhaError, match="page"):
        W.check_stream_status()
    W.cache_compact(caches[0], to_dev(table[:1]), to_dev(np.array([0])), to_dev(np.array([[0, 1, 1, 2]], np.int32)))
    with pytest.raises(W.QwhaError, match="ascend"):
        W.check_stream_status()
    W.cache_compact(caches[0], to_dev(table[:1]), to_dev(np.array([0])), to_dev(np.array([[100000]], np.int32)))
    with pytest.raises(W.QwhaError, match="page"):
        W.check_stream_status()
    for a, b in zip(before, [t for c in caches for t in (c.codes, c.scales, c.zeros)]):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_step_of_speculative_answering(dtype):
    """Prompts are appended and attended, one is forked, both draft trees, the accepted nodes move up and the rest is given
    back; then a plain step. Each step's attention against the formulas on what the caches hold by the plain quantizer."""
    import torch

    W, g = _W(), rng_for(340, dtype)
    heads, grp, D, ps, bits = 2, 2, 64, 8, 4
    t = W.page_table(40, ps, 4, 12)
    caches = tuple(W.cache_alloc(40, ps, heads, D, bits=bits, group=32, had_block=64) for _ in range(2))
    freq, factor = W.rotary_frequencies(D, scaling="ramp", factor=2.0, trained=64)
    fv = freq.cpu().numpy()
    tokens = {0: [], 1: [], 2: []}  # per sequence: (stored key, stored value) rows in the cache's frame

    def step(counts, depth_of=None, tree=None):
        """Append counts[b] tokens to each sequence and attend."""
        past = t.held.clone()
        W.pages_resize(t, past + to_dev(np.array(counts + [0] * (4 - len(counts)))))
        n = sum(counts)
        x, xv = _rows(g, (n, heads * (grp + 2), D), dtype)
        pos, slots = [], []
        table, pv = _ints(t.pages), _ints(past)
        for b, m in enumerate(counts):
            for j in range(m):
                pos.append(pv[b] + (depth_of[b][j] if depth_of else j))
                at = pv[b] + j
                slots.append(table[b, at // ps] * ps + at % ps)
        pos, slots = np.array(pos, np.int64), np.array(slots, np.int64)
        q, k = W.rotary((x[:, :heads * grp], x[:, heads * grp:heads * (grp + 1)]), to_dev(pos), freq, factor=factor)
        v = x[:, heads * (grp + 1):].contiguous()
        W.cache_write(caches, (k, v), to_dev(slots))
        starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
        lse = torch.empty(n, heads * grp, device="cuda")
        out = W.cache_attention(caches, q, t.pages[:len(counts)].contiguous(), to_dev(starts), past[:len(counts)].contiguous(),
                                tree=None if tree is None else to_dev(tree), lse=lse)
        # rotary's result is checked above; what it gave is what was written
        stored = []
        for rows in (host(k), host(v)):
            c, s, z = quantize(rows.astype(np.float32), bits, 32, 64, dtype)
            stored.append(values(pack(c, bits), s, z, bits, 32))
        stored.append(np.repeat(np.abs(s), 32, -1) * (2.0**bits - 1))
        kd, vd, sd = [], [], []
        for b, m in enumerate(counts):
            for j in range(m):
                tokens[b].append(tuple(part[starts[b] + j] for part in stored))
            for part, held in enumerate((kd, vd, sd)):
                held.append([r[part] for r in tokens[b]])
        flat = lambda l: np.array([r for s in l for r in s])  # noqa: E731
        lens = [len(s) for s in kd]
        order = np.zeros((len(counts), max(lens)), np.int64)  # page size 1: row after row
        at = 0
        for b, m in enumerate(lens):
            order[b, :m] = np.arange(at, at + m)
            at += m
        ref, _, tol, _ = R.attention(host(q), flat(kd), flat(vd), flat(sd), 64, 64, order, 1, [int(p) for p in pv[:len(counts)]], counts,
                                     tree, D**-0.5, 2.0**-11 if dtype == "bf16" else 2.0**-21)
        assert np.all(np.abs(host(out) - ref) <= tol + half_step(dtype) * np.abs(ref))

    step([19, 5])
    a, b = W.pages_fork(t, to_dev(np.array([0])), to_dev(np.array([2])))
    W.cache_copy_pages(caches, a, b)
    tokens[2] = list(tokens[0])
    parents = [[-1, 0, 0, 1, 2, 4], [-1, 0, 1], [-1, -1, 0, 2]]
    masks, depth = [], []
    for p in parents:
        mm, dd = [], []
        for j, u in enumerate(p):
            mm.append((mm[u] if u >= 0 else 0) | 1 << j)
            dd.append(dd[u] + 1 if u >= 0 else 0)
        masks += mm
        depth.append(dd)
    first = t.held.clone()
    step([6, 3, 4], depth, np.array(masks, np.int64))
    accepted = [[0, 2, 4], [0], [0, 2, 3]]  # paths of the trees
    keep = np.full((4, 6), -1, np.int32)
    for s, path in enumerate(accepted):
        keep[s, :len(path)] = path
        base = int(first[s])
        tokens[s] = tokens[s][:base] + [tokens[s][base + u] for u in path]
    W.cache_compact(caches, t.pages, first, to_dev(keep))
    W.pages_resize(t, first + to_dev(np.array([3, 1, 3, 0])))
    assert t.held.tolist() == [22, 6, 22, 0]
    step([1, 1, 1])
    step([2, 1, 3])
    W.pages_resize(t, torch.zeros_like(t.held))
    assert int(t.refs.sum()) == 0
    W.check_stream_status()
