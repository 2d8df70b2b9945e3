"""Plain statements (numpy, 64 bits) of the operators around the cache: rotary positions, attention, page table, moves."""

import functools

import numpy as np

from _serving import unpack


def random_pool(g, n_pages, page_size, heads, head_dim, bits, group, zero_top=None):
    """Any codes, scales of both signs, zero points up to zero_top."""
    rows = (n_pages, page_size, heads)
    codes = g.integers(0, 256, rows + (head_dim * bits // 8,)).astype(np.uint8)
    top = 2**bits - 1
    s = (g.choice([-1.0, 1.0], rows + (head_dim // group,)) * g.uniform(1.0, 2.0, rows + (head_dim // group,)) * 3 / top)
    z = g.integers(0, (top if zero_top is None else zero_top) + 1, rows + (head_dim // group,)).astype(np.uint8)
    return codes, s.astype(np.float32), z


def dense_pool(pool, bits, group):
    """[slots, heads, head_dim] of a pool in fp64, as stored (not rotated back)."""
    codes, s, z = pool
    with np.errstate(all="ignore"):
        v = np.repeat(s.astype(np.float64), group, -1) * (unpack(codes, bits) - np.repeat(z.astype(np.float64), group, -1))
    return v.reshape(-1, *v.shape[2:])


def largest_steps(pool, bits, group):
    """|scale| times the largest |code - zero| of any code, per value of a pool: [slots, heads, head_dim]."""
    _, s, z = pool
    with np.errstate(all="ignore"):
        v = np.repeat(np.abs(s.astype(np.float64)) * np.maximum(z, 2**bits - 1 - z.astype(np.float64)), group, -1)
    return v.reshape(-1, *v.shape[2:])


@functools.cache
def hadamard(n):
    i = np.arange(n)
    par = np.array([[bin(a & b).count("1") & 1 for b in i] for a in i])
    return (1.0 - 2.0 * par) / np.sqrt(n)


def rotate(x, n):
    return (x.reshape(*x.shape[:-1], -1, n) @ hadamard(n)).reshape(x.shape) if n else x


def spread_abs(x, n):
    """Bound of a rotated row's error from a bound x of the row's: |H| x."""
    return (x.reshape(*x.shape[:-1], -1, n) @ np.abs(hadamard(n))).reshape(x.shape) if n else x


def shuffled_table(g, totals, page_size, spare=2):
    need = [-(-t // page_size) for t in totals]
    n_pages = sum(need) + spare
    order = g.permutation(n_pages).astype(np.int32)
    table = np.full((len(totals), max(need + [1])), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, n_pages


def attention(q, kd, vd, vstep, had_k, had_v, table, page_size, past, new, tree, scale, eps, cached=0.0):
    """(out, lse, bound of out, bound of lse): fp64, for stored-frame pools kd, vd [slots, heads, D]; vstep: the largest
    |scale (code - zero)| each stored value could have. The bounds allow an arithmetic that rounds the rotated query and
    the softmax weights to relative eps each and sums in fp32, with weights below 2^-33 of the largest held to that: p
    scale is kept in f16, whose smallest numbers are 2^-24 apart, scaled so that 2^8 stands for p = 1 at the largest
    scale of a token that any row of the tile sees, or at one that is 2^10 times the largest that the row sees, whichever
    is less (where there are larger ones the rows are done in fp32; 2^11 here, since the zero points let |code - zero|
    differ twofold). cached: what rounding the cached values costs, relative
    to each: 2^-11 where scale (code - zero) is rounded to f16 (the scale itself in two pieces, 2^-22); keys' errors move
    scores as the query's do, values' the sum in proportion."""
    n, q_heads, D = q.shape
    heads = kd.shape[1]
    grp, at, f32 = q_heads // heads, 0, 2.0**-24
    out, lse = np.zeros((n, q_heads, D)), np.full((n, q_heads), -np.inf)
    tol, lse_tol = np.zeros((n, q_heads, D)), np.zeros((n, q_heads))
    for b, (p, m) in enumerate(zip(past, new)):
        t = np.arange(p + m)
        pages = table[b, t // page_size].astype(np.int64)
        u = t - p
        if tree is None:
            seen = u[None] <= np.arange(m)[:, None]
        else:
            bits = tree[at:at + m].astype(np.int64).view(np.uint64)[:, None] >> np.clip(u, 0, 63).astype(np.uint64)[None]
            seen = (u < 0)[None] | ((u < 64)[None] & (bits & np.uint64(1)).astype(bool))
        live = np.flatnonzero(pages >= 0)
        slots, seen = (pages * page_size + t % page_size)[live], seen[:, live]
        some = seen.any(1)
        if len(live) and m:
            qr = (rotate(q[at:at + m].astype(np.float64), had_k) * scale).reshape(m, heads, grp, D)
            with np.errstate(all="ignore"):
                for h in range(heads):
                    k, v = kd[slots, h], vd[slots, h]
                    used = seen.any(0)[:, None]
                    k, v = np.where(used, k, 0), np.where(used, v, 0)
                    s = np.where(seen[:, None], qr[:, h] @ k.T, -np.inf)
                    top = np.where(some[:, None], s.max(-1), 0)
                    w = np.exp(s - top[..., None])
                    total = np.where(some[:, None], w.sum(-1), 1)
                    w = w / total[..., None]
                    rows, cols = slice(at, at + m), slice(h * grp, (h + 1) * grp)
                    out[rows, cols] = rotate(w @ v, had_v)
                    lse[rows, cols] = np.where(some[:, None], top + np.log(total), -np.inf)
                    # a rounded query moves a score by eps sum |k q| at most, plus fp32 sums; weights move by twice
                    # that (their own score and the total), are rounded once, and are summed in fp32
                    count = seen.sum(1)[:, None]
                    kq = np.where(seen[:, None], np.abs(qr[:, h]) @ np.abs(k).T, 0).max(-1)
                    ds = (eps + cached * (1 + eps) + (D + 16) * f32) * kq + 4 * f32 * np.where(np.isfinite(s), np.abs(s), 0).max(-1)
                    rel = 2 * np.expm1(ds) + 2 * eps + cached * (1 + 2 * eps) + (count + 64) * f32
                    far = np.where(used, vstep[slots, h], 0)
                    own = np.where(seen[..., None], far, 0).max(1)
                    least = ((count * 2.0**-33) * np.minimum(far.max(0), 2.0**11 * own))[:, None]
                    # (whatever the weights, both results lie between the values: twice the largest is never passed)
                    moved = np.fmin(rel[..., None] * (w @ np.abs(v)), 2.1 * own[:, None])
                    tol[rows, cols] = spread_abs(moved + least, had_v) * (1 + 16 * f32) + 1e-30
                    lse_tol[rows, cols] = ds + eps + (count + 64) * f32 + 4 * f32 * np.abs(np.where(some[:, None], lse[rows, cols], 0))
        at += m
    return out, lse, tol, lse_tol


def rotary(x, positions, freq, pairs, factor, inverse):
    y = x.astype(np.float64).copy()
    r = 2 * len(freq)
    ang = positions.astype(np.float64)[:, None] * freq
    c, s = np.cos(ang)[:, None] * factor, np.sin(ang)[:, None] * factor * (-1 if inverse else 1)
    ia, ib = (np.arange(0, r, 2), np.arange(1, r, 2)) if pairs else (np.arange(r // 2), np.arange(r // 2, r))
    a, b = x[..., ia].astype(np.float64), x[..., ib].astype(np.float64)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


class Table:
    """The page table, one sequence and one page at a time."""

    def __init__(self, refs, pages, held, page_size):
        self.refs, self.pages, self.held, self.ps = refs.copy(), pages.copy(), held.copy(), page_size

    def count(self, tokens):
        return -(-int(tokens) // self.ps)

    def free(self):
        return [int(p) for p in np.flatnonzero(self.refs == 0)]

    def resize(self, want):
        room = self.pages.shape[1] * self.ps
        bad = False
        for b, w in enumerate(want):
            if w == -1:
                continue
            if w < -1 or w > room:
                bad = True
                continue
            have, to = self.count(self.held[b]), self.count(w)
            for j in range(to, have):
                self.refs[self.pages[b, j]] -= 1
                self.pages[b, j] = -1
            if to <= have:
                self.held[b] = w
        free, at = self.free(), 0
        for b, w in enumerate(want):
            if w < 0 or w > room:
                continue
            have, to = self.count(self.held[b]), self.count(w)
            if to <= have:
                continue
            at += to - have
            if at > len(free):
                continue
            got = free[at - (to - have):at]
            self.pages[b, have:to] = got
            self.refs[got] = 1
            self.held[b] = w
        return bad

    def fork(self, src, dst):
        n_seqs, held = len(self.held), self.held.copy()
        origin, fresh = np.full(len(src), -1, np.int32), np.full(len(src), -1, np.int32)
        free, at, bad, used = self.free(), 0, False, set()
        pages = self.pages.copy()
        for i, (a, b) in enumerate(zip(src, dst)):
            if a == -1:
                continue
            inside = 0 <= a < n_seqs and 0 <= b < n_seqs
            if not inside or int(b) in used or held[b] != 0:
                bad = True
                if inside:
                    used.add(int(b))
                continue
            used.add(int(b))
            full, part = int(held[a]) // self.ps, int(held[a]) % self.ps > 0
            at += part
            if at > len(free):
                continue
            if part:
                origin[i], fresh[i] = pages[a, full], free[at - 1]
                self.pages[b, full] = fresh[i]
                self.refs[fresh[i]] = 1
            self.pages[b, :full] = pages[a, :full]
            self.refs[pages[a, :full]] += 1
            self.held[b] = held[a]
        return origin, fresh, bad
