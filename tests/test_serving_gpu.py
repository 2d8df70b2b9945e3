"""The serving operators on the GPU against plain 64-bit statements: the quantized matrix-vector product, the adapted
layer on a few tokens, the quantized cache, and a decode step that uses them together."""

import numpy as np
import pytest

import oracle
from _serving import (butterflies, dense_weight, half_step, pack, quantize, random_weight, round_to, unpack, values)
from _util import bf16_dev, host, to_dev
from workloads import f32_to_bf16_bits, pack_codes, random_pattern, rng_for

pytestmark = pytest.mark.gpu

INVALID = 1


def _W():
    import walsh_hadamard_sparse_b200 as W

    return W


def _dev(x, dtype):
    return bf16_dev(f32_to_bf16_bits(x)) if dtype == "bf16" else to_dev(np.asarray(x, np.float32))


def _qweight(W, bits, group, packed, s, z):
    return W.QWeight(bits, group, to_dev(packed), to_dev(s), to_dev(z))


def _sum_tol(d_in):
    """fp32 sums of d_in products, in chains of at most d_in/16 + 64 additions; an addition on the tensor cores may
    truncate (2^-23 of the partial sum)."""
    return (d_in / 16 + 64) * 2.0**-23


def _check_base(Y, x, w, dtype, extra=0.0):
    want = x @ w.T
    tol = half_step(dtype) * np.abs(want) * 1.01 + _sum_tol(x.shape[1]) * (np.abs(x) @ np.abs(w).T) + extra + 1e-30
    err = np.abs(host(Y) - want)
    assert np.all(err <= tol), float((err / tol).max())


# d_out, d_in, group: whole tiles, one row, odd rows, widths that end inside a tile, every kind of group
SHAPES = [(64, 256, 128), (1, 128, 128), (7, 8, 8), (33, 40, 8), (129, 96, 96), (48, 320, 64), (50, 352, 32),
          (17, 1024, 1024), (200, 200, 40), (95, 4096, 256), (24, 2176, 128), (16, 4128, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("shape", SHAPES)
def test_qgemv(shape, bits, dtype):
    W = _W()
    d_out, d_in, group = shape
    g = rng_for(91, "qgemv", d_out, d_in, group, bits)
    q, packed, s, z = random_weight(g, d_out, d_in, bits, group)
    wq, w = _qweight(W, bits, group, packed, s, z), dense_weight(q, s, z, group)
    for T in (1, 2, 3, 5, 8, 9, 21, 64):
        x = round_to(g.standard_normal((T, d_in)) * np.exp(g.standard_normal((T, 1))), dtype)
        _check_base(W.qgemv(wq, _dev(x, dtype)), x.astype(np.float64), w, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_qgemv_larger_layers(dtype):
    W = _W()
    for d_out, d_in, group, bits, T in ((1000, 4096, 128, 4, 1), (4096, 1376, 32, 3, 17), (2731, 4000, 32, 2, 40),
                                        (600, 14336, 64, 4, 33)):
        g = rng_for(92, "qgemv", d_out, d_in)
        q, packed, s, z = random_weight(g, d_out, d_in, bits, group)
        x = round_to(g.standard_normal((T, d_in)), dtype)
        Y = W.qgemv(_qweight(W, bits, group, packed, s, z), _dev(x, dtype))
        _check_base(Y, x.astype(np.float64), dense_weight(q, s, z, group), dtype)


@pytest.mark.parametrize("group", [8, 32, 64, 128])
@pytest.mark.parametrize("bits", [2, 3, 4])
def test_qgemv_any_zero_point(bits, group):
    """The format's zero points are bytes: those above the codes' range, and above 127, count as well."""
    W = _W()
    g = rng_for(93, "zeros", bits, group)
    q, packed, s, z = random_weight(g, 40, 256, bits, group, zero_top=255)
    z[0, :] = 255
    z[1, :] = 128
    x = round_to(g.standard_normal((3, 256)), "bf16")
    _check_base(W.qgemv(_qweight(W, bits, group, packed, s, z), _dev(x, "bf16")), x.astype(np.float64),
                dense_weight(q, s, z, group), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [8, 32, 64, 128])
def test_qgemv_infinities_and_nan_stay_with_their_token(group, dtype):
    W = _W()
    g = rng_for(94, "inf", group)
    q, packed, s, z = random_weight(g, 40, 512, 4, group)
    q[:, 200] = 9
    z[:] = 3  # q - z = 6 at column 200
    packed = pack_codes(q, 4)
    wq, w = _qweight(W, 4, group, packed, s, z), dense_weight(q, s, z, group)
    x = round_to(g.standard_normal((9, 512)), dtype)
    clean = W.qgemv(wq, _dev(x, dtype))
    y = x.copy()
    y[2, 200], y[4, 200], y[7, 17] = np.inf, np.nan, -np.inf
    got = W.qgemv(wq, _dev(y, dtype))
    keep = [0, 1, 3, 5, 6, 8]
    assert np.array_equal(host(got)[keep], host(clean)[keep])
    assert np.array_equal(host(got)[2], np.sign(w[:, 200]) * np.inf)
    assert np.all(np.isnan(host(got)[4]))
    assert not np.any(np.isfinite(host(got)[7]))


def test_qgemv_large_and_tiny_fp32_values():
    """Values at the ends of fp32's range keep their full precision (products and sums in range)."""
    W = _W()
    g = rng_for(95, "range")
    q, packed, s, z = random_weight(g, 32, 256, 4, 128)
    wq, w = _qweight(W, 4, 128, packed, s, z), dense_weight(q, s, z, 128)
    x = g.standard_normal((3, 256)).astype(np.float32)
    x[0] *= np.float32(1e35)
    x[1] *= np.float32(1e-25)
    x[2, ::2] *= np.float32(1e-20)
    _check_base(W.qgemv(wq, _dev(x, "f32")), x.astype(np.float64), w, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 7, 40])
@pytest.mark.parametrize("bits,group", [(2, 32), (2, 64), (3, 128), (4, 128)])
def test_qgemv_a_value_far_above_the_others(bits, group, T, dtype):
    """A value of a thousand whose weight is zero (code = zero point) leaves the other columns' sums whole: fp32 sums of
    codes below 2^bits times values, 24 bits of at most 8 + 8 roundings of the largest partial sum a group."""
    W = _W()
    g = rng_for(112, "outlier", bits, group, T)
    q, packed, s, z = random_weight(g, 48, 512, bits, group)
    q[:, [5, 300]] = z[:, [5 // group, 300 // group]]
    packed = pack_codes(q, bits)
    w = dense_weight(q, s, z, group)
    x = round_to(g.standard_normal((T, 512)), dtype)
    x[:, 5], x[:, 300] = 1000.0, -997.0
    want = x.astype(np.float64) @ w.T
    top = 2.0**bits * 1000.0 * np.abs(s).max(-1)
    tol = half_step(dtype) * 1.01 * np.abs(want) + 16 * 2.0**-24 * 2 * top + 2.0**-20 * (np.abs(x) * (np.abs(x) < 100)) @ np.abs(w).T
    assert np.all(np.abs(host(W.qgemv(_qweight(W, bits, group, packed, s, z), _dev(x, dtype))) - want) <= tol)


@pytest.mark.parametrize("dtype,T,d_in", [
    ("bf16", 1, 16384), ("bf16", 1, 16416), ("bf16", 2, 8192), ("bf16", 2, 8224),  # operands made in the product or not
    ("bf16", 20, 480), ("bf16", 21, 480), ("f32", 6, 480), ("f32", 7, 480),  # the last and first of many columns
    ("bf16", 28, 480), ("bf16", 33, 480), ("f32", 10, 480), ("f32", 11, 480),  # two and three blocks of columns
    ("bf16", 64, 2176), ("f32", 42, 1376), ("f32", 43, 1376), ("f32", 64, 160)])  # empty and uneven slices, two passes
@pytest.mark.parametrize("bits,group", [(2, 32), (3, 32), (4, 160)])
def test_qgemv_borders_of_the_kernels(bits, group, dtype, T, d_in):
    W = _W()
    group = group if d_in % group == 0 else 32
    for d_out in (1, 40, 129, 300):
        g = rng_for(113, "borders", bits, T, d_in, d_out)
        q, packed, s, z = random_weight(g, d_out, d_in, bits, group, zero_top=255 if d_out == 40 else None)
        x = round_to(g.standard_normal((T, d_in)), dtype)
        Y = W.qgemv(_qweight(W, bits, group, packed, s, z), _dev(x, dtype))
        _check_base(Y, x.astype(np.float64), dense_weight(q, s, z, group), dtype)


def _decode_case(g, d_in, d_out, n, bits, group, counts, T, dtype, scale=0.05):
    rp, ci, cf = random_pattern(d_out, d_in, counts=counts, rng=g, coef_scale=scale)
    q, packed, s, z = random_weight(g, d_out, d_in, bits, group)
    x = round_to(g.standard_normal((T, d_in)), dtype)
    return rp, ci, cf, q, packed, s, z, x


def _check_decode(Y, x, w, rp, ci, cf, n, alpha, dtype):
    d_out, d_in = len(rp) - 1, x.shape[1]
    x = x.astype(np.float64)
    Z = oracle.fwht(x, n)
    F = np.zeros((d_out, d_in))
    F[oracle.csr_rows(rp), ci] = cf
    base = x @ w.T if w is not None else np.zeros((x.shape[0], d_out))
    absb = np.abs(x) @ np.abs(w).T if w is not None else 0.0
    want = base + alpha * Z @ F.T
    # Z in fp32: log2 n additions and the factor, against the block's largest possible sum; then the row's own sum
    zb = np.repeat(np.abs(x).reshape(x.shape[0], -1, n).sum(-1) / np.sqrt(n), n, axis=1) * (np.log2(n) + 2) * 2.0**-24
    cnt = np.diff(rp).max(initial=0) + 64
    tol = (half_step(dtype) * np.abs(want) * 1.01 + _sum_tol(d_in) * absb + abs(alpha) * (
        zb @ np.abs(F).T + cnt * 2.0**-24 * (np.abs(Z) @ np.abs(F).T)) + 2.0**-23 * (np.abs(base) + np.abs(want)) + 1e-30)
    err = np.abs(host(Y) - want)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(256, 64, 256, 4, 128), (320, 40, 64, 3, 32), (4096, 1032, 4096, 4, 128),
                                   (7168, 264, 1024, 2, 64), (24, 16, 8, 4, 8), (14336, 136, 2048, 3, 128),
                                   (8192, 24, 8192, 4, 64)])
def test_adapter_decode(shape, dtype):
    W = _W()
    d_in, d_out, n, bits, group = shape
    g = rng_for(96, "decode", d_in, d_out)
    counts = g.integers(0, min(d_in, 300), d_out)
    counts[0], counts[1], counts[-1] = 0, min(d_in, 2000), 1  # an empty row, a crowded one, a single entry
    for T in (1, 2, 3, 4, 6, 16, 33, 64):
        rp, ci, cf, q, packed, s, z, x = _decode_case(g, d_in, d_out, n, bits, group, counts, T, dtype)
        a = W.Adapter(d_in, d_out, n, ci.size, to_dev(rp), to_dev(ci), to_dev(cf))
        xd = _dev(x, dtype)
        Y = W.adapter_decode(a, xd, 0.75, _qweight(W, bits, group, packed, s, z))
        _check_decode(Y, x, dense_weight(q, s, z, group), rp, ci, cf, n, 0.75, dtype)
        _check_decode(W.adapter_decode(a, xd, -1.5), x, None, rp, ci, cf, n, -1.5, dtype)  # the adapter alone


def test_adapter_decode_without_entries_is_the_base_product():
    import torch

    W = _W()
    g = rng_for(97, "p0")
    q, packed, s, z = random_weight(g, 64, 512, 4, 128)
    wq = _qweight(W, 4, 128, packed, s, z)
    x = _dev(round_to(g.standard_normal((5, 512)), "bf16"), "bf16")
    rp = to_dev(np.zeros(65, np.int32))
    a = W.Adapter(512, 64, 512, 0, rp, to_dev(np.zeros(1, np.int32)), to_dev(np.zeros(1, np.float32)))
    Z = torch.empty_like(x)
    assert torch.equal(W.adapter_decode(a, x, 1.0, wq, Z_out=Z), W.qgemv(wq, x))
    assert np.allclose(host(Z), oracle.fwht(host(x), 512), atol=2e-2)
    assert torch.count_nonzero(W.adapter_decode(a, x, 1.0)).item() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_adapter_decode_z_out_feeds_the_backward(dtype):
    """Z_out is X H in X's type: adapter_bwd on it gives the gradients of these tokens."""
    import torch

    W = _W()
    d_in, d_out, n, T = 512, 128, 256, 5
    g = rng_for(98, "zout")
    rp, ci, cf, *_, x = _decode_case(g, d_in, d_out, n, 4, 64, g.integers(1, 40, d_out), T, dtype)
    a = W.plan_build(W.Adapter(d_in, d_out, n, ci.size, to_dev(rp), to_dev(ci), to_dev(cf)))
    xd = _dev(x, dtype)
    Z = torch.empty_like(xd)
    W.adapter_decode(a, xd, 0.5, Z_out=Z)
    want = oracle.fwht(x.astype(np.float64), n)
    zb = np.repeat(np.abs(x).reshape(T, -1, n).sum(-1) / np.sqrt(n), n, axis=1)
    assert np.all(np.abs(host(Z) - want) <= half_step(dtype) * 1.01 * np.abs(want) + zb * 10 * 2.0**-24)
    dY = round_to(g.standard_normal((T, d_out)), dtype)
    dc, dX = W.adapter_bwd(a, _dev(dY, dtype), Z, 0.5)
    zh = host(Z)
    rows = oracle.csr_rows(rp)
    terms = 0.5 * dY.astype(np.float64)[:, rows] * zh[:, ci]
    assert np.all(np.abs(host(dc) - terms.sum(0)) <= 2.0**-20 * np.abs(terms).sum(0) + 1e-30)
    # against differences: the loss <dY, Y> is linear in c, so a difference is the gradient up to rounding
    j = int(g.integers(0, ci.size))
    step = 1.0
    up = cf.copy()
    up[j] += step
    b = W.Adapter(d_in, d_out, n, ci.size, to_dev(rp), to_dev(ci), to_dev(up))
    if dtype == "f32":
        diff = (host(W.adapter_decode(b, xd, 0.5)) - host(W.adapter_decode(a, xd, 0.5))) * dY
        assert abs(diff.sum() / step - terms.sum(0)[j]) <= 1e-4 * np.abs(dY).sum()


def test_products_repeat_bit_for_bit_on_other_streams_and_in_graphs():
    import torch

    W = _W()
    d_in, d_out, n, T = 4096, 1032, 4096, 3
    g = rng_for(99, "graph")
    rp, ci, cf, q, packed, s, z, x = _decode_case(g, d_in, d_out, n, 4, 128, g.integers(0, 200, d_out), T, "bf16")
    a = W.Adapter(d_in, d_out, n, ci.size, to_dev(rp), to_dev(ci), to_dev(cf))
    wq = _qweight(W, 4, 128, packed, s, z)
    xs = [_dev(round_to(g.standard_normal((T, d_in)), "bf16"), "bf16") for _ in range(3)]
    want = [W.adapter_decode(a, v, 1.0, wq) for v in xs]
    base = [W.qgemv(wq, v) for v in xs]
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(20):  # two streams at once, each with its own workspace
        for st, k in ((side, 0), (other, 1)):
            with torch.cuda.stream(st):
                outs.append((k, W.adapter_decode(a, xs[k], 1.0, wq), W.qgemv(wq, xs[k])))
    torch.cuda.synchronize()
    for k, y, b in outs:
        assert torch.equal(y, want[k]) and torch.equal(b, base[k])
    xin = xs[0].clone()
    ws = torch.empty(W.workspace_size(10, d_out, d_in, a.p, T, 1), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = W.adapter_decode(a, xin, 1.0, wq, ws=ws)
        y2 = W.adapter_decode(a, xin, 1.0, wq, ws=ws)  # the same workspace, one call after the other
        b = W.qgemv(wq, xin)
    for k in (1, 2, 0):
        xin.copy_(xs[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k]) and torch.equal(y2, want[k]) and torch.equal(b, base[k])


@pytest.mark.parametrize("dtype,T,d_out", [("bf16", 64, 1032), ("f32", 24, 4096), ("bf16", 33, 104), ("bf16", 1, 1032),
                                            ("f32", 16, 520)])
def test_products_of_many_tokens_repeat_on_two_streams_and_in_graphs(dtype, T, d_out):
    """Clusters of two streams at once, each with its own workspace, and two calls of one workspace in a graph."""
    import torch

    W = _W()
    d_in = 4096
    g = rng_for(114, "many", T, d_out)
    rp, ci, cf, q, packed, s, z, x = _decode_case(g, d_in, d_out, d_in, 4, 64, g.integers(0, 200, d_out), T, dtype)
    a = W.Adapter(d_in, d_out, d_in, ci.size, to_dev(rp), to_dev(ci), to_dev(cf))
    wq = _qweight(W, 4, 64, packed, s, z)
    xs = [_dev(round_to(g.standard_normal((T, d_in)), dtype), dtype) for _ in range(2)]
    want, base = [W.adapter_decode(a, v, 1.0, wq) for v in xs], [W.qgemv(wq, v) for v in xs]
    torch.cuda.synchronize()
    outs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs.append((k, W.adapter_decode(a, xs[k], 1.0, wq), W.qgemv(wq, xs[k])))
    torch.cuda.synchronize()
    for k, y, b in outs:
        assert torch.equal(y, want[k]) and torch.equal(b, base[k])
    xin = xs[0].clone()
    with_base = 1 if dtype == "bf16" else 2
    ws = torch.empty(W.workspace_size(10, d_out, d_in, a.p, T, with_base), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = W.adapter_decode(a, xin, 1.0, wq, ws=ws)
        y2 = W.adapter_decode(a, xin, 1.0, wq, ws=ws)
        b = W.qgemv(wq, xin)
    for k in (1, 0):
        xin.copy_(xs[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k]) and torch.equal(y2, want[k]) and torch.equal(b, base[k])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_qgemv_infinities_among_many_tokens(dtype):
    W = _W()
    g = rng_for(115, "inf many")
    q, packed, s, z = random_weight(g, 200, 512, 4, 128)
    q[:, 200], z[:] = 9, 3
    packed = pack_codes(q, 4)
    wq, w = _qweight(W, 4, 128, packed, s, z), dense_weight(q, s, z, 128)
    x = round_to(g.standard_normal((64, 512)), dtype)
    clean = host(W.qgemv(wq, _dev(x, dtype)))
    x[2, 200], x[40, 200], x[63, 17] = np.inf, np.nan, -np.inf
    got = host(W.qgemv(wq, _dev(x, dtype)))
    keep = np.setdiff1d(np.arange(64), [2, 40, 63])
    assert np.array_equal(got[keep], clean[keep])
    assert np.array_equal(got[2], np.sign(w[:, 200]) * np.inf)
    assert np.all(np.isnan(got[40])) and not np.any(np.isfinite(got[63]))


# ---------------------------------------------------------------- the cache

CACHES = [  # heads, head_dim, bits, group, had_block, page_size
    (8, 128, 4, 128, 128, 16), (8, 128, 4, 32, 128, 64), (2, 128, 8, 64, 0, 16), (3, 64, 2, 64, 64, 1),
    (1, 256, 3, 64, 256, 100), (5, 80, 3, 40, 16, 16), (2, 96, 4, 96, 32, 7), (1, 8, 2, 8, 4, 3), (4, 24, 8, 24, 2, 5),
    (2, 192, 4, 192, 64, 16), (2, 256, 8, 256, 0, 32), (7, 16, 4, 8, 16, 9), (1, 120, 3, 120, 8, 4)]


def _rows(g, n, heads, head_dim, dtype):
    x = g.standard_normal((n, heads, head_dim)).astype(np.float32)
    x *= np.where(g.random((heads, head_dim)) < 0.05, 8.0, 1.0).astype(np.float32)
    return round_to(x, dtype)


def _filled(W, g, n_pages, page_size, heads, head_dim, bits, group, had_block):
    """A cache with arbitrary contents, so that untouched slots show."""
    c = W.cache_alloc(n_pages, page_size, heads, head_dim, bits, group, had_block)
    c.codes.copy_(to_dev(g.integers(0, 256, tuple(c.codes.shape)).astype(np.uint8)))
    c.scales.copy_(to_dev((g.random(tuple(c.scales.shape)) + 0.1).astype(np.float32)))
    c.zeros.copy_(to_dev(g.integers(0, 2**bits, tuple(c.zeros.shape)).astype(np.uint8)))
    return c


def _state(c):
    flat = lambda t: t.cpu().numpy().reshape(-1, *t.shape[2:])  # noqa: E731
    return flat(c.codes).copy(), flat(c.scales).copy(), flat(c.zeros).copy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", CACHES)
def test_cache_write_bit_for_bit(shape, dtype):
    W = _W()
    heads, head_dim, bits, group, had_block, page_size = shape
    g = rng_for(100, "write", *shape)
    c = _filled(W, g, 9, page_size, heads, head_dim, bits, group, had_block)
    for n in (1, 2, min(9 * page_size, 37)):
        slots = g.permutation(9 * page_size)[:n].astype(np.int64)
        if n > 2:
            slots[[0, n // 2]] = -1  # padding
        x = _rows(g, n, heads, head_dim, dtype)
        if n > 1:
            x[1, 0] = 0.0
            x[1, -1] = 1.5
        codes, scales, zeros = _state(c)
        W.cache_write(c, _dev(x, dtype), to_dev(slots))
        q, s, z = quantize(x, bits, group, had_block, dtype)
        live = slots >= 0
        codes[slots[live]], scales[slots[live]], zeros[slots[live]] = pack(q, bits)[live], s[live], z[live]
        got = _state(c)
        assert np.array_equal(got[1].view(np.int32), scales.view(np.int32))
        assert np.array_equal(got[2], zeros)
        assert np.array_equal(got[0], codes)


def test_cache_write_special_values():
    """A group with an infinity or a NaN reads as NaN and its neighbours are untouched; ranges below fp32's normal
    numbers read as zero; ties go up; the range is exact at both ends."""
    import torch

    W = _W()
    for dtype in ("bf16", "f32"):
        for bits in (2, 3, 4, 8):
            c = W.cache_alloc(1, 16, 1, 64, bits, 16, 0)
            x = round_to(rng_for(101, "special").standard_normal((16, 1, 64)), dtype)
            x[0, 0, 3], x[1, 0, 20], x[2, 0, 40] = np.inf, np.nan, -np.inf
            x[3] = 0.0
            x[4] = np.float32(2.0**-140)
            x[5, 0, :16] = np.float32(3e38) * np.where(np.arange(16) % 2, 1, -1)
            x[6, 0, :16] = np.arange(16)  # exact codes for 4 bits
            x[7] = -4.0
            x[8] = 7.0
            x[9, 0, :16] = np.arange(16) / 2 + 0.25 * (np.arange(16) % 2)
            x = round_to(x, dtype)
            W.cache_write(c, _dev(x, dtype), to_dev(np.arange(16, dtype=np.int64)))
            q, s, z = quantize(x, bits, 16, 0, dtype)
            got = _state(c)
            assert np.array_equal(np.isnan(got[1]), np.isnan(s)) and np.isnan(s).sum() >= 3
            assert np.array_equal(np.nan_to_num(got[1]), np.nan_to_num(s))
            assert np.array_equal(got[2], z) and np.array_equal(got[0], pack(q, bits))
            back = W.cache_read(c, to_dev(np.zeros((1, 1), np.int32)), to_dev(np.array([0, 16], np.int64)), 16,
                                dtype=torch.float32)
            back = host(back)
            assert np.array_equal(np.isnan(back), np.repeat(np.isnan(s), 16, axis=-1))
            assert np.all(back[3] == 0) and np.all(back[4] == 0)


def test_cache_write_a_rotated_row_with_an_infinity_is_nan_as_a_block():
    import torch

    W = _W()
    c = W.cache_alloc(1, 4, 2, 128, 4, 32, 64)
    x = rng_for(102, "inf").standard_normal((1, 2, 128)).astype(np.float32)
    x[0, 1, 70] = np.inf
    W.cache_write(c, _dev(x, "bf16"), to_dev(np.array([2], np.int64)))
    out = W.cache_read(c, to_dev(np.zeros((1, 1), np.int32)), to_dev(np.array([0, 1], np.int64)), 1,
                       first=to_dev(np.array([2], np.int64)), dtype=torch.float32)
    nan = np.isnan(host(out))[0]
    assert not nan[0].any() and not nan[1, :64].any() and nan[1, 64:].all()


def test_cache_slots_outside_are_skipped_and_reported():
    W = _W()
    import walsh_hadamard_sparse_b200._lib as L
    import ctypes
    import torch

    g = rng_for(103, "bad")
    c = _filled(W, g, 2, 4, 2, 64, 4, 64, 64)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert L.lib().qwha_check_stream_status(stream) == 0
    before = _state(c)
    x = _rows(g, 4, 2, 64, "bf16")
    W.cache_write(c, _dev(x, "bf16"), to_dev(np.array([8, -2, 1 << 40, 3], np.int64)))
    assert L.lib().qwha_check_stream_status(stream) == INVALID
    assert b"slot" in L.lib().qwha_last_error()
    assert L.lib().qwha_check_stream_status(stream) == 0  # cleared
    got = _state(c)
    keep = [i for i in range(8) if i != 3]
    for b, a in zip(before, got):
        assert np.array_equal(b[keep], a[keep])
    q, s, z = quantize(x, 4, 64, 64, "bf16")
    assert np.array_equal(got[0][3], pack(q, 4)[3])


def _table(g, lens, page_size, n_pages, width=None):
    need = [-(-int(v) // page_size) for v in lens]
    width = width or max(max(need), 1)
    order = g.permutation(n_pages)[:sum(need)]
    t = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = order[at:at + k]
        at += k
    return t


def _want_read(c, bits, group, had_block, table, first, count, page_size):
    codes, s, z = _state(c)
    slots = np.concatenate([[int(table[b, t // page_size]) * page_size + t % page_size
                             for t in range(first[b], first[b] + count[b])] for b in range(len(count))] or [[]])
    v = values(codes, s, z, bits, group)[slots.astype(np.int64)]
    return butterflies(v, had_block), np.abs(v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", CACHES)
def test_cache_read(shape, dtype):
    import torch

    W = _W()
    heads, head_dim, bits, group, had_block, page_size = shape
    g = rng_for(104, "read", *shape)
    for first, count in (([0], [1]), ([0, 0, 0], [5, 0, 23]), ([3, 0, 17, 40], [1, 33, 0, 9])):
        lens = np.add(first, count)
        n_pages = int(sum(-(-int(v) // page_size) for v in lens)) + 2
        c = _filled(W, g, n_pages, page_size, heads, head_dim, bits, group, had_block)
        table = _table(g, lens, page_size, n_pages)
        starts = np.concatenate([[0], np.cumsum(count)]).astype(np.int64)
        rows = int(starts[-1])
        out = torch.full((rows + 3, heads, head_dim), 7.5, device="cuda",
                         dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
        W.cache_read(c, to_dev(table), to_dev(starts), rows + 3, first=to_dev(np.array(first, np.int64)), out=out)
        want, mag = _want_read(c, bits, group, had_block, table, first, count, page_size)
        got = host(out)
        assert np.all(got[rows:] == 7.5)  # rows behind the last sequence
        n = had_block or 1
        blk = np.repeat(mag.reshape(rows, heads, -1, n).sum(-1) / np.sqrt(n), n, axis=-1)
        tol = half_step(dtype) * 1.01 * np.abs(want) + (np.log2(n) + 3) * 2.0**-24 * blk + 1e-30
        assert np.all(np.abs(got[:rows] - want) <= tol)


def _written_and_read(W, g, shape, n, dtype, spoil):
    """n rows in random slots, bit for bit, then read back one page after the other."""
    import torch

    heads, head_dim, bits, group, had_block, page_size = shape
    n_pages = -(-n // page_size) + 1
    c = _filled(W, g, n_pages, page_size, heads, head_dim, bits, group, had_block)
    slots = g.permutation(n_pages * page_size)[:n].astype(np.int64)
    slots[n // 3] = -1
    x = _rows(g, n, heads, head_dim, dtype)
    for i, v in enumerate(spoil):  # one value in a group, the rows around it stay whole
        x[(5 * i + 1) % n, i % heads, (37 * i) % head_dim] = v
    codes, scales, zeros = _state(c)
    W.cache_write(c, _dev(x, dtype), to_dev(slots))
    with np.errstate(invalid="ignore", over="ignore"):
        q, s, z = quantize(x, bits, group, had_block, dtype)
    live = slots >= 0
    codes[slots[live]], scales[slots[live]], zeros[slots[live]] = pack(q, bits)[live], s[live], z[live]
    got = _state(c)
    assert np.array_equal(np.isnan(got[1]), np.isnan(scales))
    assert np.array_equal(np.nan_to_num(got[1]), np.nan_to_num(scales))
    assert np.array_equal(got[2], zeros)
    assert np.array_equal(got[0], codes)
    table = g.permutation(n_pages).astype(np.int32)[None]
    rows = n_pages * page_size
    out = W.cache_read(c, to_dev(table), to_dev(np.array([0, rows], np.int64)), rows,
                       dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    want, mag = _want_read(c, bits, group, had_block, table, [0], [rows], page_size)
    m = had_block or 1
    blk = np.repeat(mag.reshape(rows, heads, -1, m).sum(-1) / np.sqrt(m), m, axis=-1)
    tol = half_step(dtype) * 1.01 * np.abs(want) + (np.log2(m) + 3) * 2.0**-24 * blk + 1e-30
    got = host(out)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.all((np.abs(got - want) <= tol) | np.isnan(want))


@pytest.mark.parametrize("had_block", [0, 2, 4, 8, 16, 32, 64, 128])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("bits", [2, 3, 4, 8])
def test_cache_units_of_128(bits, group, had_block):
    """Every block with every group and code in rows that make up units of 128 elements: an odd number of units to a
    token, values that spoil a group."""
    W = _W()
    g = rng_for(110, "units", bits, group, had_block)
    for dtype in ("bf16", "f32"):
        _written_and_read(W, g, (3, 128, bits, group, had_block, 5), 23, dtype, (np.inf, np.nan, -np.inf))
        if group <= 64 and had_block <= 64:
            _written_and_read(W, g, (2, 64, bits, group, had_block, 16), 9, dtype, ())


@pytest.mark.parametrize("shape,n", [((300, 128, 4, 64, 128, 16), 9), ((8, 32, 4, 32, 32, 64), 5000),
                                     ((1, 128, 3, 128, 64, 16), 20000), ((6, 64, 8, 32, 16, 32), 4000),
                                     ((4, 256, 2, 256, 64, 16), 40)])
def test_cache_many_units_to_a_tile(shape, n):
    """Tiles of several tokens, tokens of more units than a tile holds, groups of two units."""
    g = rng_for(111, "tiles", *shape)
    _written_and_read(_W(), g, shape, n, "bf16", (np.inf,))


def test_cache_read_bad_pages_are_left_and_reported():
    W = _W()
    import walsh_hadamard_sparse_b200._lib as L
    import ctypes
    import torch

    g = rng_for(105, "pages")
    c = _filled(W, g, 3, 4, 2, 64, 4, 64, 0)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert L.lib().qwha_check_stream_status(stream) == 0
    table = np.array([[2, -1], [0, 3]], np.int32)  # no page; a page outside
    starts = np.array([0, 6, 15], np.int64)  # 9 rows of sequence 1: one beyond the page table
    out = torch.full((15, 2, 64), 7.5, device="cuda")
    W.cache_read(c, to_dev(table), to_dev(starts), 15, out=out)
    assert L.lib().qwha_check_stream_status(stream) == INVALID
    assert b"page" in L.lib().qwha_last_error()
    got = host(out)
    codes, s, z = _state(c)
    v = values(codes, s, z, 4, 64)
    assert np.allclose(got[:4], v[8:12], rtol=1e-6) and np.allclose(got[6:10], v[0:4], rtol=1e-6)
    assert np.all(got[4:6] == 7.5) and np.all(got[10:] == 7.5)
    # capacity below the sequences: only the rows that fit
    small = torch.full((5, 2, 64), 7.5, device="cuda")
    W.cache_read(c, to_dev(np.array([[2, 1], [0, 1]], np.int32)), to_dev(starts), 5, out=small)
    assert np.allclose(host(small)[:4], v[8:12], rtol=1e-6)
    assert L.lib().qwha_check_stream_status(stream) == 0


def test_validate_slots():
    W = _W()
    c = W.cache_alloc(4, 16, 1, 64)
    ok = np.array([0, 63, -1, 5, -1, 32], np.int64)
    W.validate_slots(c, to_dev(ok))
    for bad, text in ((64, "outside"), (-2, "outside"), (5, "twice")):
        s = ok.copy()
        s[4] = bad
        with pytest.raises(W.QwhaError, match=text) as e:
            W.validate_slots(c, to_dev(s))
        assert "(at 4)" in str(e.value) or bad == 5


def test_cache_pair_is_two_single_calls_and_replays_in_a_graph():
    import torch

    W = _W()
    g = rng_for(106, "pair")
    mk = lambda: (W.cache_alloc(8, 16, 4, 128, 4, 64, 128), W.cache_alloc(8, 16, 2, 64, 8, 64, 0))  # noqa: E731
    pair, single, captured = mk(), mk(), mk()
    slots = to_dev(g.permutation(128)[:50].astype(np.int64))
    k, v = (_dev(_rows(g, 50, h, d, "bf16"), "bf16") for h, d in ((4, 128), (2, 64)))
    W.cache_write(pair, (k, v), slots)
    W.cache_write(single[0], k, slots)
    W.cache_write(single[1], v, slots)
    table = to_dev(np.arange(8, dtype=np.int32)[None])
    starts = to_dev(np.array([0, 128], np.int64))
    kr, vr = W.cache_read(pair, table, starts, 128)
    assert torch.equal(kr, W.cache_read(single[0], table, starts, 128))
    assert torch.equal(vr, W.cache_read(single[1], table, starts, 128))
    kin, vin = torch.zeros_like(k), torch.zeros_like(v)
    W.cache_write(captured, (kin, vin), slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.cache_write(captured, (kin, vin), slots)
        out = W.cache_read(captured, table, starts, 128)
    for _ in range(2):
        kin.copy_(k)
        vin.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], kr) and torch.equal(out[1], vr)


def test_arguments_that_do_not_fit_are_refused():
    import torch

    W = _W()
    g = rng_for(107, "refuse")
    _, packed, s, z = random_weight(g, 64, 256, 4, 64)
    wq = _qweight(W, 4, 64, packed, s, z)
    x = torch.zeros(3, 256, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="qweight"):
        W.qgemv(wq, x[:, :128].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        W.qgemv(wq, torch.zeros(3, 512, device="cuda", dtype=torch.bfloat16)[:, ::2])
    with pytest.raises(TypeError):
        W.qgemv(wq, x.half())
    with pytest.raises(ValueError, match="Y"):
        W.qgemv(wq, x, Y=torch.zeros(3, 64, device="cuda"))
    with pytest.raises(W.QwhaError) as e:
        W.qgemv(wq, torch.zeros(65, 256, device="cuda", dtype=torch.bfloat16))
    assert e.value.status == 3
    assert W.qgemv(wq, x[:0]).shape == (0, 64)
    c = W.cache_alloc(2, 8, 2, 64)
    rows = torch.zeros(3, 2, 64, device="cuda")
    slots = torch.arange(3, device="cuda")
    with pytest.raises(ValueError, match="slots"):
        W.cache_write(c, rows, slots.int())
    with pytest.raises(ValueError, match="rows"):
        W.cache_write(c, rows[:, :1], slots)
    with pytest.raises(ValueError, match="one or two"):
        W.cache_write((c, c), rows, slots)
    with pytest.raises(ValueError, match="row_start"):
        W.cache_read(c, torch.zeros(1, 1, device="cuda", dtype=torch.int32), torch.zeros(3, device="cuda").long(), 4)
    W.cache_write(c, rows[:0], slots[:0])


def test_a_decode_step_uses_them_together():
    """Three steps of a small attention layer: adapted q, k, v projections, keys and values into the cache, the
    sequences read back, attention over them, the adapted output projection. Against the same layer in fp64 on the
    cache's own (quantized) contents."""
    import torch

    W = _W()
    g = rng_for(108, "step")
    B, d, heads, hd, page = 3, 256, 4, 64, 4
    layers = {}
    for name in "qkvo":
        q, packed, s, z = random_weight(g, d, d, 4, 64)
        rp, ci, cf = random_pattern(d, d, counts=g.integers(0, 30, d), rng=g, coef_scale=0.05)
        F = np.zeros((d, d))
        F[oracle.csr_rows(rp), ci] = cf
        w = dense_weight(q, s, z, 64) + 0.5 * butterflies(F, d)
        a = W.Adapter(d, d, d, ci.size, to_dev(rp), to_dev(ci), to_dev(cf))
        layers[name] = (a, _qweight(W, 4, 64, packed, s, z), w)
    proj = lambda n, t: W.adapter_decode(layers[n][0], t, 0.5, layers[n][1])  # noqa: E731
    kv = (W.cache_alloc(8, page, heads, hd, 4, 32, 64), W.cache_alloc(8, page, heads, hd, 8, 64, 0))
    table = to_dev(np.array([[5, 1], [0, 7], [3, 2]], np.int32))
    lens = np.array([0, 2, 3])
    for step in range(3):
        x = round_to(g.standard_normal((B, d)), "bf16")
        xd = _dev(x, "bf16")
        qh, kh, vh = proj("q", xd), proj("k", xd), proj("v", xd)
        tab = table.cpu().numpy()
        slots = np.array([tab[b, lens[b] // page] * page + lens[b] % page for b in range(B)], np.int64)
        W.cache_write(kv, (kh.view(B, heads, hd), vh.view(B, heads, hd)), to_dev(slots))
        lens = lens + 1
        starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        ks, vs = W.cache_read(kv, table, to_dev(starts), int(starts[-1]))
        outs = []
        for b in range(B):
            k, v = (t[starts[b]:starts[b + 1]].float() for t in (ks, vs))
            att = torch.softmax(torch.einsum("hd,thd->ht", qh[b].float().view(heads, hd), k) / hd**0.5, -1)
            outs.append(torch.einsum("ht,thd->hd", att, v).reshape(d))
        mix = torch.stack(outs).to(torch.bfloat16)
        y = proj("o", mix)
        # the same in fp64, projections from the definition, keys and values as the cache holds them
        for n, t, got in (("q", host(xd), qh), ("k", host(xd), kh), ("v", host(xd), vh), ("o", host(mix), y)):
            want = t @ layers[n][2].T
            assert np.linalg.norm(host(got) - want) <= 2.0**-8 * np.linalg.norm(want)
        for c, rows, new in ((kv[0], ks, kh), (kv[1], vs, vh)):
            codes, s, z = _state(c)
            q2, s2, z2 = quantize(host(new).reshape(B, heads, hd).astype(np.float32), c.bits, c.group, c.had_block,
                                  "bf16")
            assert np.array_equal(codes[slots], pack(q2, c.bits)) and np.array_equal(s[slots], s2)
            assert np.array_equal(unpack(codes[slots], c.bits), q2) and np.array_equal(z[slots], z2)
            back = butterflies(values(codes[slots], s[slots], z[slots], c.bits, c.group), c.had_block)
            last = host(rows)[starts[1:] - 1]
            assert np.all(np.abs(last - back) <= 2.0**-8 * 1.01 * np.abs(back) + 1e-5 * np.abs(back).max())
