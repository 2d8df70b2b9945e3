"""The serving operators at the ends of their ranges: values and zero points that a documented call may hold and that
ordinary inputs do not."""

import numpy as np
import pytest

from _serving import dense_weight, half_step, random_weight, round_to
from _util import host, to_dev
from test_serving_gpu import (_W, _check_base, _check_decode, _decode_case, _dev, _filled,
                              _qweight, _sum_tol, _want_read)
from workloads import pack_codes, rng_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 6, 8, 24])
@pytest.mark.parametrize("bits,group", [(4, 128), (3, 64), (2, 32), (4, 8)])
def test_qgemv_columns_of_tiny_values(bits, group, T, dtype):
    """128 neighbouring columns whose largest value is the smallest normal number, twice that, or a denormal, by
    themselves and beside ordinary ones. With scales of 2^100 the tiny columns' sums are ordinary numbers, held to the
    precision of any other."""
    W = _W()
    g = rng_for(120, "tiny", bits, group, T)
    q, packed, s, z = random_weight(g, 40, 384, bits, group)
    s = (s * np.float32(2.0**100)).astype(np.float32)
    wq, w = _qweight(W, bits, group, packed, s, z), dense_weight(q, s, z, group)
    for top in (2.0**-125, 2.0**-126, 2.0**-130 if dtype == "bf16" else 2.0**-140):
        for beside in (False, True):
            x = g.standard_normal((T, 384)).astype(np.float32) if beside else np.zeros((T, 384), np.float32)
            x[:, 128:256] = g.uniform(-1, 1, (T, 128)) * top
            x[:, 130] = top
            x[0, 128:256] = 0.0
            x[0, 200] = -top  # one value among zeros
            x = round_to(x, dtype)
            _check_base(W.qgemv(wq, _dev(x, dtype)), x.astype(np.float64), w, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 3, 24])
def test_adapter_decode_columns_of_tiny_values(T, dtype):
    W = _W()
    d_in, d_out, n = 512, 40, 128
    g = rng_for(121, "tiny decode", T)
    rp, ci, cf, q, packed, s, z, x = _decode_case(g, d_in, d_out, n, 4, 128, g.integers(0, 40, d_out), T, dtype)
    s = (s * np.float32(2.0**100)).astype(np.float32)
    a = W.Adapter(d_in, d_out, n, ci.size, to_dev(rp), to_dev(ci), to_dev(cf))
    for top in (2.0**-125, 2.0**-126, 2.0**-130):
        y = x.copy()
        y[:, 128:256] = round_to(y[:, 128:256] * np.float32(top / 8), dtype)
        y[:, 140] = top
        Y = W.adapter_decode(a, _dev(y, dtype), 0.75, _qweight(W, 4, 128, packed, s, z))
        _check_decode(Y, y, dense_weight(q, s, z, 128), rp, ci, cf, n, 0.75, dtype)


@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("shape", [(3, 128, 128), (3, 128, 64), (4, 64, 32), (1, 80, 40)])
def test_cache_read_any_zero_point(shape, bits):
    """Zero points are bytes of any value, as the weight's are: also above the largest code and above 128."""
    import torch

    W = _W()
    heads, head_dim, group = shape
    g = rng_for(122, "zeros", *shape, bits)
    for had_block in [n for n in (0, 2, 16, 32, 64, 128) if n == 0 or head_dim % n == 0]:
        c = _filled(W, g, 6, 16, heads, head_dim, bits, group, had_block)
        z = g.integers(0, 256, tuple(c.zeros.shape)).astype(np.uint8)
        z[0], z[1], z[2], z[3] = 255, 128, 129, 2**bits - 1  # page by page
        c.zeros.copy_(to_dev(z))
        c.codes[0].zero_()  # codes of 0 under zero points of 255: the largest sums there are
        table = np.arange(6, dtype=np.int32)[None]
        out = W.cache_read(c, to_dev(table), to_dev(np.array([0, 96], np.int64)), 96, dtype=torch.float32)
        want, mag = _want_read(c, bits, group, had_block, table, [0], [96], 16)
        n = had_block or 1
        blk = np.repeat(mag.reshape(96, heads, -1, n).sum(-1) / np.sqrt(n), n, axis=-1)
        tol = half_step("f32") * 1.01 * np.abs(want) + (np.log2(n) + 3) * 2.0**-24 * blk + 1e-30
        err = np.abs(host(out) - want)
        assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 6, 8, 24, 64])
@pytest.mark.parametrize("bits,group", [(4, 128), (3, 64), (2, 32), (4, 8)])
def test_qgemv_values_near_the_largest(bits, group, T, dtype):
    """Values near the type's largest: a group's sum is beyond fp32's range before its scale, the result is not."""
    W = _W()
    g = rng_for(124, "huge", bits, group, T)
    q, packed, s, z = random_weight(g, 40, 512, bits, group)
    s = (s * np.float32(1e-4)).astype(np.float32)
    wq, w = _qweight(W, bits, group, packed, s, z), dense_weight(q, s, z, group)
    x = round_to(g.uniform(0.5, 1.0, (T, 512)) * 3e38, dtype)
    x[T // 2] = round_to(g.standard_normal(512), dtype)  # an ordinary token among them
    _check_base(W.qgemv(wq, _dev(x, dtype)), x.astype(np.float64), w, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 6, 8, 20, 24])
@pytest.mark.parametrize("bits,group", [(4, 128), (3, 64), (2, 32), (4, 8), (3, 256)])
def test_qgemv_values_on_zero_weights_vanish(bits, group, T, dtype):
    """Values of 1e5 whose weight is zero (code = zero point) add nothing: the sum over the other columns is held as if
    they were not there. fp32 sums of d_in products, and a value below 2^-24 of the largest among its 128 columns is
    held to 2^-32 of that."""
    W = _W()
    g = rng_for(123, "vanish", bits, group, T)
    q, packed, s, z = random_weight(g, 48, 512, bits, group, zero_top=None if bits == 3 else 255)
    z[:, [5 // group, 300 // group]] %= 2**bits
    q[:, [5, 300]] = z[:, [5 // group, 300 // group]]
    packed = pack_codes(q, bits)
    w = dense_weight(q, s, z, group)
    assert not w[:, [5, 300]].any()
    x = round_to(g.standard_normal((T, 512)), dtype)
    x[:, 5], x[:, 300] = round_to(np.array([1e5, -98765.0]), dtype)
    want = x.astype(np.float64) @ w.T
    top = np.repeat(np.abs(x).reshape(T, -1, 128).max(-1), 128, axis=-1)
    low = np.where(np.abs(x) < 2.0**-24 * top, 2.0**-32 * top, 0.0)
    live = np.abs(x) * (np.abs(x) < 100)
    tol = half_step(dtype) * 1.01 * np.abs(want) + (_sum_tol(512) * live + low) @ np.abs(w).T
    err = np.abs(host(W.qgemv(_qweight(W, bits, group, packed, s, z), _dev(x, dtype))) - want)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 8, 9])
@pytest.mark.parametrize("n_entries", [20, 400, 1500])
def test_adapter_decode_infinities_stay_in_their_block(n_entries, T, dtype):
    """An infinity or a NaN reaches, of the adapter's sums, the rows with an entry in its Hadamard block; others keep
    their value, whatever their length, and columns outside the layer are skipped."""
    W = _W()
    d_in, d_out, n = 4096, 40, 1024
    g = rng_for(125, "block", n_entries)
    F = np.zeros((d_out, d_in), np.float32)
    for i in range(d_out):
        lo = 0 if i % 4 == 0 else 1024  # every fourth row has entries in the first block
        k = max(1, n_entries - 3 * i)
        F[i, lo + g.permutation(d_in - lo)[:k]] = g.standard_normal(k) * 0.05 + 0.2
        if i % 4 == 0:
            F[i, 17] = 0.25
    rows, ci = np.nonzero(F)
    cf = F[rows, ci]
    rp = np.concatenate([[0], np.cumsum(np.bincount(rows, minlength=d_out))]).astype(np.int32)
    ci = ci.astype(np.int32)
    last = rp[1:] - 1
    ci[last[1]], ci[last[2]] = -1, d_in + 5  # outside: skipped
    a = W.Adapter(d_in, d_out, n, ci.size, to_dev(rp), to_dev(ci), to_dev(cf))
    x = round_to(g.standard_normal((T, d_in)), dtype)
    clean = host(W.adapter_decode(a, _dev(x, dtype), 0.5))
    y = x.copy()
    y[T // 2, 3], y[T - 1, 700] = np.inf, np.nan
    got = host(W.adapter_decode(a, _dev(y, dtype), 0.5))
    assert np.all(np.isfinite(clean))
    whole = [t for t in range(T) if t not in (T // 2, T - 1)]
    assert np.array_equal(got[whole], clean[whole])
    touched = np.arange(d_out) % 4 == 0
    assert np.array_equal(got[:, ~touched], clean[:, ~touched])
    assert not np.any(np.isfinite(got[[T // 2, T - 1]][:, touched]))


def test_validate_slots_names_the_first_failure():
    """The first row whose slot is outside the cache or is another row's too, the same on every call."""
    W = _W()
    c = W.cache_alloc(1024, 64, 1, 64)
    g = rng_for(126, "slots")
    for outside, pairs in (((), 11), ((60000, 64000), 5), ((9, 10), 5), ((40000,), 0)):
        s = g.permutation(65536).astype(np.int64)
        s[::50] = -1
        for i in range(pairs):
            s[1001 + 700 * i] = s[64999 - 600 * i]
        s[list(outside)] = [-2, 65536][:len(outside)]
        first = min(list(outside) + ([1001] if pairs else []))
        text = "outside" if first in outside else "twice"
        for _ in range(20):
            with pytest.raises(W.QwhaError, match=rf"{text}.*\(at {first}\)"):
                W.validate_slots(c, to_dev(s))
    W.validate_slots(c, to_dev(g.permutation(65536).astype(np.int64)))


def test_what_the_kernels_met_is_reported_through_the_package():
    import torch

    W = _W()
    c = W.cache_alloc(2, 4, 2, 64)
    W.check_stream_status()
    W.cache_write(c, torch.ones(3, 2, 64, device="cuda"), to_dev(np.array([1, 8, -1], np.int64)))
    with pytest.raises(W.QwhaError, match="slot") as e:
        W.check_stream_status()
    assert e.value.status == 1
    W.check_stream_status()  # the report is cleared
    out = torch.full((8, 2, 64), 7.5, device="cuda")
    W.cache_read(c, to_dev(np.array([[0, 2]], np.int32)), to_dev(np.array([0, 8], np.int64)), 8, out=out)
    with pytest.raises(W.QwhaError, match="page"):
        W.check_stream_status()
    assert torch.allclose(out[1], torch.ones(2, 64, device="cuda"), rtol=1e-6) and torch.all(out[4:] == 7.5)
    W.check_stream_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d_in,n,T", [(40960, 8192, 3), (51200, 2048, 2), (65536, 32768, 1), (65536, 32768, 3)])
def test_adapter_decode_wide_inputs(d_in, n, T, dtype):
    """Inputs whose Z of one token fills shared memory (no room for a second one, then none for entries) or does not fit
    there; the largest Hadamard block."""
    W = _W()
    g = rng_for(127, "wide", d_in, T)
    d_out = 24
    counts = g.integers(0, 300, d_out)
    counts[0], counts[1], counts[2], counts[-1] = 0, 3000, 700, 1
    rp, ci, cf, q, packed, s, z, x = _decode_case(g, d_in, d_out, n, 4, 128, counts, T, dtype)
    a = W.Adapter(d_in, d_out, n, ci.size, to_dev(rp), to_dev(ci), to_dev(cf))
    Y = W.adapter_decode(a, _dev(x, dtype), 0.75, _qweight(W, 4, 128, packed, s, z))
    _check_decode(Y, x, dense_weight(q, s, z, 128), rp, ci, cf, n, 0.75, dtype)
    _check_decode(W.adapter_decode(a, _dev(x, dtype), -1.5), x, None, rp, ci, cf, n, -1.5, dtype)


def test_stage_report_counts_the_launches_of_a_pair():
    """Caches that need different kernels take a launch each."""
    import torch

    W = _W()
    wide = [W.cache_alloc(2, 4, 2, 64, 4, 64, 64) for _ in range(2)]
    odd = [W.cache_alloc(2, 4, 2, 24, 4, 8, 8) for _ in range(2)]
    slots = to_dev(np.arange(5, dtype=np.int64))
    where = (to_dev(np.array([[0, 1]], np.int32)), to_dev(np.array([0, 5], np.int64)), 5)
    rows = lambda pair: [torch.ones(5, 2, c.head_dim, device="cuda", dtype=torch.bfloat16) for c in pair]  # noqa: E731
    W.stage_timing(True)
    try:
        W.stage_report()
        for pair, launches in ((wide[0], odd[0]), 2), ((odd[0], wide[0]), 2), (wide, 1), (odd, 1):
            W.cache_write(pair, rows(pair), slots)
            W.cache_read(pair, *where)
            rep = W.stage_report()
            assert rep["cache_write"][:2] == (1, launches) and rep["cache_read"][:2] == (1, launches)
        W.cache_write((wide[0], odd[0]), [r.float() for r in rows((wide[0], odd[0]))], slots)  # one kernel for fp32 rows
        assert W.stage_report()["cache_write"][:2] == (1, 1)
    finally:
        W.stage_timing(False)
