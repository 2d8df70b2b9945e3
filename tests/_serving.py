"""Plain statements of the serving operators for the tests (numpy, from the formulas)."""

import numpy as np

from workloads import bf16_bits_to_f32, f32_to_bf16_bits, pack_codes

HALF = 0.5 + 2.0**-12


def round_to(x, dtype):
    x = np.asarray(x, dtype=np.float32)
    return bf16_bits_to_f32(f32_to_bf16_bits(x)).reshape(x.shape) if dtype == "bf16" else x


def half_step(dtype):
    """Largest relative error of one rounding to the type."""
    return 2.0**-8 if dtype == "bf16" else 2.0**-24


def random_weight(g, d_out, d_in, bits, group, zero_top=None):
    """(codes, packed, scales, zeros): any codes, positive and negative scales, zero points up to zero_top."""
    q = g.integers(0, 2**bits, (d_out, d_in)).astype(np.uint8)
    s = (g.standard_normal((d_out, d_in // group)) * 0.02).astype(np.float32)
    z = g.integers(0, (2**bits if zero_top is None else zero_top + 1), (d_out, d_in // group)).astype(np.uint8)
    return q, pack_codes(q, bits), s, z


def dense_weight(q, s, z, group):
    rep = lambda a: np.repeat(a.astype(np.float64), group, axis=1)  # noqa: E731
    return rep(s) * (q.astype(np.float64) - rep(z))


def butterflies(x, n):
    """x H_n block by block along the last axis in x's own type: stages 1, 2, 4, ..., then the factor 1/sqrt(n)."""
    if not n:
        return x
    shape, h = x.shape, 1
    while h < n:
        y = x.reshape(-1, 2, h)
        x = np.stack((y[:, 0] + y[:, 1], y[:, 0] - y[:, 1]), axis=1)
        h *= 2
    return x.reshape(shape) * x.dtype.type(1.0 / np.sqrt(float(n)))


def quantize(rows, bits, group, had_block, dtype):
    """(codes, scales, zeros) of rows [..., head_dim] by the documented rule: fp32 for bf16 rows, fp64 for fp32 rows."""
    t = np.float32 if dtype == "bf16" else np.float64
    with np.errstate(all="ignore"):
        v = butterflies(rows.astype(t), had_block)
        v = v.reshape(*v.shape[:-1], -1, group)
        lo = np.minimum(v.min(-1), t(0))
        hi = np.maximum(v.max(-1), t(0))
        top = t(2**bits - 1)
        s = ((hi - lo) * (t(1) / top)).astype(np.float32)
        bad = ~np.isfinite(s) | np.isnan(v).any(-1)
        s = np.where(s < np.float32(2.0**-126), np.float32(1), s)
        inv = t(1) / s.astype(t)
        z = np.minimum(np.floor(-lo * inv + t(HALF)), top)
        q = np.clip(np.floor(v * inv[..., None] + (z + t(HALF))[..., None]), t(0), top)
    s = np.where(bad, np.float32(np.nan), s)
    z = np.where(bad, 0, z).astype(np.uint8)
    q = np.where(bad[..., None], 0, q).astype(np.uint8)
    return q.reshape(rows.shape), s, z


def pack(q, bits):
    return pack_codes(q.reshape(-1, q.shape[-1]), bits).reshape(*q.shape[:-1], -1)


def unpack(codes, bits):
    flat = codes.reshape(-1, codes.shape[-1])
    b = np.unpackbits(flat, axis=1, bitorder="little").reshape(flat.shape[0], -1, bits)
    q = (b.astype(np.int64) << np.arange(bits)).sum(-1)
    return q.reshape(*codes.shape[:-1], -1)


def values(codes, s, z, bits, group):
    """s (q - z) in fp64."""
    rep = lambda a: np.repeat(a.astype(np.float64), group, axis=-1)  # noqa: E731
    return rep(s) * (unpack(codes, bits) - rep(z))
