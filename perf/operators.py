"""Cases of the serving operators: the quantized matrix-vector product (`qgemv`), the adapted layer on a few tokens
(`adapter_decode`) and the quantized key/value cache (`cache_write`, `cache_read`).

`run` computes each operator in its plain form (elementary torch operations in fp32), or, with `own` set, through the
package's entry points. Sizes are the layer shapes of the workload table (LLaMA-3-8B-shaped linears and the q_proj
layer, LoRA r=64 budgets, 2/3/4-bit codes in groups of 32..128) and generic ones.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ALPHA = 0.75


# ---------------------------------------------------------------- cases


def _gemv(name, d_out, d_in, bits, group, T, dtype):
    return dict(name=name, op="qgemv", d_out=d_out, d_in=d_in, bits=bits, group=group, T=T, dtype=dtype)


def _decode(name, d_out, d_in, had_block, bits, group, T, dtype, r=64):
    return dict(name=name, op="adapter_decode", d_out=d_out, d_in=d_in, had_block=had_block, bits=bits, group=group,
                T=T, dtype=dtype, p=r * (d_out + d_in))


def _append(name, seqs, past, new, heads, head_dim, bits, group, had_block, page_size, dtype):
    return dict(name=name, op="cache_append", seqs=seqs, past=past, new=new, heads=heads, head_dim=head_dim, bits=bits,
                group=group, had_block=had_block, page_size=page_size, dtype=dtype)


def _read(name, seqs, longest, heads, head_dim, bits, group, had_block, page_size, dtype):
    return dict(name=name, op="cache_read", seqs=seqs, longest=longest, heads=heads, head_dim=head_dim, bits=bits,
                group=group, had_block=had_block, page_size=page_size, dtype=dtype)


def listed():
    return [
        # one token through a key projection: the smallest product, launch latency counts
        _gemv("gemv_k_proj_t1", 1024, 4096, 4, 128, 1, "bf16"),
        # one token through an MLP up projection: the ordinary step of a single stream
        _gemv("gemv_up_t1", 14336, 4096, 3, 128, 1, "bf16"),
        # eight streams through the MLP's down projection: the long reduction
        _gemv("gemv_down_t8", 4096, 14336, 4, 128, 8, "bf16"),
        # odd row count, a width that ends inside every tile, small groups, 2-bit codes, fp32 activations
        _gemv("gemv_odd_f32_t3", 2731, 4000, 2, 32, 3, "f32"),
        # the widest batch the operator takes, on the largest layer
        _gemv("gemv_gate_t64", 14336, 4096, 4, 128, 64, "bf16"),
        # one token through the adapted q_proj layer
        _decode("decode_q_proj_t1", 4096, 4096, 4096, 4, 128, 1, "bf16"),
        # five tokens through the adapted down projection (seven Hadamard blocks), 2-bit base, fp32 activations
        _decode("decode_down_f32_t5", 4096, 14336, 2048, 2, 64, 5, "f32"),
        # sixteen streams through the adapted gate projection
        _decode("decode_gate_t16", 14336, 4096, 4096, 4, 128, 16, "bf16"),
        # a decode step of 64 streams: each appends one token, and the attention reads that token's row back
        _append("append_decode", 64, 1500, 1, 8, 128, 4, 128, 128, 16, "bf16"),
        # prefill of 8 x 4096 tokens, rotated heads, read back as the attention sees them
        _append("append_prefill", 8, 0, 4096, 8, 128, 4, 64, 128, 64, "bf16"),
        # a few short ragged sequences, odd head length, no rotation, 3-bit codes, fp32 rows
        _read("read_ragged_f32", 5, 700, 6, 80, 3, 40, 0, 16, "f32"),
        # long contexts: 8 ragged sequences of up to 32768 tokens
        _read("read_long", 8, 32768, 8, 128, 4, 128, 128, 64, "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qgemv", "adapter_decode", "cache_append", "cache_read"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "qgemv":
        group = rng.choice([8, 32, 64, 128, 128])
        d_in = group * _log(rng, max(1, 256 // group), 14336 // group)
        d_out = _log(rng, 64, min(14336, 14336 * 4096 // d_in))
        return dict(op=op, d_out=d_out, d_in=d_in, bits=rng.choice([2, 3, 4, 4]), group=group, T=_log(rng, 1, 64),
                    dtype=dtype)
    if op == "adapter_decode":
        n = rng.choice([64, 256, 1024, 2048, 4096])
        d_in = n * rng.randint(1, min(7, max(1, 14336 // n)))
        d_out = 8 * _log(rng, 8, min(1792, 14336 * 512 // d_in))
        group = rng.choice([32, 64, 64, 128])
        group = group if d_in % group == 0 else 64
        r = rng.choice([4, 16, 64])
        return dict(op=op, d_out=d_out, d_in=d_in, had_block=n, bits=rng.choice([2, 3, 4, 4]), group=group,
                    T=_log(rng, 1, 16), dtype=dtype, p=min(r * (d_out + d_in), d_out * d_in // 2))
    head_dim, group, had_block = rng.choice([(64, 64, 64), (64, 32, 0), (80, 40, 16), (96, 96, 32), (128, 128, 128),
                                             (128, 64, 128), (128, 32, 0), (256, 64, 256), (256, 256, 0)])
    heads = rng.choice([1, 2, 3, 8, 8])
    bits = rng.choice([2, 3, 4, 4, 8])
    page_size = rng.choice([1, 16, 16, 64, 100])
    if op == "cache_append":
        total = _log(rng, 1, 32768 * 1024 // (heads * head_dim))
        seqs = _log(rng, 1, min(total, 64))
        return dict(op=op, seqs=seqs, past=rng.choice([0, 37, 900]), new=min(4096, max(1, total // seqs)), heads=heads,
                    head_dim=head_dim, bits=bits, group=group, had_block=had_block, page_size=page_size, dtype=dtype)
    seqs = _log(rng, 1, 64)
    longest = _log(rng, 1, min(32768, 8 * 32768 * 1024 // (2 * seqs * heads * head_dim)))
    return dict(op=op, seqs=seqs, longest=longest, heads=heads, head_dim=head_dim, bits=bits, group=group,
                had_block=had_block, page_size=page_size, dtype=dtype)


# ---------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _pack(q, bits):
    """Codes (uint8, last dimension a multiple of 8) to their little-endian bit stream."""
    if bits == 8:
        return q.contiguous()
    run = q.reshape(*q.shape[:-1], -1, 8).to(torch.int32)
    word = (run << (bits * torch.arange(8, device=q.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    by = (word[..., None] >> (8 * torch.arange(bits, device=q.device, dtype=torch.int32))) & 255
    return by.to(torch.uint8).reshape(*q.shape[:-1], q.shape[-1] * bits // 8)


def _weight(g, d_out, d_in, bits, group):
    """A round-to-nearest quantized weight: normal values with a few outliers, as the base weights of the layers."""
    w = torch.randn(d_out, d_in, generator=g, device=DEV).mul_(0.02)
    w = torch.where(torch.rand(d_out, d_in, generator=g, device=DEV) < 0.001, w * 20, w).view(d_out, -1, group)
    mn, mx = w.amin(-1, keepdim=True), w.amax(-1, keepdim=True)
    top = 2**bits - 1
    s = (mx - mn) / top
    z = torch.round(-mn / s).clamp_(0, top)
    q = (torch.round(w / s) + z).clamp_(0, top).to(torch.uint8).view(d_out, d_in)
    return _pack(q, bits), s.squeeze(-1).contiguous(), z.squeeze(-1).to(torch.uint8).contiguous()


def _tokens(g, T, d_in, dtype):
    """Activations with 1 % outlier channels."""
    x = torch.randn(T, d_in, generator=g, device=DEV)
    big = torch.rand(d_in, generator=g, device=DEV) < 0.01
    return torch.where(big, x * 20, x).to(DTYPES[dtype])


def _pattern(g, d_out, d_in, p):
    """E by rows: budgets that follow a skewed error norm, at least two entries a row, distinct ascending columns."""
    e = torch.exp(torch.randn(d_out, generator=g, device=DEV))
    least = min(2, p // d_out)
    b = least + torch.floor((p - least * d_out) * (e / e.sum())).long()
    b = b.clamp_(max=d_in)
    key = torch.rand(d_out, d_in, generator=g, device=DEV)
    last = key.sort(1).values.gather(1, (b - 1).clamp_(min=0)[:, None])
    mask = (key <= last) & (b > 0)[:, None]
    row_ptr = torch.zeros(d_out + 1, dtype=torch.int32, device=DEV)
    row_ptr[1:] = mask.sum(1).cumsum(0)
    col = mask.nonzero()[:, 1].to(torch.int32)
    coef = torch.randn(col.numel(), generator=g, device=DEV).mul_(0.03)
    return row_ptr, col, coef


def _pool(g, c, n_pages):
    """A cache pool that earlier tokens have filled: codes, scales and zero points of every slot."""
    rows = (n_pages, c["page_size"], c["heads"])
    codes = torch.randint(0, 256, rows + (c["head_dim"] * c["bits"] // 8,), generator=g, device=DEV, dtype=torch.uint8)
    ng = c["head_dim"] // c["group"]
    top = 2 ** c["bits"] - 1
    scales = (3.0 + 3.0 * torch.rand(rows + (ng,), generator=g, device=DEV)) / top
    zeros = torch.randint(top // 3, (2 * top) // 3 + 1, rows + (ng,), generator=g, device=DEV, dtype=torch.uint8)
    return [codes, scales, zeros]


def _paged(g, lens, page_size):
    """A page table of shuffled pages for sequences of these lengths, the page count, and slots of all positions."""
    need = (lens + page_size - 1) // page_size
    width = int(need.max())
    order = torch.randperm(int(need.sum()), generator=g, device=DEV).to(torch.int32)
    at = torch.cumsum(need, 0) - need
    j = torch.arange(width, device=DEV)
    idx = (at[:, None] + j).clamp_(max=max(order.numel() - 1, 0))
    table = torch.where(j < need[:, None], order[idx], torch.full_like(order[idx], -1)).contiguous()
    return table, order.numel()


def _lengths(c):
    """(tokens a sequence holds before the rows of this pass, rows of this pass) per sequence: ragged, spread over
    [0, past] and [longest / 2, longest] by multiples of the golden section."""
    at = [(i + 1) * 0.6180339887 % 1.0 for i in range(c["seqs"])]
    if c["op"] == "cache_append":
        return [int(u * (c["past"] + 1)) for u in at], [c["new"]] * c["seqs"]
    return [0] * c["seqs"], [max(1, c["longest"] - int(u * (c["longest"] // 2 + 1))) for u in at]


def _starts(lens):
    s = torch.zeros(lens.numel() + 1, dtype=torch.int64, device=DEV)
    s[1:] = torch.cumsum(lens, 0)
    return s


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    st = {"case": c}
    if c["op"] in ("qgemv", "adapter_decode"):
        st["w"] = _weight(g, c["d_out"], c["d_in"], c["bits"], c["group"])
        st["x"] = _tokens(g, c["T"], c["d_in"], c["dtype"])
        if c["op"] == "adapter_decode":
            st["e"] = _pattern(g, c["d_out"], c["d_in"], c["p"])
        return st
    B = c["seqs"]
    first, count = (torch.tensor(v, dtype=torch.int64, device=DEV) for v in _lengths(c))
    st["table"], n_pages = _paged(g, first + count, c["page_size"])
    st["first"], st["starts"], st["rows"] = first, _starts(count), sum(_lengths(c)[1])
    st["k"], st["v"] = _pool(g, c, n_pages), _pool(g, c, n_pages)
    if c["op"] == "cache_append":
        st["slots"] = _slots(st["table"], first, st["starts"], st["rows"], c["page_size"])
        shape = (st["rows"], c["heads"], c["head_dim"])
        k = torch.randn(shape, generator=g, device=DEV)  # keys have a few large channels, values are plain
        k *= torch.where(torch.rand(shape[1:], generator=g, device=DEV) < 0.05, 8.0, 1.0)
        st["kx"] = k.to(DTYPES[c["dtype"]])
        st["vx"] = torch.randn(shape, generator=g, device=DEV).to(DTYPES[c["dtype"]])
    return st


# ---------------------------------------------------------------- one pass


def _slots(table, first, starts, rows, page_size):
    """The slot of each packed row of the sequences."""
    i = torch.arange(rows, device=DEV)
    b = torch.searchsorted(starts, i, right=True) - 1
    pos = first[b] + i - starts[b]
    return table[b, pos // page_size].long() * page_size + pos % page_size


def _codes(packed, bits):
    """The codes of a little-endian bit stream, one int32 each."""
    if bits == 8:
        return packed.to(torch.int32)
    by = packed.reshape(*packed.shape[:-1], -1, bits).to(torch.int32)
    word = (by << (8 * torch.arange(bits, device=by.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    q = (word[..., None] >> (bits * torch.arange(8, device=by.device, dtype=torch.int32))) & (2**bits - 1)
    return q.reshape(*packed.shape[:-1], packed.shape[-1] * 8 // bits)


def _values(packed, scales, zeros, bits, group):
    """scales * (code - zero) in fp32."""
    q = _codes(packed, bits)
    q = q.view(*q.shape[:-1], -1, group)
    return (scales[..., None] * (q - zeros[..., None].to(torch.int32)).float()).flatten(-2)


def _rotate(x, n):
    """x H for blocks of n along the last dimension, in x's type: the stages 1, 2, 4, ..., then the factor 1/sqrt(n)."""
    if not n:
        return x
    shape, h = x.shape, 1
    while h < n:
        x = x.reshape(-1, 2, h)
        x = torch.stack((x[:, 0] + x[:, 1], x[:, 0] - x[:, 1]), 1)
        h *= 2
    return x.reshape(shape) * (1.0 / math.sqrt(n))


def _quantize(v, bits, group):
    """Codes, scales and zero points of rows: a range that holds zero, in 2^bits - 1 steps of the fp32 scale. Values
    half-way between two codes, which bf16 rows hit often, go up: the border lies 2^-12 of a step below the half."""
    top, half = 2**bits - 1, 0.5 + 2.0**-12
    v = v.view(*v.shape[:-1], -1, group)
    mn, mx = v.amin(-1).clamp(max=0.0), v.amax(-1).clamp(min=0.0)
    s = ((mx - mn) * (1.0 / top)).float()
    s = torch.where(s < 2.0**-126, torch.ones_like(s), s)
    inv = torch.reciprocal(s.to(v.dtype))
    z = torch.floor(-mn * inv + half).clamp(0, top)
    q = torch.floor(v * inv[..., None] + (z + half)[..., None]).clamp(0, top)
    return q.to(torch.uint8).flatten(-2), s, z.to(torch.uint8)


def _plain_write(pool, rows, slots, c):
    # fp32 rows are quantized in fp64: a code next to a border decides a step, far more than fp32 carries
    wide = rows.double() if c["dtype"] == "f32" else rows.float()
    q, s, z = _quantize(_rotate(wide, c["had_block"]), c["bits"], c["group"])
    codes, scales, zeros = (t.flatten(0, 1) for t in pool)
    codes[slots] = _pack(q, c["bits"])
    scales[slots] = s
    zeros[slots] = z


def _plain_read(pool, st, c):
    slots = _slots(st["table"], st["first"], st["starts"], st["rows"], c["page_size"])
    codes, scales, zeros = (t.flatten(0, 1)[slots] for t in pool)
    v = _values(codes, scales, zeros, c["bits"], c["group"])
    return _rotate(v, c["had_block"]).to(DTYPES[c["dtype"]])


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_plain(st):
    c = st["case"]
    if c["op"] in ("qgemv", "adapter_decode"):
        x = st["x"].float()
        y = x @ _values(*st["w"], c["bits"], c["group"]).T
        if c["op"] == "adapter_decode":
            row_ptr, col, coef = st["e"]
            row = torch.repeat_interleave(torch.arange(c["d_out"], device=DEV), row_ptr.diff().long(),
                                          output_size=col.numel())
            F = torch.zeros(c["d_out"], c["d_in"], device=DEV)
            F[row, col.long()] = coef
            y = y + ALPHA * (_rotate(x, c["had_block"]) @ F.T)
        return y.to(st["x"].dtype)
    if c["op"] == "cache_append":
        _plain_write(st["k"], st["kx"], st["slots"], c)
        _plain_write(st["v"], st["vx"], st["slots"], c)
    out = [_plain_read(st["k"], st, c), _plain_read(st["v"], st, c)]
    if c["op"] == "cache_append":
        out += [st["k"][1], st["v"][1], st["k"][2], st["v"][2]]
    return out


def _run_own(st):
    import walsh_hadamard_sparse_b200 as W

    c = st["case"]
    if c["op"] == "qgemv":
        return W.qgemv(W.QWeight(c["bits"], c["group"], *st["w"]), st["x"])
    if c["op"] == "adapter_decode":
        row_ptr, col, coef = st["e"]
        a = W.Adapter(c["d_in"], c["d_out"], c["had_block"], col.numel(), row_ptr, col, coef)
        return W.adapter_decode(a, st["x"], ALPHA, W.QWeight(c["bits"], c["group"], *st["w"]))
    kv = tuple(W.QCache(c["bits"], c["group"], c["had_block"], *st[t]) for t in ("k", "v"))
    if c["op"] == "cache_append":
        W.cache_write(kv, (st["kx"], st["vx"]), st["slots"])
    out = list(W.cache_read(kv, st["table"], st["starts"], st["rows"], first=st["first"], dtype=DTYPES[c["dtype"]]))
    if c["op"] == "cache_append":
        out += [st["k"][1], st["v"][1], st["k"][2], st["v"][2]]
    return out


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_codes(packed, bits):
    """Codes of a row's bit stream, bit by bit: code k is bits [bits k, bits k + bits)."""
    b = (packed[..., None] >> torch.arange(8, device=DEV, dtype=torch.uint8)) & 1
    b = b.view(*packed.shape[:-1], -1, bits)
    return (b * (1 << torch.arange(bits, device=DEV, dtype=torch.uint8))).sum(-1, dtype=torch.int16).double()


def _exact_weight(packed, scales, zeros, bits, group):
    rep = lambda t: t.double().repeat_interleave(group, -1)  # noqa: E731
    return rep(scales) * (_exact_codes(packed, bits) - rep(zeros))


def _hadamard(n):
    """H[i][j] = (-1)^popcount(i & j) / sqrt(n), fp64."""
    i = torch.arange(n, device=DEV)
    par = torch.zeros(n, n, dtype=torch.int64, device=DEV)
    both = i[:, None] & i
    for k in range(n.bit_length()):
        par ^= (both >> k) & 1
    return (1.0 - 2.0 * par.double()) / math.sqrt(n)


def _exact_rotate(x, n):
    return (x.double().view(*x.shape[:-1], -1, n) @ _hadamard(n)).view(x.shape) if n else x.double()


def exact(case, seed):
    c = dict(case)
    st = prepare(c, seed)
    if c["op"] in ("qgemv", "adapter_decode"):
        W = _exact_weight(*st["w"], c["bits"], c["group"])
        if c["op"] == "adapter_decode":
            row_ptr, col, coef = st["e"]
            F = torch.zeros(c["d_out"], c["d_in"], dtype=torch.float64, device=DEV)
            j = torch.arange(col.numel(), device=DEV)
            F[torch.searchsorted(row_ptr.long(), j, right=True) - 1, col.long()] = coef.double()
            return st["x"].double() @ W.T + ALPHA * (_exact_rotate(st["x"], c["had_block"]) @ F.T)
        return st["x"].double() @ W.T
    n, bits, group, out = c["had_block"], c["bits"], c["group"], []
    slots = _slots(st["table"], st["first"], st["starts"], st["rows"], c["page_size"])
    if c["op"] == "cache_read":
        for t in ("k", "v"):
            v = _exact_weight(*(x.flatten(0, 1)[slots] for x in st[t]), bits, group)
            out.append(_exact_rotate(v, n))
        return out
    top, state = 2**bits - 1, []
    for t, x in (("k", st["kx"]), ("v", st["vx"])):
        v = _exact_rotate(x, n).view(*x.shape[:-1], -1, group)
        lo = torch.minimum(v.min(-1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device=DEV))
        hi = torch.maximum(v.max(-1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device=DEV))
        s = ((hi - lo) / top).float().double()  # codes count steps of the scale that is stored
        s[s == 0] = 1.0
        z = torch.floor(-lo / s + 0.5 + 2.0**-12).clamp(0, top)
        q = torch.floor(v / s + z + 0.5 + 2.0**-12).clamp(0, top)
        out.append(_exact_rotate((s * (q - z)).flatten(-2), n))
        scales = st[t][1].double().flatten(0, 1)
        scales[slots] = s.squeeze(-1)
        state.append(scales.view(st[t][1].shape))
    return out + state + [None, None]


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    c = case
    esz = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("qgemv", "adapter_decode"):
        n, T = c["d_out"] * c["d_in"], c["T"]
        by = n * c["bits"] / 8 + 5 * n / c["group"] + T * (c["d_in"] + c["d_out"]) * esz
        fl = 2 * T * n
        if c["op"] == "adapter_decode":
            by += 8 * c["p"] + 4 * (c["d_out"] + 1)
            fl += 2 * T * c["p"] + T * c["d_in"] * math.log2(c["had_block"])
        return {"bytes": by, "flops": fl}
    rows = sum(_lengths(c)[1])
    values = 2 * rows * c["heads"] * c["head_dim"]
    held = values * c["bits"] / 8 + 5 * values / c["group"]
    moved = values * esz * (2 if c["op"] == "cache_append" else 1)
    passes = 2 if c["op"] == "cache_append" else 1
    return {"bytes": held + moved, "flops": passes * values * (4 + (math.log2(c["had_block"]) if c["had_block"] else 0))}
