"""Cases of the operators around the quantized cache: rotary positions (`rotary`), attention over the cache
(`cache_attention`), the page table (`pages_resize`, `pages_fork`) and the moves of cached rows (`cache_copy_pages`,
`cache_compact`).

`run` computes each operator in its plain form (elementary torch operations), or, with `own` set, through the package's
entry points. Sizes are generic ones of a decoder with 32 query and 8 key heads of 128, contexts of up to 32768 tokens,
cache formats as in the package's tests, and odd ones.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases


def _rotary(name, n, q_heads, heads, head_dim, rot, layout, scaling, longest, inverse, dtype):
    return dict(name=name, op="rotary", n=n, q_heads=q_heads, heads=heads, head_dim=head_dim, rot=rot, layout=layout,
                scaling=scaling, longest=longest, inverse=inverse, dtype=dtype)


def _attention(name, seqs, past, new, tree, q_heads, heads, head_dim, bits, bits_v, group, had_block, page_size, dtype):
    return dict(name=name, op="cache_attention", seqs=seqs, past=past, new=new, tree=tree, q_heads=q_heads, heads=heads,
                head_dim=head_dim, bits=bits, bits_v=bits_v, group=group, had_block=had_block, page_size=page_size,
                dtype=dtype)


def _pages(name, seqs, forks, past, new, page_size, spare):
    return dict(name=name, op="pages", seqs=seqs, forks=forks, past=past, new=new, page_size=page_size, spare=spare)


def _move(name, seqs, past, draft, keep, heads, head_dim, bits, group, page_size):
    return dict(name=name, op="move", seqs=seqs, past=past, draft=draft, keep=keep, heads=heads, head_dim=head_dim,
                bits=bits, group=group, page_size=page_size)


def listed():
    return [
        # a decode step of 64 streams: the smallest call, queries and keys are slices of the fused projection
        _rotary("rotary_decode", 64, 32, 8, 128, 128, "half", "none", 8192, False, "bf16"),
        # the backward of a training batch: part of the head, neighbouring channels paired, stretched context, fp32
        _rotary("rotary_back_f32", 16381, 32, 8, 80, 32, "pairs", "ramp", 131072, True, "f32"),
        # one stream, one token, a short context: latency
        _attention("attn_one", 1, 700, 1, False, 32, 8, 128, 4, 4, 128, 128, 16, "bf16"),
        # 64 ragged streams of a batch, one token each
        _attention("attn_batch", 64, 4096, 1, False, 32, 8, 128, 4, 4, 128, 128, 16, "bf16"),
        # long contexts, one token each, keys in 4 and values in 2 bits, groups of 64
        _attention("attn_long", 8, 32768, 1, False, 32, 8, 128, 4, 2, 64, 128, 64, "bf16"),
        # drafted trees of 64 tokens over ragged contexts
        _attention("attn_tree", 16, 4096, 64, True, 32, 8, 128, 4, 4, 128, 128, 16, "bf16"),
        # chunks of prompts behind what is cached of them, causal
        _attention("attn_chunk", 4, 2048, 1021, False, 32, 8, 128, 8, 8, 128, 0, 64, "bf16"),
        # odd heads of 80 in groups of 40, 3 bits, small trees, an odd share of query heads, pages of 100, fp32
        _attention("attn_odd_f32", 5, 700, 7, True, 9, 3, 80, 3, 3, 40, 16, 100, "f32"),
        # a step of the page table of 64 streams: forks, growth for a draft, release
        _pages("pages_step", 64, 8, 1500, 16, 16, 512),
        # the table of a large pool: 2048 streams, 200 thousand pages
        _pages("pages_large", 2048, 512, 1500, 64, 16, 12288),
        # after verification of drafts: one stream, its fork's page is copied and the accepted tokens move up
        _move("move_step", 1, 1500, 16, 5, 8, 128, 4, 128, 16),
        # the same for 512 streams with trees of 64, pages of 64, groups of 32
        _move("move_batch", 512, 4000, 64, 8, 8, 128, 8, 32, 64),
    ]


FORMATS = [(64, 64, 64), (64, 32, 0), (80, 40, 16), (96, 96, 32), (128, 128, 128), (128, 128, 0), (128, 64, 128),
           (128, 32, 0), (256, 64, 256), (256, 256, 0)]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "cache_attention", "cache_attention", "cache_attention", "pages", "move"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    head_dim, group, had_block = rng.choice(FORMATS)
    heads = rng.choice([1, 2, 3, 4, 8, 8])
    page_size = rng.choice([1, 16, 16, 64, 100])
    if op == "rotary":
        q_heads = heads * rng.choice([1, 2, 4, 4, 7])
        rot = rng.choice([head_dim, head_dim, head_dim // 2, 16])
        top = max(1, 16381 * 40 * 80 // ((q_heads + heads) * head_dim))
        return dict(op=op, n=_log(rng, 1, min(16381, top)), q_heads=q_heads, heads=heads, head_dim=head_dim, rot=rot,
                    layout=rng.choice(["half", "half", "pairs"]), scaling=rng.choice(["none", "linear", "ramp", "bands"]),
                    longest=_log(rng, 512, 1 << 20), inverse=rng.random() < 0.3, dtype=dtype)
    if op == "pages":
        seqs = _log(rng, 1, 2048)
        return dict(op=op, seqs=seqs, forks=min(seqs, _log(rng, 1, 512)), past=_log(rng, 1, 1500),
                    new=_log(rng, 1, 64), page_size=rng.choice([1, 16, 16, 64, 100]) if seqs < 128 else 16,
                    spare=_log(rng, 16, 12288))
    if op == "move":
        draft = _log(rng, 2, 64)
        return dict(op=op, seqs=_log(rng, 1, 512), past=_log(rng, 1, 4000), draft=draft,
                    keep=rng.randint(1, min(draft, 12)), heads=heads, head_dim=head_dim, bits=rng.choice([2, 3, 4, 4, 8]),
                    group=group, page_size=rng.choice([1, 16, 16, 64]))
    grp = rng.choice([1, 2, 3, 4, 4, 7, 8])
    kind = rng.choice(["one", "one", "tree", "chain"])
    seqs = _log(rng, 1, 64)
    new = 1 if kind == "one" else _log(rng, 2, 64 if kind == "tree" else 1021)
    # no more cached values than attn_long has, no more products than attn_chunk
    past = 8 * 32768 * 8 * 128 // (seqs * heads * head_dim)
    flops = 4 * 1021 * 32 * 128 * 2048
    past = min(past, flops // (seqs * new * grp * heads * head_dim))
    past = rng.choice([0, _log(rng, 1, max(1, min(32768, past)))]) if kind != "one" else _log(rng, 1, max(1, min(32768, past)))
    if kind == "chain":
        new = max(2, min(new, 8 * 32768 * 8 * 128 // (seqs * heads * head_dim) - past))
    bits = rng.choice([2, 3, 4, 4, 8])
    return dict(op=op, seqs=seqs, past=past, new=new, tree=kind == "tree", q_heads=grp * heads, heads=heads,
                head_dim=head_dim, bits=bits, bits_v=rng.choice([bits, bits, 2]), group=group, had_block=had_block,
                page_size=page_size, dtype=dtype)


# ---------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _spread(count, longest):
    """Lengths of [longest / 2, longest], spread by multiples of the golden section."""
    return [longest - int(((i + 1) * 0.6180339887 % 1.0) * (longest // 2 + 1)) for i in range(count)]


def _new(c):
    """Tokens that each sequence of an attention case brings: one, or ragged drafts and chunks."""
    if c["new"] == 1:
        return [1] * c["seqs"]
    return [max(1, c["new"] - 3 * (i % 4)) if i % 7 < 6 else c["new"] for i in range(c["seqs"])]


def _past(c):
    return _spread(c["seqs"], c["past"]) if c["past"] else [0] * c["seqs"]


def _starts(lens):
    s = torch.zeros(len(lens) + 1, dtype=torch.int64, device=DEV)
    s[1:] = torch.cumsum(torch.tensor(lens, dtype=torch.int64), 0)
    return s


def _pool(g, n_pages, c, bits):
    """A cache pool that earlier tokens have filled: codes, scales and zero points of every slot."""
    rows = (n_pages, c["page_size"], c["heads"])
    codes = torch.randint(0, 256, rows + (c["head_dim"] * bits // 8,), generator=g, device=DEV, dtype=torch.uint8)
    ng, top = c["head_dim"] // c["group"], 2**bits - 1
    scales = (3.0 + 3.0 * torch.rand(rows + (ng,), generator=g, device=DEV)) / top
    zeros = torch.randint(top // 3, (2 * top) // 3 + 1, rows + (ng,), generator=g, device=DEV, dtype=torch.uint8)
    return [codes, scales, zeros]


def _paged(g, lens, page_size, spare=0):
    """A page table of shuffled pages for sequences of these lengths, and the page count."""
    need = (torch.tensor(lens, dtype=torch.int64) + page_size - 1) // page_size
    width, total = max(1, int(need.max())), int(need.sum())
    need = need.to(DEV)
    order = torch.randperm(total + spare, generator=g, device=DEV).to(torch.int32)
    at = torch.cumsum(need, 0) - need
    j = torch.arange(width, device=DEV)
    idx = (at[:, None] + j).clamp_(max=max(total - 1, 0))
    table = torch.where(j < need[:, None], order[idx], torch.full_like(order[idx], -1)).contiguous()
    return table, total + spare


def _frequencies(c):
    """(frequencies fp64 [rot / 2], factor of the rotated channels): plain ones, or stretched to a longer context."""
    r, base, trained, stretch = c["rot"], 10000.0, 8192, 4.0
    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    if c["scaling"] == "none":
        return f.to(DEV), 1.0
    if c["scaling"] == "linear":
        return (f / stretch).to(DEV), 1.0
    turns = trained * f / (2 * math.pi)  # full turns within the trained context
    if c["scaling"] == "ramp":  # by the index of the channel between 32 turns and one
        at = [r * math.log(trained / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
        u = ((torch.arange(r // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return (f / stretch * u + f * (1 - u)).to(DEV), 0.1 * math.log(stretch) + 1.0
    u = ((turns - 1.0) / 3.0).clamp(0, 1)  # bands: between one and four turns
    return (f / stretch * (1 - u) + f * u).to(DEV), 1.0


def _tree_masks(g, counts):
    """Masks of drafted trees, packed: bit u of token j's mask is set where u is j itself or an ancestor. The last of
    every fourth draft is padding, which sees no drafted token."""
    B, most = len(counts), max(counts)
    parent = (torch.rand(B, most, generator=g, device=DEV) * torch.arange(most, device=DEV)).long()
    parent = torch.where(torch.rand(B, most, generator=g, device=DEV) < 0.1, torch.full_like(parent, -1), parent)
    m = torch.zeros(B, most, dtype=torch.int64, device=DEV)
    one = torch.ones((), dtype=torch.int64, device=DEV)
    for j in range(most):
        p = parent[:, j] if j else torch.full_like(parent[:, 0], -1)
        above = torch.where(p >= 0, m.gather(1, p.clamp(min=0)[:, None]).squeeze(1), torch.zeros_like(p))
        m[:, j] = above | (one << j)
    for b in range(3, B, 4):
        m[b, counts[b] - 1] = 0
    keep = torch.arange(most, device=DEV) < torch.tensor(counts, device=DEV)[:, None]
    return m[keep].contiguous()


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    st = {"case": c}
    if c["op"] == "rotary":
        wide = torch.randn(c["n"], c["q_heads"] + 2 * c["heads"], c["head_dim"], generator=g, device=DEV).to(DTYPES[c["dtype"]])
        st["q"], st["k"] = wide[:, :c["q_heads"]], wide[:, c["q_heads"]:c["q_heads"] + c["heads"]]
        st["pos"] = torch.randint(0, c["longest"], (c["n"],), generator=g, device=DEV)
        st["freq"], st["factor"] = _frequencies(c)
    elif c["op"] == "cache_attention":
        past, new = _past(c), _new(c)
        st["lens"] = (past, new)
        st["table"], n_pages = _paged(g, [a + b for a, b in zip(past, new)], c["page_size"])
        st["past"], st["starts"] = torch.tensor(past, dtype=torch.int64, device=DEV), _starts(new)
        st["k"], st["v"] = _pool(g, n_pages, c, c["bits"]), _pool(g, n_pages, c, c["bits_v"])
        # queries that prefer some keys: scores spread over a few units
        st["q"] = (2.0 * torch.randn(sum(new), c["q_heads"], c["head_dim"], generator=g, device=DEV)).to(DTYPES[c["dtype"]])
        st["tree"] = _tree_masks(g, new) if c["tree"] else None
    elif c["op"] == "pages":
        lens = _spread(c["seqs"], c["past"])
        live, n_pages = _paged(g, lens, c["page_size"], c["spare"])
        n_seqs, width = c["seqs"] + c["forks"], -(-(c["past"] + c["new"]) // c["page_size"])
        table = torch.full((n_seqs, width), -1, dtype=torch.int32, device=DEV)
        table[:c["seqs"], :live.shape[1]] = live
        refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        refs[live[live >= 0].long()] = 1
        held = torch.tensor(lens + [0] * c["forks"], dtype=torch.int64, device=DEV)
        st["refs"], st["pages"], st["held"] = refs, table, held
        st["src"] = torch.randint(0, c["seqs"], (c["forks"],), generator=g, device=DEV)
        st["dst"] = c["seqs"] + torch.randperm(c["forks"], generator=g, device=DEV)
        st["grow"] = torch.cat((held[:c["seqs"]], held[st["src"]][torch.argsort(st["dst"])])) + c["new"]
        st["back"] = held.clone()
    else:
        lens = [n + c["draft"] for n in _spread(c["seqs"], c["past"])]
        ps = c["page_size"]
        tails = [((n - c["draft"]) // ps, -(-n // ps)) for n in lens]  # the pages that hold a draft
        count = sum(b - a for a, b in tails)
        order = torch.randperm(2 * count, generator=g, device=DEV).to(torch.int32)
        st["from"], st["to"] = order[:count].contiguous(), order[count:].contiguous()
        table = torch.full((c["seqs"], max(b for _, b in tails)), -1, dtype=torch.int32)
        rows = torch.repeat_interleave(torch.arange(c["seqs"]), torch.tensor([b - a for a, b in tails]))
        cols = torch.cat([torch.arange(a, b) for a, b in tails])
        table[rows, cols] = st["to"].cpu()
        st["pages"] = table.to(DEV)
        st["first"] = torch.tensor([n - c["draft"] for n in lens], dtype=torch.int64, device=DEV)
        # accepted nodes of the draft: ascending, between one and `keep` of them, -1 behind
        pick = torch.rand(c["seqs"], c["draft"], generator=g, device=DEV).argsort(1)[:, :c["keep"]].sort(1).values
        much = 1 + (torch.rand(c["seqs"], generator=g, device=DEV) * c["keep"]).long()
        st["keep"] = torch.where(torch.arange(c["keep"], device=DEV) < much[:, None], pick, torch.full_like(pick, -1)).to(torch.int32)
        st["k"], st["v"] = _pool(g, 2 * count, c, c["bits"]), _pool(g, 2 * count, c, c["bits"])
    return st


# ---------------------------------------------------------------- one pass


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _plain_rotary(x, st, c):
    angle = st["pos"].double()[:, None] * st["freq"]
    cos = (angle.cos() * st["factor"]).float()[:, None]
    sin = (angle.sin() * st["factor"]).float()[:, None]
    if c["inverse"]:
        sin = -sin
    r, v = c["rot"], x.float()
    if c["layout"] == "half":
        a, b = v[..., :r // 2], v[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = v[..., 0:r:2], v[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, v[..., r:]), -1).to(x.dtype)


def _codes(packed, bits):
    """The codes of a little-endian bit stream, one int32 each."""
    if bits == 8:
        return packed.to(torch.int32)
    by = packed.reshape(*packed.shape[:-1], -1, bits).to(torch.int32)
    word = (by << (8 * torch.arange(bits, device=by.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    q = (word[..., None] >> (bits * torch.arange(8, device=by.device, dtype=torch.int32))) & (2**bits - 1)
    return q.reshape(*packed.shape[:-1], packed.shape[-1] * 8 // bits)


def _rotate(x, n):
    """x H for blocks of n along the last dimension: the stages 1, 2, 4, ..., then the factor 1/sqrt(n)."""
    if not n:
        return x
    shape, h = x.shape, 1
    while h < n:
        x = x.reshape(-1, 2, h)
        x = torch.stack((x[:, 0] + x[:, 1], x[:, 0] - x[:, 1]), 1)
        h *= 2
    return x.reshape(shape) * (1.0 / math.sqrt(n))


def _dense(pool, slots, bits, c):
    """The rows [slots, heads, head_dim] of a pool in fp32."""
    codes, scales, zeros = (t.flatten(0, 1)[slots] for t in pool)
    q = _codes(codes, bits)
    q = q.view(*q.shape[:-1], -1, c["group"])
    return _rotate((scales[..., None] * (q - zeros[..., None].to(torch.int32)).float()).flatten(-2), c["had_block"])


def _plain_attention(st, c):
    out = torch.empty_like(st["q"])
    grp, at = c["q_heads"] // c["heads"], 0
    for b, (past, new) in enumerate(zip(*st["lens"])):
        t = torch.arange(past + new, device=DEV)
        slots = st["table"][b, t // c["page_size"]].long() * c["page_size"] + t % c["page_size"]
        k, v = _dense(st["k"], slots, c["bits"], c), _dense(st["v"], slots, c["bits_v"], c)
        u, j = t - past, torch.arange(new, device=DEV)[:, None]
        if st["tree"] is None:
            seen = u <= j
        else:
            seen = (u < 0) | ((st["tree"][at:at + new, None] >> u.clamp(min=0)) & 1).bool()
        q = st["q"][at:at + new].float().view(new, c["heads"], grp, -1).permute(1, 2, 0, 3).flatten(1, 2)
        s = q @ k.permute(1, 2, 0) * (1.0 / math.sqrt(c["head_dim"]))
        s = s.view(c["heads"], grp, new, -1).masked_fill(~seen, -math.inf).flatten(1, 2)
        top = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = p.sum(-1, keepdim=True)
        o = (p @ v.permute(1, 0, 2)) / torch.where(total == 0, torch.ones_like(total), total)
        out[at:at + new] = o.view(c["heads"], grp, new, -1).permute(2, 0, 1, 3).flatten(1, 2).to(out.dtype)
        at += new
    return out


def _plain_fork(refs, pages, held, src, dst, ps):
    n, width = src.numel(), pages.shape[1]
    tokens = held[src]
    full, part = tokens // ps, tokens % ps > 0
    free = (refs == 0).nonzero().squeeze(1)
    rank = torch.cumsum(part, 0)
    good = rank <= free.numel()
    part = part & good
    j = torch.arange(width, device=DEV)
    shared = (j < full[:, None]) & good[:, None]
    rows = pages[src]
    refs.index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    fresh = torch.where(part, free[(rank - 1).clamp(0, max(free.numel() - 1, 0))].int(), torch.full_like(rows[:, 0], -1)) \
        if free.numel() else torch.full_like(rows[:, 0], -1)
    origin = torch.where(part, rows.gather(1, full.clamp(max=width - 1)[:, None]).squeeze(1), torch.full_like(fresh, -1))
    new_rows = torch.where(shared, rows, torch.full_like(rows, -1))
    i = torch.arange(n, device=DEV)[part]
    new_rows[i, full[part]] = fresh[part]
    refs[fresh[part].long()] = 1
    pages[dst] = new_rows
    held[dst] = torch.where(good, tokens, torch.zeros_like(tokens))
    return origin, fresh


def _plain_resize(refs, pages, held, want, ps):
    have, to = (held + ps - 1) // ps, (want + ps - 1) // ps
    j = torch.arange(pages.shape[1], device=DEV)
    drop = (j >= to[:, None]) & (j < have[:, None])
    gone = pages[drop]
    refs.index_add_(0, gone.long(), -torch.ones_like(gone))
    pages[drop] = -1
    need = (to - have).clamp(min=0)
    upto = torch.cumsum(need, 0)
    free = (refs == 0).nonzero().squeeze(1)
    good = (need == 0) | (upto <= free.numel())
    add = (j >= have[:, None]) & (j < to[:, None]) & good[:, None]
    got = free[((upto - need)[:, None] + j - have[:, None])[add]].int()
    pages[add] = got
    refs[got.long()] = 1
    held.copy_(torch.where(good, want, held))


def _plain_move(pool, st, c):
    for t in pool:
        t[st["to"].long()] = t[st["from"].long()]
    ps = c["page_size"]
    live = st["keep"] >= 0
    row = torch.arange(c["seqs"], device=DEV)[:, None].expand_as(live)[live]
    at = st["first"][row]
    old, new = at + st["keep"][live], at + torch.arange(live.shape[1], device=DEV).expand_as(live)[live]
    for t in pool:
        flat = t.flatten(0, 1)
        rows = flat[st["pages"][row, old // ps].long() * ps + old % ps]
        flat[st["pages"][row, new // ps].long() * ps + new % ps] = rows


def _run_plain(st):
    c = st["case"]
    if c["op"] == "rotary":
        return [_plain_rotary(st["q"], st, c), _plain_rotary(st["k"], st, c)]
    if c["op"] == "cache_attention":
        return _plain_attention(st, c)
    if c["op"] == "pages":
        refs, pages, held, ps = st["refs"], st["pages"], st["held"], c["page_size"]
        origin, fresh = _plain_fork(refs, pages, held, st["src"], st["dst"], ps)
        _plain_resize(refs, pages, held, st["grow"], ps)
        mid = [refs.clone(), pages.clone(), held.clone()]
        _plain_resize(refs, pages, held, st["back"], ps)
        return [origin, fresh] + mid + [refs, pages, held]
    _plain_move(st["k"], st, c)
    _plain_move(st["v"], st, c)
    return st["k"] + st["v"]


def _run_own(st):
    import walsh_hadamard_sparse_b200 as W

    c = st["case"]
    if c["op"] == "rotary":
        return list(W.rotary((st["q"], st["k"]), st["pos"], st["freq"], interleaved=c["layout"] == "pairs",
                             factor=st["factor"], inverse=c["inverse"]))
    if c["op"] == "cache_attention":
        kv = tuple(W.QCache(c[b], c["group"], c["had_block"], *st[t]) for t, b in (("k", "bits"), ("v", "bits_v")))
        return W.cache_attention(kv, st["q"], st["table"], st["starts"], st["past"], tree=st["tree"])
    if c["op"] == "pages":
        t = W.PageTable(c["page_size"], st["refs"], st["pages"], st["held"])
        origin, fresh = W.pages_fork(t, st["src"], st["dst"])
        W.pages_resize(t, st["grow"])
        mid = [t.refs.clone(), t.pages.clone(), t.held.clone()]
        W.pages_resize(t, st["back"])
        return [origin, fresh] + mid + [t.refs, t.pages, t.held]
    kv = tuple(W.QCache(c["bits"], c["group"], 0, *st[t]) for t in ("k", "v"))
    W.cache_copy_pages(kv, st["from"], st["to"])
    W.cache_compact(kv, st["pages"], st["first"], st["keep"])
    return st["k"] + st["v"]


# ---------------------------------------------------------------- the definition in 64 bits


def _hadamard(n):
    """H[i][j] = (-1)^popcount(i & j) / sqrt(n), fp64."""
    i = torch.arange(n, device=DEV)
    par = torch.zeros(n, n, dtype=torch.int64, device=DEV)
    both = i[:, None] & i
    for k in range(n.bit_length()):
        par ^= (both >> k) & 1
    return (1.0 - 2.0 * par.double()) / math.sqrt(n)


def _exact_rows(pool, b, past, new, st, bits, c):
    """Rows [tokens, heads, head_dim] of sequence b, token by token from its pages."""
    ps, total = c["page_size"], past + new
    pages = st["table"][b, :-(-total // ps)].long()
    packed, scales, zeros = (t[pages].flatten(0, 1)[:total] for t in pool)
    bit = (packed[..., None] >> torch.arange(8, device=DEV, dtype=torch.uint8)) & 1
    bit = bit.view(*packed.shape[:-1], -1, bits)
    q = (bit * (1 << torch.arange(bits, device=DEV, dtype=torch.uint8))).sum(-1, dtype=torch.int16).double()
    w = scales.double().repeat_interleave(c["group"], -1) * (q - zeros.double().repeat_interleave(c["group"], -1))
    n = c["had_block"]
    return (w.view(*w.shape[:-1], -1, n) @ _hadamard(n)).view(w.shape) if n else w


def _exact_move(pool, st, c):
    """The scales after the move: token i of the accepted ones is node keep[i] of the page that was copied."""
    ps, before = c["page_size"], pool[1].double()
    after = before.clone()
    after.index_copy_(0, st["to"].long(), before.index_select(0, st["from"].long()))
    drafted = after.clone()
    for i in range(c["keep"]):
        b = (st["keep"][:, i] >= 0).nonzero().squeeze(1)
        to, fr = st["first"][b] + i, st["first"][b] + st["keep"][b, i]
        after[st["pages"][b, to // ps].long(), to % ps] = drafted[st["pages"][b, fr // ps].long(), fr % ps]
    return [None, after, None]


def exact(case, seed):
    c = dict(case)
    if c["op"] == "pages":
        return None  # whole numbers
    st = prepare(c, seed)
    if c["op"] == "move":
        return _exact_move(st["k"], st, c) + _exact_move(st["v"], st, c)
    if c["op"] == "rotary":
        turn = torch.polar(torch.full((c["n"], c["rot"] // 2), st["factor"], dtype=torch.float64, device=DEV),
                           st["pos"].double()[:, None] * st["freq"] * (-1.0 if c["inverse"] else 1.0))[:, None]
        out = []
        for x in (st["q"].double(), st["k"].double()):
            y, r = x.clone(), c["rot"]
            at = (slice(0, r // 2), slice(r // 2, r)) if c["layout"] == "half" else (slice(0, r, 2), slice(1, r, 2))
            z = torch.complex(x[..., at[0]], x[..., at[1]]) * turn
            y[..., at[0]], y[..., at[1]] = z.real, z.imag
            out.append(y)
        return out
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    at, grp = 0, c["q_heads"] // c["heads"]
    for b, (past, new) in enumerate(zip(_past(c), _new(c))):
        k = _exact_rows(st["k"], b, past, new, st, c["bits"], c)
        v = _exact_rows(st["v"], b, past, new, st, c["bits_v"], c)
        seen = torch.ones(new, past + new, dtype=torch.bool, device=DEV)
        for u in range(new):
            if c["tree"]:
                seen[:, past + u] = (st["tree"][at:at + new] >> u) % 2 == 1
            else:
                seen[:u, past + u] = False
        for h in range(c["q_heads"]):
            s = st["q"][at:at + new, h].double() @ k[:, h // grp].T / math.sqrt(c["head_dim"])
            w = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
            out[at:at + new, h] = torch.where(seen.any(1, keepdim=True), w, torch.zeros_like(w)) @ v[:, h // grp]
        at += new
    return out


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    c = case
    if c["op"] == "rotary":
        values = c["n"] * (c["q_heads"] + c["heads"]) * c["head_dim"]
        return {"bytes": 2 * values * (4 if c["dtype"] == "f32" else 2) + 8 * c["n"] + 4 * c["rot"],
                "flops": 3 * values * c["rot"] // c["head_dim"]}
    if c["op"] == "cache_attention":
        past, new = _past(c), _new(c)
        rows = sum(past) + sum(new)
        values = rows * c["heads"] * c["head_dim"]
        by = values * (c["bits"] + c["bits_v"]) / 8 + 10 * values / c["group"]
        by += 2 * sum(new) * c["q_heads"] * c["head_dim"] * (4 if c["dtype"] == "f32" else 2) + 4 * rows / c["page_size"]
        pairs = sum(a * b + b * (b + 1) / 2 for a, b in zip(past, new))
        return {"bytes": by, "flops": 4 * pairs * c["q_heads"] * c["head_dim"]}
    if c["op"] == "pages":
        ps, lens = c["page_size"], _spread(c["seqs"], c["past"])
        used = sum(-(-n // ps) for n in lens)
        shared = c["forks"] * used / c["seqs"]
        grown = (c["seqs"] + c["forks"]) * c["new"] / ps
        by = 4 * (used + c["spare"]) + 4 * (4 * shared + 2 * grown) + 24 * (c["seqs"] + c["forks"])
        return {"bytes": by, "flops": used + c["spare"] + 4 * shared}
    ps = c["page_size"]
    row = c["heads"] * (c["head_dim"] * c["bits"] / 8 + 5 * c["head_dim"] / c["group"])
    pages = sum(-(-n // ps) - (n - c["draft"]) // ps for n in (m + c["draft"] for m in _spread(c["seqs"], c["past"])))
    moved = 2 * (pages * ps + c["seqs"] * (c["keep"] + 1) / 2) * row
    return {"bytes": 2 * moved + 8 * pages + 4 * c["seqs"] * c["keep"], "flops": moved}
