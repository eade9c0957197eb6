"""Cases of the operators that serve more requests from the same memory: the factored cache in 8 bits
(rows quantised with a scale for each block of 16 tokens and head, a decode step over them) and the
pages of a paged cache (fork, extend with copies on write, compact).

`run` computes the plain form (elementary torch operations, 32 bits) or, with `own`, calls the
framework.  `exact` restates the computed numbers in 64 bits along another route: keys rebuilt per
head, the rounding to 8 bits from its definition.
"""
import math

import torch

own = False

PAGE = 256          # rows per page of the paged caches of decode and quantize cases
BLOCK = 16          # rows that share a scale
E4M3 = torch.float8_e4m3fn


def _framework():
    from compressed_cache_decode_gb300 import lrkv
    return lrkv


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one short sequence of the smallest bf16 decode workload: latency of a lone request
        dict(name="decode_one", op="decode", batch=1, heads=16, dim=64, rank=28, lo=517, hi=517, cap=576,
             paged=False, empty=False),
        # a batch of contexts of one length (the 8 x 4K-row decode workload)
        dict(name="decode_batch", op="decode", batch=8, heads=16, dim=64, rank=28, lo=4096, hi=4096, cap=4096,
             paged=False, empty=False),
        # batched serving from pages, ragged lengths (the batched decode workload's shape)
        dict(name="decode_paged", op="decode", batch=32, heads=32, dim=128, rank=56, lo=1024, hi=8192, cap=8192,
             paged=True, empty=True),
        # few long contexts (the long-context workload): split over the length and joined
        dict(name="decode_long", op="decode", batch=4, heads=32, dim=128, rank=48, lo=65536, hi=65536, cap=65536,
             paged=False, empty=False),
        # the new token of every sequence of a batch, into blocks that were begun before
        dict(name="quantize_step", op="quantize", batch=32, new=1, heads=32, dim=128, rank=56, lo=1025, hi=8191,
             cap=8192, paged=True, ragged=False),
        # prompts of different lengths into an empty cache
        dict(name="quantize_prompts", op="quantize", batch=8, new=8192, heads=32, dim=128, rank=48, lo=0, hi=0,
             cap=8192, paged=False, ragged=True),
        # a beam search step: every beam goes on from one of its request's beams
        dict(name="fork_beams", op="fork", batch=64, group=4, blocks=64, page=64, lo=600, hi=4000, spare=900,
             beams=True),
        # requests that end, are cut back or sampled several times from one prompt
        dict(name="fork_requests", op="fork", batch=512, group=8, blocks=512, page=64, lo=1, hi=32768, spare=5000,
             beams=False),
        # room for the next token of every beam: pages shared by beams are copied before they are written
        dict(name="extend_step", op="extend", batch=256, group=4, blocks=32, page=64, lo=65, hi=2000, grow=1,
             spare=400, heads=32, dim=128, rank=48, cache="e4m3"),
        # room for the next turn of a conversation, sampled twice
        dict(name="extend_turns", op="extend", batch=64, group=2, blocks=40, page=256, lo=300, hi=8000, grow=2000,
             spare=800, heads=16, dim=64, rank=28, cache="bf16"),
        # the few pages that a night's requests left behind in an 8-bit pool
        dict(name="compact_few", op="compact", batch=24, blocks=16, page=64, lo=1, hi=1024, live=0.4,
             heads=16, dim=64, rank=28, cache="e4m3"),
        # a large pool brought down to its live pages
        dict(name="compact_pool", op="compact", batch=64, blocks=64, page=64, lo=100, hi=4096, live=0.5,
             heads=32, dim=128, rank=48, cache="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "quantize", "fork", "extend", "compact"])
    heads, dim = rng.choice([(16, 64), (32, 64), (16, 128), (32, 128)])
    rank = rng.choice([28, 32, 48, 56, 64])
    if op == "decode":
        batch = _log(rng, 1, 32)
        hi = _log(rng, 16, max(64, 4 * 65536 // batch // 2))
        return dict(op=op, batch=batch, heads=heads, dim=dim, rank=rank, lo=rng.randint(1, hi), hi=hi,
                    cap=-(-hi // PAGE) * PAGE, paged=rng.random() < 0.5, empty=rng.random() < 0.3)
    if op == "quantize":
        batch = _log(rng, 1, 32)
        new = _log(rng, 1, 32768 // batch)
        hi = rng.choice([0, _log(rng, 1, 8192)])
        return dict(op=op, batch=batch, new=new, heads=heads, dim=dim, rank=rank, lo=rng.randint(0, hi), hi=hi,
                    cap=-(-(hi + new) // PAGE) * PAGE, paged=rng.random() < 0.5, ragged=rng.random() < 0.5)
    page = rng.choice([16, 64, 128, 256])
    if op == "fork":
        batch, blocks = _log(rng, 1, 512), _log(rng, 4, 512)
        hi = rng.randint(1, blocks * page)
        return dict(op=op, batch=batch, group=rng.choice([1, 2, 4, 8]), blocks=blocks, page=page,
                    lo=rng.randint(0, hi), hi=hi, spare=_log(rng, 1, 2000), beams=rng.random() < 0.5)
    cache = rng.choice(["bf16", "e4m3"])
    if op == "extend":
        batch = _log(rng, 1, 128)
        blocks = _log(rng, 2, max(2, 131072 // (batch * page)))
        hi = rng.randint(1, blocks * page)
        grow = rng.choice([1, 1, rng.randint(1, blocks * page)])
        return dict(op=op, batch=batch, group=rng.choice([1, 2, 4]), blocks=blocks, page=page, lo=rng.randint(0, hi),
                    hi=hi, grow=grow, spare=rng.randint(0, 2 * batch * (1 + grow // page)), heads=heads, dim=dim,
                    rank=rank, cache=cache)
    batch = _log(rng, 1, 64)
    blocks = _log(rng, 2, max(2, 131072 // (batch * page)))
    hi = rng.randint(1, blocks * page)
    return dict(op=op, batch=batch, blocks=blocks, page=page, lo=rng.randint(0, hi), hi=hi,
                live=rng.uniform(0.2, 1.0), heads=heads, dim=dim, rank=rank, cache=cache)


def _lens(case):
    """Lengths spread over [lo, hi], the longest first, the last one empty where the case says so."""
    span = case["hi"] - case["lo"]
    lens = [case["hi"] - int(span * ((b * 0.6180339887) % 1.0)) for b in range(case["batch"])]
    if case.get("empty") and len(lens) > 1:
        lens[-1] = 0
    return lens


def _new(case):
    """Rows that each sequence of a quantize case brings."""
    if not case["ragged"]:
        return [case["new"]] * case["batch"]
    return [max(1, int(case["new"] * (1 - 0.5 * ((b * 0.6180339887) % 1.0)))) for b in range(case["batch"])]


def _row8(case):
    """Bytes of a token's rows and its share of the scales, in 8 bits and in bf16."""
    H, d, r = case["heads"], case["dim"], case["rank"]
    return 2 * (d + H * r) + 8 * (1 + H) / BLOCK, 4 * (d + H * r)


def _page_bytes(case, rows):
    row8, row16 = _row8(case)
    return rows * (row8 if case["cache"] == "e4m3" else row16)


def work(case):
    op, B = case["op"], case["batch"]
    if op == "decode":
        H, d, r, total = case["heads"], case["dim"], case["rank"], sum(_lens(case))
        return {"bytes": total * _row8(case)[0] + 2 * 2 * H * d * r + B * H * (6 * d + 4),
                "flops": total * H * 4 * (d + r) + B * H * 4 * d * r}
    if op == "quantize":
        row8, row16 = _row8(case)
        return {"bytes": sum(_new(case)) * (row8 + row16), "flops": 2 * sum(_new(case)) * row16 / 2}
    table = 8 * B * case["blocks"]
    if op == "fork":
        return {"bytes": table + 8 * _pages(case) + 16 * B, "flops": B * case["blocks"]}
    if op == "extend":
        # all but one of the sequences that share a begun page copy its rows
        begun = [n % case["page"] for n in _shared_lens(case)]
        copied = sum(n for b, n in enumerate(begun) if b % case["group"])
        return {"bytes": table + 8 * _pages(case) + 2 * _page_bytes(case, copied), "flops": B * case["blocks"]}
    live = sum(-(-n // case["page"]) for n in _lens(case))
    moved = live * (1 - live / _pages(case))
    return {"bytes": table + 12 * _pages(case) + 2 * moved * _page_bytes(case, case["page"]), "flops": moved}


# ----------------------------------------------------------------- inputs --

def _rand(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _widths(case):
    """(name, heads, columns per head) of the cache tensors; a shared row is one head."""
    H, d, r = case["heads"], case["dim"], case["rank"]
    return [("k_s", 1, d), ("v_s", 1, d), ("z_k", H, r), ("z_v", H, r)]


def _shape(lead, name, heads, width):
    return (*lead, heads, width) if name.startswith("z") else (*lead, width)


def _blocks_of(name, heads):
    return (heads,) if name.startswith("z") else ()


def _shared_lens(case):
    """Lengths of sequences in groups that share a history: one length per group."""
    return [n for n in _lens(dict(case, batch=-(-case["batch"] // case["group"]))) for _ in range(case["group"])][
        : case["batch"]]


def _pages(case):
    """Pages of the pool of a pages case."""
    page = case["page"]
    if case["op"] == "compact":
        return max(1, int(sum(-(-n // page) for n in _lens(case)) / case["live"])) + 1
    lens = _shared_lens(case)
    return sum(-(-n // page) for b, n in enumerate(lens) if b % case["group"] == 0) + case["spare"] + 1


def _pool(case, gen, pages):
    """Pools of a paged cache of every type: rows, and for 8 bits the scales of their blocks."""
    pools = {}
    for name, heads, width in _widths(case):
        lead = (pages, case["page"])
        if case["cache"] == "bf16":
            pools[name] = _rand(gen, *_shape(lead, name, heads, width))
        else:
            pools[name] = torch.randint(0, 120, _shape(lead, name, heads, width), generator=gen, device="cuda",
                                        dtype=torch.uint8).view(E4M3)
            lead = (pages, case["page"] // BLOCK, *_blocks_of(name, heads))
            pools[name + "_scale"] = torch.exp2(torch.randint(-9, -5, lead, generator=gen, device="cuda").float())
    return pools


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    s = {"case": case}
    if case["op"] in ("fork", "extend", "compact"):
        return _prepare_pages(s, case, gen)
    B, H, d, r, cap = case["batch"], case["heads"], case["dim"], case["rank"], case["cap"]
    rows, s["block_table"] = (B, cap), None
    if case["paged"]:
        blocks = cap // PAGE
        pages = B * blocks + 3
        rows = (pages, PAGE)
        order = torch.randperm(pages, generator=gen, device="cuda")
        s["block_table"] = order[: B * blocks].reshape(B, blocks).to(torch.int32)
    s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    s["cache"] = {}
    for name, heads, width in _widths(case):
        x = _rand(gen, *_shape(rows, name, heads, width))
        if name == "k_s":   # a few tokens stand out
            x *= torch.where(torch.rand(*rows, 1, generator=gen, device="cuda") < 0.05, 8, 1).to(x.dtype)
        lead = (rows[0], -(-rows[1] // BLOCK))
        s["cache"][name] = torch.zeros(x.shape, dtype=torch.uint8, device="cuda").view(E4M3)
        s["cache"][name + "_scale"] = torch.ones(*lead, *_blocks_of(name, heads), device="cuda")
        if case["op"] == "decode" or case["hi"]:
            v, scale = _round8(x.float().reshape(*rows, heads, width))
            s["cache"][name].copy_(v.reshape(x.shape).to(E4M3))
            s["cache"][name + "_scale"].copy_(scale.reshape(s["cache"][name + "_scale"].shape))
    if case["op"] == "quantize":
        n = case["new"]
        for name, heads, width in _widths(case):
            s[name] = _rand(gen, *_shape((B, n), name, heads, width))
        # later tokens stand out now and then: a begun block's scale grows
        s["k_s"] *= torch.where(torch.rand(B, n, 1, generator=gen, device="cuda") < 0.05, 8, 1).to(torch.bfloat16)
        s["new_lens"] = torch.tensor(_new(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        if own:
            lrkv = _framework()
            s["ws"] = torch.zeros(16, dtype=torch.uint8, device="cuda")
            s["cache8"] = lrkv.Cache8(**s["cache"])
        return s
    s["b_k"] = (torch.randn(H, d, r, generator=gen, device="cuda") / math.sqrt(r)).bfloat16()
    s["b_v"] = (torch.randn(H, d, r, generator=gen, device="cuda") / math.sqrt(r)).bfloat16()
    s["q"] = _rand(gen, B, H, d)
    s["out"] = torch.empty(B, H, d, device="cuda")
    s["lse"] = torch.empty(B, H, device="cuda")
    if own:
        lrkv = _framework()
        s["ws"] = lrkv.decode8_workspace(lrkv.make_dims(B, H, d, r, cap, torch.bfloat16), device="cuda")
        s["cache8"] = lrkv.Cache8(**s["cache"])
    return s


def _prepare_pages(s, case, gen):
    B, blocks, page, pages = case["batch"], case["blocks"], case["page"], _pages(case)
    lens = torch.tensor(_lens(case) if case["op"] == "compact" else _shared_lens(case), device="cuda")
    group = case.get("group", 1)
    used = -(-lens // page)
    col = torch.arange(blocks, device="cuda")
    lead = torch.arange(B, device="cuda") // group * group
    first = torch.where(lead == torch.arange(B, device="cuda"), used, 0).cumsum(0) - used
    order = torch.randperm(pages, generator=gen, device="cuda")
    at = first[lead][:, None] + col
    inside = col < used[:, None]
    s["table"] = torch.where(inside, order[at.clamp(0, pages - 1)], -1).to(torch.int32).contiguous()
    s["lens"] = lens.to(torch.int32)
    named = torch.where(inside, s["table"].long(), pages).flatten()
    s["refs"] = torch.zeros(pages + 1, dtype=torch.int32, device="cuda").index_add_(
        0, named, torch.ones_like(named, dtype=torch.int32))[:pages].contiguous()
    s["table_out"], s["lens_out"] = torch.empty_like(s["table"]), torch.empty_like(s["lens"])
    s["refs_out"] = torch.empty_like(s["refs"])
    if case["op"] == "fork":
        one = torch.arange(B, device="cuda")
        pick = torch.randint(0, group, (B,), generator=gen, device="cuda")
        if case["beams"]:
            s["parent"], s["keep"] = torch.clamp(lead + pick, max=B - 1).to(torch.int32), None
        else:   # a quarter ends, a quarter is sampled again from its group's first, a quarter is cut back
            fate = torch.randint(0, 4, (B,), generator=gen, device="cuda")
            s["parent"] = torch.where(fate == 0, -1, torch.where(fate == 1, lead, one)).to(torch.int32)
            cut = (torch.rand(B, generator=gen, device="cuda") * (lens + 1)).long()
            s["keep"] = torch.where(fate == 2, cut, lens).to(torch.int32)
    else:
        s["pools"] = _pool(case, gen, pages)
    if case["op"] == "extend":
        s["new_lens"] = torch.clamp(lens + case["grow"], max=blocks * page).to(torch.int32)
        s["missing"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "compact":
        s["moved"] = torch.empty_like(s["refs"])
        s["live"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        s["ws"] = _framework().pages_workspace(B, blocks, pages, device="cuda")
    return s


# ------------------------------------------------------------- plain form --

def _need(amax):
    """Smallest power of two s, 2^-126 at least, with amax <= 448 s."""
    m, e = torch.frexp(amax)
    k = torch.where(amax > 0, torch.where(m <= 0.875, e - 9, e - 8), -126).clamp(-126, 127)
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _amax(x):
    """Largest finite magnitude over the blocks of rows and the columns of x [.., rows, heads, width]."""
    x = torch.where(torch.isfinite(x), x.abs(), 0.0)
    return x.unflatten(-3, (-1, BLOCK)).amax(dim=(-3, -1))


def _per_row(scale):
    """A scale for each row of its block, [.., rows, heads, 1]."""
    return scale.repeat_interleave(BLOCK, dim=-2)[..., None]


def _to8(x):
    return x.clamp(-448, 448).to(E4M3)


def _round8(x):
    """(8-bit values, scales of the blocks) of rows x [.., rows, heads, width] that fill their blocks from the start."""
    rows = x.shape[-3]
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -rows % BLOCK))
    scale = _need(_amax(x))
    return _to8(x / _per_row(scale))[..., :rows, :, :], scale


def _places(s, row):
    """Index of logical rows [batch, n] among all rows of the cache (of its pool where it is paged)."""
    if s["block_table"] is None:
        return torch.arange(row.shape[0], device="cuda")[:, None] * s["case"]["cap"] + row
    page = s["block_table"].long().gather(1, row // PAGE)
    return page * PAGE + row % PAGE


def _logical(s, name, heads, width):
    """[batch, rows, heads, width] fp32 values that the 8-bit cache stands for."""
    cap = s["case"]["cap"]
    x, scale = s["cache"][name].reshape(-1, heads, width), s["cache"][name + "_scale"].reshape(-1, heads)
    row = torch.arange(cap, device="cuda").expand(s["case"]["batch"], cap)
    at = _places(s, row)
    blocks = s["cache"][name + "_scale"].shape[1]
    rows = s["cache"][name].shape[1]
    return x.view(torch.uint8)[at].view(E4M3).float() * scale[at // rows * blocks + at % rows // BLOCK][..., None]


def _plain_decode(s):
    case = s["case"]
    k_s, v_s, z_k, z_v = (_logical(s, *w) for w in _widths(case))
    q = s["q"].float()
    p = torch.einsum("bhd,hdr->bhr", q, s["b_k"].float())
    score = torch.einsum("bhd,bld->bhl", q, k_s[:, :, 0]) + torch.einsum("bhr,blhr->bhl", p, z_k)
    score = score / math.sqrt(case["dim"])
    seen = torch.arange(case["cap"], device="cuda") < s["lens"].long()[:, None]
    score = torch.where(seen[:, None], score, -math.inf)
    lse = torch.logsumexp(score, dim=-1)
    a = torch.where(torch.isinf(score), 0.0, torch.exp(score - lse[..., None]))
    out = torch.einsum("bhl,bld->bhd", a, v_s[:, :, 0])
    out = out + torch.einsum("bhr,hdr->bhd", torch.einsum("bhl,blhr->bhr", a, z_v), s["b_v"].float())
    return {"out": out, "lse": lse}


def _plain_quantize(s):
    """Over the blocks that a call may touch, from the one that holds its first row on."""
    case = s["case"]
    B, n, cap = case["batch"], case["new"], case["cap"]
    start = s["lens"].long()[:, None]
    end = start + (s["new_lens"].long()[:, None] if s["new_lens"] is not None else n)
    wide = -(-(n + BLOCK - 1) // BLOCK) * BLOCK
    row = start // BLOCK * BLOCK + torch.arange(wide, device="cuda")
    there = row < cap
    fresh, before = there & (row >= start) & (row < end), row < start
    at = _places(s, row.clamp(max=cap - 1))
    for name, heads, width in _widths(case):
        held, scales = s["cache"][name], s["cache"][name + "_scale"]
        rows, blocks = held.shape[1], scales.shape[1]
        flat = held.view(torch.uint8).reshape(-1, heads, width)
        block_at = (at // rows * blocks + at % rows // BLOCK)[:, ::BLOCK]
        new = s[name].reshape(B, n, heads, width).float()
        new = new.gather(1, (row - start).clamp(0, n - 1)[:, :, None, None].expand(-1, -1, heads, width))
        new = torch.where(fresh[..., None, None], new, 0.0)
        had, has = (m.unflatten(1, (-1, BLOCK)).any(-1)[..., None] for m in (before, fresh))
        old_scale = scales.reshape(-1, heads)[block_at]
        scale = torch.maximum(_need(_amax(new)), torch.where(had, old_scale, 0.0))
        old = flat[at].view(E4M3).float() * _per_row(torch.where(had, old_scale, 1.0) / scale)
        grown = _per_row((had & has & (scale > old_scale)).float()) > 0
        put = torch.where(fresh[..., None, None], _to8(new / _per_row(scale)).view(torch.uint8),
                          _to8(old).view(torch.uint8))
        change = (fresh[..., None, None] | (grown & (before & there)[..., None, None])).expand_as(put)
        b, i = change.any(-1).any(-1).nonzero(as_tuple=True)
        flat[at[b, i]] = torch.where(change[b, i], put[b, i], flat[at[b, i]])
        b, i = has[..., 0].nonzero(as_tuple=True)
        scales.reshape(-1, heads)[block_at[b, i]] = scale[b, i]
    return dict(s["cache"])


def _in_use(table, lens, page, pages):
    """Which entries of a table name a page of the pool that holds rows."""
    col = torch.arange(table.shape[1], device="cuda")
    return (col < -(-lens.long()[:, None] // page)) & (table >= 0) & (table < pages)


def _named(table, use, pages):
    """How many of the entries in use name each page."""
    at = torch.where(use, table.long(), pages).flatten()
    return torch.zeros(pages + 1, dtype=torch.int32, device="cuda").index_add_(
        0, at, torch.ones_like(at, dtype=torch.int32))[:pages]


def _plain_fork(s):
    page, pages = s["case"]["page"], s["refs"].shape[0]
    parent = s["parent"].long()
    lens = torch.where(parent >= 0, s["lens"][parent.clamp(min=0)], 0)
    if s["keep"] is not None:
        lens = torch.minimum(lens, s["keep"])
    col = torch.arange(s["case"]["blocks"], device="cuda")
    table = torch.where(col < -(-lens.long()[:, None] // page), s["table"][parent.clamp(min=0)], -1)
    refs = s["refs"] - _named(s["table"], _in_use(s["table"], s["lens"], page, pages), pages)
    refs = refs + _named(table, _in_use(table, lens, page, pages), pages)
    return {"table": table, "lens": lens, "refs": refs}


def _plain_extend(s):
    case = s["case"]
    B, page, pages = case["batch"], case["page"], s["refs"].shape[0]
    one = torch.arange(B, device="cuda")
    length, refs = s["lens"].long(), s["refs"].long()
    new = torch.maximum(length, s["new_lens"].long())
    begun = torch.where(length % page > 0, length // page, 0)
    mine = s["table"].long().gather(1, begun[:, None])[:, 0]
    writes = (new > length) & (length % page > 0)
    at = torch.where(writes, mine, pages)
    writers = torch.zeros(pages + 1, dtype=torch.int64, device="cuda").index_add_(0, at, torch.ones_like(at))
    last = torch.full((pages + 1,), -1, device="cuda").scatter_reduce_(0, at, one, "amax")
    count = refs[mine.clamp(min=0)]
    copies = writes & (count > 1) & ~((count == writers[at]) & (last[at] == one))
    have, want = -(-length // page), -(-new // page)
    need = want - have + copies
    first = need.cumsum(0) - need
    free = s["refs"] == 0
    rank = free.cumsum(0) - 1
    page_of = torch.full((pages + 1,), -1, device="cuda").scatter_(
        0, torch.where(free, rank, pages), torch.arange(pages, device="cuda"))
    missing = (need.sum() - free.sum()).clamp(min=0)
    done = missing == 0
    col = torch.arange(case["blocks"], device="cuda")
    fresh = (col >= have[:, None]) & (col < want[:, None])
    taken = first[:, None] + copies[:, None] + col - have[:, None]
    own_copy = copies[:, None] & (col == begun[:, None])
    taken = torch.where(own_copy, first[:, None], taken)
    put = page_of[taken.clamp(0, pages)]
    table = torch.where(done & (fresh | own_copy), put, s["table"].long()).to(torch.int32)
    back = torch.zeros(pages + 1, dtype=torch.int64, device="cuda").index_add_(
        0, torch.where(copies, mine, pages), torch.ones_like(mine))[:pages]
    refs_out = torch.where(done, torch.where(free & (rank < need.sum()), 1, refs - back), refs).to(torch.int32)
    b = (copies & done).nonzero()[:, 0]
    to, frm, rows = page_of[first[b]], mine[b], (length % page)[b]
    for name, pool in s["pools"].items():
        each = page // pool.shape[1]
        raw = pool.view(torch.uint8) if pool.dtype == E4M3 else pool
        keep = torch.arange(pool.shape[1], device="cuda") * each < rows[:, None]
        keep = keep.reshape(*keep.shape, *[1] * (pool.dim() - 2))
        raw[to] = torch.where(keep, raw[frm], raw[to])
    return {"table": table, "lens": torch.where(done, new, length).to(torch.int32), "refs": refs_out,
            "missing": missing.to(torch.int32).reshape(1)} | s["pools"]


def _plain_compact(s):
    page, pages = s["case"]["page"], s["refs"].shape[0]
    at = torch.arange(pages, device="cuda")
    held = s["refs"] > 0
    live = held.sum()
    high, hole = held & (at >= live), ~held & (at < live)
    # the k-th live page past the end goes into the k-th free one before it
    hole_of = torch.full((pages + 1,), -1, device="cuda").scatter_(
        0, torch.where(hole, hole.cumsum(0) - 1, pages), at)
    moved = torch.where(high, hole_of[(high.cumsum(0) - 1).clamp(min=0)], torch.where(held, at, -1))
    frm = high.nonzero()[:, 0]
    to = moved[frm]
    for pool in s["pools"].values():
        raw = pool.view(torch.uint8) if pool.dtype == E4M3 else pool
        raw[to] = raw[frm]
    refs = torch.where(at < live, s["refs"], 0)
    refs[to] = s["refs"][frm]
    use = _in_use(s["table"], s["lens"], page, pages)
    table = torch.where(use, moved[s["table"].long().clamp(0, pages - 1)].to(torch.int32), s["table"])
    return {"table": table, "refs": refs, "moved": moved.to(torch.int32),
            "live": live.to(torch.int32).reshape(1)} | s["pools"]


# -------------------------------------------------------------------- run --

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"decode": _plain_decode, "quantize": _plain_quantize, "fork": _plain_fork, "extend": _plain_extend,
                "compact": _plain_compact}[op](s)
    lrkv = _framework()
    if op == "decode":
        lrkv.decode8(s["q"], s["cache8"], s["b_k"], s["b_v"], s["lens"], block_table=s["block_table"],
                     out=s["out"], lse=s["lse"], ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "quantize":
        lrkv.quantize(s["k_s"], s["v_s"], s["z_k"], s["z_v"], s["lens"], s["cache8"], new_lens=s["new_lens"],
                      block_table=s["block_table"], ws=s["ws"])
        return dict(s["cache"])
    if op == "fork":
        lrkv.pages_fork(s["table"], s["lens"], s["refs"], case["page"], parent=s["parent"], keep=s["keep"],
                        table_out=s["table_out"], lens_out=s["lens_out"], refs_out=s["refs_out"], ws=s["ws"])
        return {"table": s["table_out"], "lens": s["lens_out"], "refs": s["refs_out"]}
    pools = list(s["pools"].values())
    if op == "extend":
        lrkv.pages_extend(pools, s["table"], s["lens"], s["refs"], case["page"], s["new_lens"],
                          table_out=s["table_out"], lens_out=s["lens_out"], refs_out=s["refs_out"],
                          missing=s["missing"], ws=s["ws"])
        return {"table": s["table_out"], "lens": s["lens_out"], "refs": s["refs_out"],
                "missing": s["missing"]} | s["pools"]
    lrkv.pages_compact(pools, s["table"], s["lens"], s["refs"], case["page"], table_out=s["table_out"],
                       refs_out=s["refs_out"], moved=s["moved"], live=s["live"], ws=s["ws"])
    return {"table": s["table_out"], "refs": s["refs_out"], "moved": s["moved"], "live": s["live"]} | s["pools"]


# ------------------------------------------------------------ definitions --

def _sequence(s, name, heads, width, b, n):
    """[n, heads, width] fp64 values of sequence b's first n rows, page by page."""
    x, scale = s["cache"][name], s["cache"][name + "_scale"]
    if s["block_table"] is None:
        rows, blocks = x[b].double(), scale[b].double()
    else:
        pages = s["block_table"][b].long()
        rows = x.view(torch.uint8)[pages].view(E4M3).flatten(0, 1).double()
        blocks = scale[pages].flatten(0, 1).double()
    rows, blocks = rows[:n].reshape(n, heads, width), blocks.reshape(-1, heads)
    return rows * blocks[torch.arange(n, device="cuda") // BLOCK][..., None]


def _exact_decode(case, s):
    outs, lses = [], []
    for b, n in enumerate(_lens(case)):
        if n == 0:
            outs.append(torch.zeros(case["heads"], case["dim"], dtype=torch.float64, device="cuda"))
            lses.append(torch.full((case["heads"],), -math.inf, dtype=torch.float64, device="cuda"))
            continue
        k_s, v_s, z_k, z_v = (_sequence(s, *w, b, n) for w in _widths(case))
        out, lse = [], []
        for h in range(case["heads"]):
            key = k_s[:, 0] + z_k[:, h] @ s["b_k"][h].double().T
            x = key @ s["q"][b, h].double() / math.sqrt(case["dim"])
            e = torch.exp(x - x.max())
            value = v_s[:, 0] + z_v[:, h] @ s["b_v"][h].double().T
            out.append((e / e.sum()) @ value)
            lse.append(x.max() + torch.log(e.sum()))
        outs.append(torch.stack(out))
        lses.append(torch.stack(lse))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _nearest8(x):
    """fp64 values rounded to the nearest of sign, 4 bits of exponent and 3 of mantissa, ties to even, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_quantize(case, s):
    """Block by block of each sequence: the cache is laid out anew in 64 bits."""
    cap = case["cap"]
    got = {}
    for name, heads, width in _widths(case):
        values, scales = s["cache"][name].double(), s["cache"][name + "_scale"].double()
        for b, (start, n) in enumerate(zip(_lens(case), _new(case))):
            new = s[name][b, :n].double().reshape(n, heads, width)
            at = torch.arange(start, start + n, device="cuda")
            first, last = start // BLOCK, -(-(start + n) // BLOCK)
            padded = torch.zeros((last - first) * BLOCK, heads, width, dtype=torch.float64, device="cuda")
            padded[at - first * BLOCK] = new
            top = padded.abs().unflatten(0, (-1, BLOCK)).amax(dim=(1, 3))
            scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(min=-126))
            scale = torch.where(top > 448 * scale, 2 * scale, scale)   # (a logarithm next to a whole number)
            row = torch.arange(first * BLOCK, min(last * BLOCK, cap), device="cuda")
            if s["block_table"] is None:
                lead, inner = torch.full_like(row, b), row
            else:
                lead, inner = s["block_table"][b].long()[row // PAGE], row % PAGE
            blk = (lead[::BLOCK], inner[::BLOCK] // BLOCK)
            held = scales[blk].reshape(-1, heads)
            if start % BLOCK:
                scale[0] = torch.maximum(scale[0], held[0])
                k = start % BLOCK
                old = values[lead[:k], inner[:k]].reshape(k, heads, width)
                values[lead[:k], inner[:k]] = _nearest8(old * (held[0] / scale[0])[None, :, None]).reshape(
                    values[lead[:k], inner[:k]].shape)
            mine = (row >= start) & (row < start + n)
            put = _nearest8(new / scale[at // BLOCK - first][..., None])
            values[lead[mine], inner[mine]] = put.reshape(values[lead[mine], inner[mine]].shape)
            scales[blk] = scale.reshape(scales[blk].shape)
        got[name], got[name + "_scale"] = values, scales
    return got


def exact(case, seed):
    if case["op"] not in ("decode", "quantize"):
        return None   # whole numbers and copies
    s = prepare(case, seed)
    return _exact_decode(case, s) if case["op"] == "decode" else _exact_quantize(case, s)
