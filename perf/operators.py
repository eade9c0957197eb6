"""Cases of the operators that keep a factored cache inside a token budget: attention weights
accumulated per cache row (by a decode step, by a prompt's queries), eviction of the rows that
gathered least, and rotary positions with several axes for rows that no longer sit at their position.

`run` computes the plain form (elementary torch operations, 32 bits, angles in 64) or, with `own`,
calls the framework.  `exact` restates the definitions in 64 bits along another route: keys rebuilt
per head, rotations as complex numbers, the selection as a sort on the host.
"""
import math

import numpy as np
import torch

own = False

PAGE = 256          # rows per page of the paged cases
BASE = 10000.0      # frequency base of the rotary cases


def _framework():
    from compressed_cache_decode_gb300 import lrkv
    return lrkv


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one short sequence of the smallest bf16 decode workload: latency of a lone request
        dict(name="decode_weights_one", op="decode", batch=1, heads=16, dim=64, rank=28, lo=517, hi=517, cap=576,
             paged=False, normed=False, empty=False),
        # batched serving from pages, ragged lengths (the batched decode workload's shape)
        dict(name="decode_weights_paged", op="decode", batch=32, heads=32, dim=128, rank=56, lo=1024, hi=8192,
             cap=8192, paged=True, normed=False, empty=False),
        # few long contexts (the long-context workload): split over the length and joined
        dict(name="decode_weights_long", op="decode", batch=4, heads=32, dim=128, rank=48, lo=65536, hi=65536,
             cap=65536, paged=False, normed=False, empty=False),
        # a prompt scored by its last 32 queries before its cache is cut down
        dict(name="prompt_weights_window", op="prompt", batch=4, heads=32, dim=128, rank=64, lo=15000, hi=16384,
             cap=16384, new=128, window=32, paged=False, normed=False),
        # every query of a prompt (the prefill workload's shape)
        dict(name="prompt_weights_full", op="prompt", batch=2, heads=32, dim=128, rank=64, lo=4096, hi=4096,
             cap=4096, new=4096, window=4096, paged=False, normed=False),
        # a cache at its budget: one row goes for each new token
        dict(name="evict_step", op="evict", batch=32, heads=32, dim=128, rank=56, lo=4097, hi=4097, cap=4352,
             budget=4096, sink=4, recent=256, paged=True, normed=False, axes=0, order=True, dtype="bf16"),
        # prompts of different lengths brought down to the budget, normalised keys, positions carried along
        dict(name="evict_prompts", op="evict", batch=8, heads=32, dim=128, rank=48, lo=9001, hi=16384, cap=16384,
             budget=4096, sink=4, recent=512, paged=False, normed=True, axes=3, order=False, dtype="bf16"),
        # one very long document
        dict(name="evict_long", op="evict", batch=1, heads=16, dim=64, rank=32, lo=262144, hi=262144, cap=262144,
             budget=32768, sink=16, recent=2048, paged=False, normed=False, axes=0, order=True, dtype="f32"),
        # the queries of one decode step, text after an image
        dict(name="rotate_step", op="rotate", batch=32, new=1, heads=32, dim=128, axes=3, dtype="bf16"),
        # the queries of a long prompt of text, images and video
        dict(name="rotate_prompt", op="rotate", batch=2, new=4096, heads=32, dim=128, axes=3, dtype="bf16"),
        # decode over short evicted caches whose rows carry image positions
        dict(name="rope_axes_short", op="rope", batch=8, heads=16, dim=64, rank=32, lo=700, hi=3001, cap=3008,
             axes=3, weighted=True, empty=True),
        # decode over long caches of text, images and video
        dict(name="rope_axes_long", op="rope", batch=4, heads=32, dim=128, rank=48, lo=32768, hi=32768, cap=32768,
             axes=3, weighted=True, empty=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "prompt", "evict", "rotate", "rope"])
    if op == "rotate":
        heads, dim, axes = rng.choice([1, 5, 8, 16, 32]), rng.choice([32, 64, 80, 128]), rng.randint(1, 4)
        batch = _log(rng, 1, 32)
        new = _log(rng, 1, max(1, (2 * 4096 * 32 * 128) // (batch * heads * dim * 2)))
        return dict(op=op, batch=batch, new=min(new, 20000), heads=heads, dim=dim, axes=axes,
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "prompt":
        heads, dim, rank = rng.choice([8, 16, 32]), rng.choice([64, 128]), rng.choice([16, 32, 48, 56, 64])
        batch = _log(rng, 1, 8)
        hi = _log(rng, 64, int(4096 * math.sqrt(2 / batch)))
        lo = rng.randint(max(1, hi // 2), hi)
        new = rng.randint(1, lo)
        return dict(op=op, batch=batch, heads=heads, dim=dim, rank=rank, lo=lo, hi=hi,
                    cap=-(-hi // PAGE) * PAGE, new=new, window=min(new, _log(rng, 1, new)),
                    paged=rng.random() < 0.4, normed=rng.random() < 0.3)
    if op == "evict":
        heads, dim, rank = rng.choice([8, 16, 32]), rng.choice([64, 128]), rng.choice([16, 32, 48, 56, 64])
        batch = _log(rng, 1, 32)
        hi = _log(rng, 64, max(128, 65536 // batch))
        lo = rng.randint(max(1, hi // 2), hi)
        budget = rng.randint(2, hi)
        recent = rng.randint(0, budget // 2)
        return dict(op=op, batch=batch, heads=heads, dim=dim, rank=rank, lo=lo, hi=hi,
                    cap=-(-hi // PAGE) * PAGE, budget=budget, sink=rng.randint(0, min(8, budget - recent)),
                    recent=recent, paged=rng.random() < 0.4, normed=rng.random() < 0.4, axes=rng.choice([0, 1, 3, 4]),
                    order=rng.random() < 0.6, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "rope":
        heads, dim, rank = rng.choice([8, 16, 32]), rng.choice([64, 128]), rng.choice([16, 32, 48, 64])
        batch = _log(rng, 1, 16)
        hi = _log(rng, 16, max(32, 4 * 32768 // batch * 32 // heads // 2))
        return dict(op=op, batch=batch, heads=heads, dim=dim, rank=rank, lo=rng.randint(1, hi), hi=hi,
                    cap=hi + rng.randint(0, 40), axes=rng.randint(1, 4), weighted=rng.random() < 0.7,
                    empty=rng.random() < 0.3)
    heads, dim = rng.choice([(16, 64), (32, 64), (16, 128), (32, 128)])
    rank = rng.choice([28, 32, 48, 56, 64])
    batch = _log(rng, 1, 32)
    hi = _log(rng, 16, max(64, 4 * 65536 // batch // 2))
    return dict(op="decode", batch=batch, heads=heads, dim=dim, rank=rank, lo=rng.randint(1, hi), hi=hi,
                cap=-(-hi // PAGE) * PAGE, paged=rng.random() < 0.4, normed=rng.random() < 0.3,
                empty=rng.random() < 0.3)


def _lens(case):
    """Lengths spread over [lo, hi], the longest first, the last one empty where the case says so."""
    span = case["hi"] - case["lo"]
    lens = [case["hi"] - int(span * ((b * 0.6180339887) % 1.0)) for b in range(case["batch"])]
    if case.get("empty") and len(lens) > 1:
        lens[-1] = 0
    return lens


def _sections(case):
    """Pairs of each axis: halves and quarters as vision models split them, in whole pairs."""
    pairs, axes = case["dim"] // 2, case["axes"]
    first = pairs // 4 if axes > 1 else pairs
    rest = [(pairs - first) // (axes - 1)] * (axes - 1) if axes > 1 else []
    if rest:
        rest[-1] += pairs - first - sum(rest)
    return [first] + rest


def work(case):
    op = case["op"]
    if op == "rotate":
        n = case["batch"] * case["new"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (2 * case["heads"] * case["dim"] * size + 4 * case["axes"]),
                "flops": 3 * n * case["heads"] * case["dim"]}
    B, H, d, r, lens = case["batch"], case["heads"], case["dim"], case["rank"], _lens(case)
    total = sum(lens)
    key, scale = 2 * (d + H * r), 4 * H if case.get("normed") else 0
    if op == "decode":
        return {"bytes": total * (2 * key + scale + 8) + 2 * 2 * H * d * r + B * H * (6 * d + 4),
                "flops": total * H * 4 * (d + r) + B * H * 4 * d * r}
    if op == "rope":
        return {"bytes": total * (2 * key + 4 * case["axes"] + (8 if case["weighted"] else 0)) + 2 * 2 * H * d * r
                + B * H * (6 * d + 4),
                "flops": total * H * (4 * d + 4 * r + 2 * d * r)}
    if op == "prompt":
        seen = [max(0, L - case["window"]) * case["window"] + case["window"] * (case["window"] + 1) // 2 for L in lens]
        return {"bytes": total * (key + scale + 8) + 2 * H * d * r + B * H * case["window"] * (2 * d + 4),
                "flops": sum(seen) * H * 2 * (d + r) + B * case["window"] * H * 2 * d * r}
    size = 2 if case["dtype"] == "bf16" else 4
    row = 2 * size * (d + H * r) + scale + 4 * case["axes"]
    moved = 0.0
    for L in lens:
        new = min(L, case["budget"])
        if L > new:
            held = min(case["recent"], L - new)      # protected rows past the budget
            free = L - case["recent"] - case["sink"]
            moved += held + max(0, new - case["recent"] - case["sink"]) * max(0, L - new - held) / max(1, free)
    kept = sum(min(L, case["budget"]) for L in lens)
    return {"bytes": total * (8 if case["order"] else 4) + kept * 12 + 2 * moved * row, "flops": total}


# ----------------------------------------------------------------- inputs --

def _rand(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _positions(case, gen, n):
    """[batch, n, axes] int32: runs of text (all axes advance together) between images (a grid at one time)."""
    at = torch.arange(n, device="cuda").expand(case["batch"], n)
    run, side = 600, 20
    base = at // run * (run - 300) + torch.randint(0, 500, (case["batch"], 1), generator=gen, device="cuda")
    inside = at % run
    image = inside >= 200                     # 200 text tokens, then a 20 x 20 image
    cell = inside - 200
    steps = [torch.zeros_like(cell), cell // side, cell % side, cell // (side * 4)][: case["axes"]]
    return torch.stack([base + torch.where(image, 200 + s, inside) for s in steps], dim=-1).to(torch.int32).contiguous()


def _max_pos(case):
    n = case["new"] if case["op"] == "rotate" else case["cap"]
    return n // 600 * 300 + 1200


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    op, B, H, d = case["op"], case["batch"], case["heads"], case["dim"]
    s = {"case": case}
    if op in ("rotate", "rope"):
        s["sections"] = _sections(case)
        if own:
            s["table"] = _framework().rope_table(_max_pos(case), d, BASE)
    if op == "rotate":
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["x"] = _rand(gen, B, case["new"], H, d, dtype=dtype)
        s["positions"] = _positions(case, gen, case["new"])
        s["out"] = torch.empty_like(s["x"])
        return s

    r, cap = case["rank"], case["cap"]
    dtype = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    rows = (B, cap)
    if case.get("paged"):
        blocks = cap // PAGE
        pages = B * blocks + 3
        rows = (pages, PAGE)
        order = torch.randperm(pages, generator=gen, device="cuda")
        s["table_of_pages"] = order[: B * blocks].reshape(B, blocks).to(torch.int32)
    else:
        s["table_of_pages"] = None
    names = ("k_s", "z_k") if op == "prompt" else ("k_s", "v_s", "z_k", "z_v")
    for name in names:
        s[name] = _rand(gen, *rows, *((H, r) if name.startswith("z") else (d,)), dtype=dtype)
    s["key_scale"] = (0.5 + 0.5 * torch.rand(B, H, cap, generator=gen, device="cuda")) if case.get("normed") else None

    if op == "evict":
        # most rows gather next to nothing, a few almost everything; rows nothing looked at tie at zero
        u = torch.rand(B, cap, generator=gen, device="cuda")
        s["weights"] = torch.where(u < 0.3, torch.zeros_like(u), (1.0 - u).pow(-0.7) - 1.0)
        s["weights_out"] = torch.zeros_like(s["weights"])
        s["positions"] = _positions(case, gen, cap) if case["axes"] else None
        s["order"] = None
        if case["order"]:
            # tokens seen so far: rows left by earlier evictions lie in any order, later rows behind them
            back = min(case["budget"], min(_lens(case))) // 2
            age = torch.arange(cap, device="cuda").repeat(B, 1)
            head = torch.rand(B, back, generator=gen, device="cuda").argsort(dim=1)
            age[:, :back] = head
            s["order"] = (age * 3).to(torch.int32).contiguous()
        s["order_out"] = torch.zeros(B, cap, dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.zeros_like(s["lens"])
        s["kept"] = torch.zeros(B, case["budget"], dtype=torch.int32, device="cuda")
        if own:
            s["ws"] = _framework().evict_workspace(B, cap, case["budget"], device="cuda")
        return s

    s["b_k"] = (torch.randn(H, d, r, generator=gen, device="cuda") / math.sqrt(r)).bfloat16()
    s["weights_out"] = torch.zeros(B, cap, device="cuda")
    # what earlier queries left: a few rows stand out, the others are of the size of one call's own share
    share = H * case.get("window", 1) / case["hi"]
    s["weights"] = (torch.rand(B, cap, generator=gen, device="cuda").pow(-0.5) - 1.0) * share
    s["decay"] = 0.97
    if op == "prompt":
        s["q"] = _rand(gen, B, case["new"], H, d)
        at = _logical(s, "k_s"), _logical(s, "z_k")
        w = case["window"]
        lse = torch.logsumexp(_window_scores(s, *at), dim=-1)
        s["lse"] = torch.zeros(B, H, case["new"], device="cuda")
        s["lse"][:, :, case["new"] - w:] = lse
        if own:
            lrkv = _framework()
            s["ws"] = lrkv.prefill_weights_workspace(
                lrkv.make_dims(B, H, d, r, cap, torch.bfloat16), w, device="cuda")
        return s
    s["b_v"] = (torch.randn(H, d, r, generator=gen, device="cuda") / math.sqrt(r)).bfloat16()
    s["q"] = _rand(gen, B, H, d)
    s["out"] = torch.empty(B, H, d, device="cuda")
    s["lse"] = torch.empty(B, H, device="cuda")
    if op == "rope":
        s["positions"] = _positions(case, gen, cap)
    if own:
        lrkv = _framework()
        dims = lrkv.make_dims(B, H, d, r, cap, torch.bfloat16)
        s["ws"] = (lrkv.decode_rope_axes_workspace(dims, device="cuda") if op == "rope"
                   else lrkv.decode_weighted_workspace(dims, device="cuda"))
    return s


# ------------------------------------------------------------- plain form --

def _logical(s, name):
    """[batch, rows, ...] of a cache tensor, through the block table where the cache is paged."""
    t = s[name]
    if s["table_of_pages"] is None:
        return t
    t = t[s["table_of_pages"].long()]
    return t.flatten(1, 2)


def _window_scores(s, k_s, z_k):
    """[batch, heads, window, rows] fp32 scaled scores of the window's queries, -inf where a query does not look."""
    case = s["case"]
    w, new, rows = case["window"], case["new"], k_s.shape[1]
    q = s["q"][:, new - w:].float()
    p = torch.einsum("bthd,hdr->bthr", q, s["b_k"].float())
    score = torch.einsum("bthd,bld->bhtl", q, k_s.float())
    score = score + torch.einsum("bthr,blhr->bhtl", p, z_k.float())
    score = score / math.sqrt(case["dim"])
    if s["key_scale"] is not None:
        score = score * s["key_scale"][:, :, None, :]
    at = s["lens"].long()[:, None] - w + torch.arange(w, device="cuda")
    seen = torch.arange(rows, device="cuda") <= at[:, :, None]
    return torch.where(seen[:, None], score, -math.inf)


def _carry(s, fresh, new):
    """decay times the earlier weights of the rows that were there, plus the fresh ones; rows past the lengths stay."""
    row = torch.arange(fresh.shape[1], device="cuda")
    lens = s["lens"].long()[:, None]
    old = torch.where(row < lens - new, s["weights"], 0.0)
    return torch.where(row < lens, s["decay"] * old + fresh, s["weights_out"])


def _angles(positions, sections, dim):
    """[..., dim / 2] fp64 angle of every pair: its axis' position times its frequency."""
    k = torch.arange(dim // 2, device="cuda", dtype=torch.float64)
    axis = torch.repeat_interleave(torch.arange(len(sections), device="cuda"), torch.tensor(sections, device="cuda"))
    return positions[..., axis].double() * BASE ** (-2.0 * k / dim)


def _turn(x, angle):
    """Every pair (2k, 2k + 1) of x turned by angle[..., k]."""
    c, n = angle.cos().float(), angle.sin().float()
    a, b = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack((a * c - b * n, a * n + b * c), dim=-1).flatten(-2)


def _softmax_out(s, score, v_s, z_v):
    """(out, lse, weights of each row summed over the heads) from masked scores [batch, heads, rows]."""
    lse = torch.logsumexp(score, dim=-1)
    a = torch.where(torch.isinf(score), 0.0, torch.exp(score - lse[..., None]))
    out = torch.einsum("bhl,bld->bhd", a, v_s.float())
    out = out + torch.einsum("bhr,hdr->bhd", torch.einsum("bhl,blhr->bhr", a, z_v.float()), s["b_v"].float())
    return out, lse, a.sum(dim=1)


def _plain_decode(s):
    case = s["case"]
    k_s, v_s, z_k, z_v = (_logical(s, n) for n in ("k_s", "v_s", "z_k", "z_v"))
    q = s["q"].float()
    p = torch.einsum("bhd,hdr->bhr", q, s["b_k"].float())
    score = torch.einsum("bhd,bld->bhl", q, k_s.float()) + torch.einsum("bhr,blhr->bhl", p, z_k.float())
    score = score / math.sqrt(case["dim"])
    if s["key_scale"] is not None:
        score = score * s["key_scale"]
    seen = torch.arange(k_s.shape[1], device="cuda") < s["lens"].long()[:, None]
    out, lse, fresh = _softmax_out(s, torch.where(seen[:, None], score, -math.inf), v_s, z_v)
    return {"out": out, "lse": lse, "weights": _carry(s, fresh, 1)}


def _plain_rope(s):
    case = s["case"]
    key = s["k_s"].float()[:, :, None] + torch.einsum("blhr,hdr->blhd", s["z_k"].float(), s["b_k"].float())
    key = _turn(key, _angles(s["positions"], s["sections"], case["dim"])[:, :, None])
    score = torch.einsum("bhd,blhd->bhl", s["q"].float(), key) / math.sqrt(case["dim"])
    seen = torch.arange(key.shape[1], device="cuda") < s["lens"].long()[:, None]
    out, lse, fresh = _softmax_out(s, torch.where(seen[:, None], score, -math.inf), s["v_s"], s["z_v"])
    got = {"out": out, "lse": lse}
    if case["weighted"]:
        got["weights"] = _carry(s, fresh, 1)
    return got


def _plain_prompt(s):
    score = _window_scores(s, _logical(s, "k_s"), _logical(s, "z_k"))
    w = s["case"]["window"]
    lse = s["lse"][:, :, s["case"]["new"] - w:, None]
    fresh = torch.where(torch.isinf(score), 0.0, torch.exp(score - lse)).sum(dim=(1, 2))
    return {"weights": _carry(s, fresh, s["case"]["new"])}


def _plain_evict(s):
    case = s["case"]
    B, cap, budget = case["batch"], case["cap"], case["budget"]
    row = torch.arange(cap, device="cuda")
    lens = s["lens"].long()
    there = row < lens[:, None]
    age = s["order"].long() if s["order"] is not None else row.expand(B, cap)
    seen = torch.where(there, age, -1).amax(dim=1) + 1
    held = there & ((age < case["sink"]) | (age >= seen[:, None] - case["recent"]))
    # rows by weight, the held ones first and the absent ones last; equal weights by index
    w = torch.where(torch.isnan(s["weights"]), -math.inf, s["weights"])
    by_weight = torch.sort(w, dim=1, descending=True, stable=True).indices
    group = torch.where(held, 0, torch.where(there, 1, 2))
    by_group = torch.sort(group.gather(1, by_weight), dim=1, stable=True).indices
    ranked = by_weight.gather(1, by_group)
    rank = torch.empty_like(ranked).scatter_(1, ranked, row.expand(B, cap).contiguous())
    new = torch.minimum(lens, torch.full_like(lens, budget))
    keep = rank < new[:, None]
    holes = (~keep & (row < new[:, None])).nonzero()
    moved = (keep & (row >= new[:, None])).nonzero()
    source = row.repeat(B, 1)
    source[holes[:, 0], holes[:, 1]] = moved[:, 1]

    inside = row < new[:, None]
    s["weights_out"].copy_(torch.where(inside, s["weights"].gather(1, source), s["weights_out"]))
    s["order_out"].copy_(torch.where(inside, age.gather(1, source).to(torch.int32), s["order_out"]))
    s["new_lens"].copy_(new)
    s["kept"].copy_(torch.where(inside, source, -1)[:, :budget])
    b, to, frm = holes[:, 0], holes[:, 1], moved[:, 1]
    pages = s["table_of_pages"]
    for name in ("k_s", "v_s", "z_k", "z_v"):
        if pages is None:
            s[name][b, to] = s[name][b, frm]
        else:
            s[name][pages[b, to // PAGE].long(), to % PAGE] = s[name][pages[b, frm // PAGE].long(), frm % PAGE]
    if s["key_scale"] is not None:
        s["key_scale"][b, :, to] = s["key_scale"][b, :, frm]
    if s["positions"] is not None:
        s["positions"][b, to] = s["positions"][b, frm]
    return _evicted(s)


def _evicted(s):
    names = ("new_lens", "kept", "weights_out", "order_out", "k_s", "v_s", "z_k", "z_v", "key_scale", "positions")
    return {n: s[n] for n in names if s[n] is not None}


# -------------------------------------------------------------------- run --

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "rotate":
            angle = _angles(s["positions"], s["sections"], case["dim"])[:, :, None]
            return _turn(s["x"], angle).to(s["x"].dtype)
        return {"decode": _plain_decode, "rope": _plain_rope, "prompt": _plain_prompt, "evict": _plain_evict}[op](s)
    lrkv = _framework()
    if op == "rotate":
        return lrkv.rope_rotate(s["x"], s["positions"], s["table"], s["sections"], out=s["out"])
    if op == "decode":
        lrkv.decode_weighted(s["q"], s["k_s"], s["v_s"], s["z_k"], s["z_v"], s["b_k"], s["b_v"], s["lens"],
                             s["weights"], decay=s["decay"], weights_out=s["weights_out"],
                             key_scale=s["key_scale"], block_table=s["table_of_pages"], out=s["out"], lse=s["lse"],
                             ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"], "weights": s["weights_out"]}
    if op == "rope":
        weights = s["weights"] if case["weighted"] else None
        lrkv.decode_rope_axes(s["q"], s["k_s"], s["v_s"], s["z_k"], s["z_v"], s["b_k"], s["b_v"], s["table"],
                              s["positions"], s["sections"], s["lens"], weights=weights, decay=s["decay"],
                              weights_out=s["weights_out"] if case["weighted"] else None, out=s["out"],
                              lse=s["lse"], ws=s["ws"])
        got = {"out": s["out"], "lse": s["lse"]}
        if case["weighted"]:
            got["weights"] = s["weights_out"]
        return got
    if op == "prompt":
        lrkv.prefill_weights(s["q"], s["k_s"], s["z_k"], s["b_k"], s["lse"], s["lens"], s["weights"],
                             window=case["window"], decay=s["decay"], weights_out=s["weights_out"],
                             key_scale=s["key_scale"], block_table=s["table_of_pages"], ws=s["ws"])
        return {"weights": s["weights_out"]}
    lrkv.evict(s["k_s"], s["v_s"], s["z_k"], s["z_v"], s["weights"], s["lens"], case["budget"], sink=case["sink"],
               recent=case["recent"], order=s["order"], key_scale=s["key_scale"], positions=s["positions"],
               block_table=s["table_of_pages"], weights_out=s["weights_out"], order_out=s["order_out"],
               new_lens=s["new_lens"], kept=s["kept"], ws=s["ws"])
    return _evicted(s)


# ------------------------------------------------------------ definitions --

def _pairs_as_complex(x):
    return torch.view_as_complex(x.double().unflatten(-1, (-1, 2)).contiguous())


def _unit(case, s, b, n):
    """[n, dim / 2] complex rotations of sequence b's first n rows, axis by axis."""
    theta = torch.pow(torch.tensor(BASE, dtype=torch.float64), -torch.arange(0, case["dim"], 2).double() / case["dim"])
    parts, k = [], 0
    for axis, count in enumerate(s["sections"]):
        turn = s["positions"][b, :n, axis].cpu().double()[:, None] * theta[k:k + count]
        parts.append(torch.polar(torch.ones_like(turn), turn))
        k += count
    return torch.cat(parts, dim=1).cuda()


def _exact_attention(case, s, b, n):
    """(out [H, d], lse [H], weights [n]) of sequence b in fp64: every head's keys and values rebuilt."""
    H, d = case["heads"], case["dim"]
    if n == 0:
        return (torch.zeros(H, d, dtype=torch.float64, device="cuda"),
                torch.full((H,), -math.inf, dtype=torch.float64, device="cuda"),
                torch.zeros(0, dtype=torch.float64, device="cuda"))
    rows = {}
    for name in ("k_s", "v_s", "z_k", "z_v"):
        t = s[name] if s["table_of_pages"] is None else s[name][s["table_of_pages"][b].long()].flatten(0, 1)
        rows[name] = (t[b] if s["table_of_pages"] is None else t)[:n]
    unit = _unit(case, s, b, n) if case["op"] == "rope" else None
    outs, lses, weights = [], [], torch.zeros(n, dtype=torch.float64, device="cuda")
    for h in range(H):
        key = rows["k_s"].double() + rows["z_k"][:, h].double() @ s["b_k"][h].double().T
        if unit is not None:
            key = torch.view_as_real(_pairs_as_complex(key) * unit).flatten(-2)
        x = key @ s["q"][b, h].double() / math.sqrt(d)
        if s["key_scale"] is not None:
            x = x * s["key_scale"][b, h, :n].double()
        top = x.max()
        e = torch.exp(x - top)
        total = e.sum()
        value = rows["v_s"].double() + rows["z_v"][:, h].double() @ s["b_v"][h].double().T
        outs.append((e / total) @ value)
        lses.append(top + torch.log(total))
        weights += e / total
    return torch.stack(outs), torch.stack(lses), weights


def exact(case, seed):
    s = prepare(case, seed)
    op, B = case["op"], case["batch"]
    if op == "rotate":
        unit = torch.stack([_unit(case, s, b, case["new"]) for b in range(B)])
        return torch.view_as_real(_pairs_as_complex(s["x"]) * unit[:, :, None]).flatten(-2)
    lens = _lens(case)
    if op == "evict":
        return _exact_evict(case, s, lens)
    weights = s["weights_out"].double()
    if op == "prompt":
        w, new, d = case["window"], case["new"], case["dim"]
        for b, n in enumerate(lens):
            pages = s["table_of_pages"]
            k_s = (s["k_s"][b] if pages is None else s["k_s"][pages[b].long()].flatten(0, 1))[:n].double()
            z_k = (s["z_k"][b] if pages is None else s["z_k"][pages[b].long()].flatten(0, 1))[:n]
            look = torch.ones(w, n, device="cuda", dtype=torch.bool).tril(n - w)
            fresh = torch.zeros(n, dtype=torch.float64, device="cuda")
            for h in range(case["heads"]):
                key = k_s + z_k[:, h].double() @ s["b_k"][h].double().T
                x = s["q"][b, new - w:, h].double() @ key.T / math.sqrt(d)
                if s["key_scale"] is not None:
                    x = x * s["key_scale"][b, h, :n].double()
                a = torch.exp(x - s["lse"][b, h, new - w:, None].double())
                fresh += torch.where(look, a, 0.0).sum(dim=0)
            weights[b, :n] = fresh
            weights[b, :n - new] += s["decay"] * s["weights"][b, :n - new].double()
        return {"weights": weights}
    outs, lses = [], []
    for b, n in enumerate(lens):
        o, lse, fresh = _exact_attention(case, s, b, n)
        outs.append(o)
        lses.append(lse)
        if n:
            weights[b, :n] = fresh
            weights[b, :n - 1] += s["decay"] * s["weights"][b, :n - 1].double()
    got = {"out": torch.stack(outs), "lse": torch.stack(lses)}
    if op == "decode" or case["weighted"]:
        got["weights"] = weights
    return got


def _exact_evict(case, s, lens):
    """Lengths, kept rows, weights and order after the eviction, one sequence at a time on the host; the cache rows are copies."""
    budget = case["budget"]
    weights, out = s["weights"].cpu().numpy(), s["weights_out"].cpu().numpy().astype(np.float64)
    order_out = s["order_out"].cpu().numpy()
    kept = np.full((case["batch"], budget), -1, dtype=np.int32)
    new_lens = np.zeros(case["batch"], dtype=np.int32)
    for b, n in enumerate(lens):
        age = s["order"][b, :n].cpu().numpy().astype(np.int64) if s["order"] is not None else np.arange(n)
        new = min(n, budget)
        rows = np.arange(n)
        if n > budget:
            seen = int(age.max()) + 1
            free = ~((age < case["sink"]) | (age >= seen - case["recent"]))
            value = np.where(np.isnan(weights[b, :n]), -np.inf, weights[b, :n])
            best = np.lexsort((rows, -value, free))[:new]
            keep = np.zeros(n, dtype=bool)
            keep[best] = True
            rows = np.arange(new)
            rows[~keep[:new]] = np.nonzero(keep[new:])[0] + new
        kept[b, :new] = rows
        new_lens[b] = new
        out[b, :new] = weights[b, rows]
        order_out[b, :new] = age[rows]
    got = {"new_lens": torch.from_numpy(new_lens).cuda(), "kept": torch.from_numpy(kept).cuda(),
           "weights_out": torch.from_numpy(out).cuda(), "order_out": torch.from_numpy(order_out).cuda()}
    names = ("k_s", "v_s", "z_k", "z_v", "key_scale", "positions")
    return got | {n: None for n in names if s[n] is not None}
