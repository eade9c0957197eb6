"""The factored cache in 8 bits against the 64-bit oracle: lrkv_quantize bit for
bit, lrkv_decode8 within bounds derived in _cache8_util, over head layouts,
ranks, lengths, pages, scales and what lies past the sequences."""
import numpy as np
import pytest
import torch

import _budget_util as T
import _cache8_util as C
from _lib_util import ensure_built
from compressed_cache_decode_gb300 import lrkv
from oracle import lrkv_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    lrkv.load()


DECODES = [
    # B, H, d_h, r, max_len, lengths, page
    (1, 8, 128, 48, 128, [128], 0),                       # one full tile
    (1, 16, 16, 2, 1, [1], 0),                        # one row
    (1, 3, 64, 0, 200, [130], 0),                         # no latents, heads that do not fill a group
    (3, 8, 64, 2, 40, [1, 15, 33], 0),
    (2, 5, 80, 16, 200, [200, 129], 0),                   # a width that ends inside a step
    (2, 9, 128, 48, 300, [300, 0], 0),                    # a group of one head; an empty sequence
    (1, 16, 64, 28, 576, [517], 0),
    (4, 32, 128, 56, 512, [512, 1, 0, 385], 256),
    (3, 32, 128, 48, 1040, [1040, 31, 640], 16),          # pages of a block, a capacity that no tile divides
    (2, 12, 256, 64, 200, [200, 77], 0),                  # shared rows of two boxes, latents of four
    (2, 24, 128, 64, 384, [384, 250], 64),
    (2, 8, 32, 62, 160, [127, 160], 32),
    (1, 256, 16, 2, 64, [50], 0),                         # 32 groups
    (70, 8, 64, 32, 160, [(7 * b) % 161 for b in range(70)], 0),   # pieces of many sequences in a CTA
    (2, 16, 128, 20, 20000, [19999, 12001], 0),
    (5, 4, 48, 4, 640, [640, 639, 513, 128, 17], 128),
]


@pytest.mark.parametrize("shape", DECODES)
def test_decode8(shape):
    B, H, dh, r, L, lens, page = shape
    case = C.Case(B, H, dh, r, L, lens, seed=L + r)
    q, cache, b_k, b_v, n, table = case.cuda(page, seed=B)
    out, lse, ws = lrkv.decode8(q, cache, b_k, b_v, n, block_table=table)
    torch.cuda.synchronize()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    case.check(out, lse)


@pytest.mark.parametrize("sms", [1, 2, 7, 400])
def test_decode8_of_any_split(sms, monkeypatch):
    """One CTA for everything (1,300 sequences: more than a CTA joins at a time), few, and more than there are SMs."""
    B = 1300 if sms == 1 else 40
    lens = [(11 * b) % 34 if sms == 1 else (97 * b) % 700 for b in range(B)]
    case = C.Case(B, 8, 16, 2, max(lens), lens, seed=sms)
    q, cache, b_k, b_v, n, table = case.cuda()
    monkeypatch.setenv("LRKV_SM_COUNT", str(sms))
    out, lse, ws = lrkv.decode8(q, cache, b_k, b_v, n)
    torch.cuda.synchronize()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    case.check(out, lse, pairs={(b, b % 8) for b in range(B)})


@pytest.mark.parametrize("sms, shape, offset", [
    (2, (9, 12, 256, 64, 330, [(150 * b) % 331 for b in range(9)]), 0),   # a CTA joins many sequences, heads in slices
    (2, (9, 12, 256, 64, 330, [(150 * b) % 331 for b in range(9)]), 2),   # bases read 4 bytes at a time
    (6, (7, 16, 64, 28, 700, [(333 * b) % 701 for b in range(7)]), 4),    # 8 bytes at a time; some joined, some shared
    (400, (2, 8, 64, 32, 9000, [9000, 700]), 0),                          # more pieces than a warp has lanes
    (152, (4096, 8, 16, 2, 16, [b % 17 for b in range(4096)]), 0),        # the largest batch
])
def test_decode8_joins(sms, shape, offset, monkeypatch):
    B, H, dh, r, L, lens = shape
    case = C.Case(B, H, dh, r, L, lens, seed=sms)
    q, cache, b_k, b_v, n, _ = case.cuda()
    flat = torch.empty(offset + b_v.numel(), dtype=torch.bfloat16, device="cuda")
    flat[offset:] = b_v.view(-1)
    monkeypatch.setenv("LRKV_SM_COUNT", str(sms))
    out, lse, ws = lrkv.decode8(q, cache, b_k, flat[offset:].view(b_v.shape), n)
    torch.cuda.synchronize()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    case.check(out, lse, pairs={(b, b % H) for b in range(0, B, max(1, B // 200))})


def test_decode8_over_a_long_cache():
    """More than 2^32 bytes of latents: offsets past 32 bits (the shared rows and most latents are zero)."""
    B, H, dh, r, L = 2, 32, 64, 64, 1 << 20
    lens = [L, 9]
    cache = lrkv.empty_cache8(B, L, H, dh, r)
    for t in cache.pools():
        t.view(torch.uint8).zero_()
    gen = torch.Generator().manual_seed(1)
    q = torch.randn(B, H, dh, generator=gen).bfloat16().cuda()
    b_k, b_v = (torch.randn(H, dh, r, generator=gen).bfloat16().cuda() for _ in range(2))
    # rows far in are the only ones whose scores are not zero
    at = [L - 3, L - 200, 17]
    values = torch.randint(0, 0x60, (len(at), H, r), generator=gen, dtype=torch.uint8).cuda()
    for k, j in enumerate(at):
        cache.z_k.view(torch.uint8)[0, j] = values[k]
        cache.z_v.view(torch.uint8)[0, j] = values[k]
        cache.z_k_scale[0, j // 16] = 2.0 ** -6
        cache.z_v_scale[0, j // 16] = 2.0 ** -6
    out, lse, ws = lrkv.decode8(q, cache, b_k, b_v, torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    z = values.view(torch.float8_e4m3fn).double().cpu().numpy() * 2.0 ** -6
    for h in (0, 13, 31):
        qh, Bk, Bv = T.f64(q[0, h]), T.f64(b_k)[h], T.f64(b_v)[h]
        s = (z[:, h] @ Bk.T) @ qh / 8
        mag = np.abs(z[:, h]) @ (np.abs(qh) @ np.abs(Bk)) / 8
        # the scores of the zero rows are exact; the three others are off by err
        err = (2 * C.U * (dh + 3 * r + 24) + 2.0 ** -23) * mag
        total = np.exp(s).sum() + L - len(at)
        want = np.log(total)
        rel = np.expm1(err.max() + 4 * C.U * (np.abs(s).max() + 4))
        # the denominator: a tile's 128 in pairs of threads' sums, 8,192 tiles a thread adds one after another
        assert abs(T.f64(lse)[0, h] - want) <= rel + (want + 4 + L / 128 + 160) * 2 * C.U
        V = z[:, h] @ Bv.T
        o = (np.exp(s)[:, None] * V).sum(0) / total
        bound = (np.exp(s) @ np.abs(V)) / total * (2 * rel + (L / 128 + 400) * 2 * C.U) + 2.0 ** -37 * 448 * 2.0 ** -6 * 3 * r
        assert np.all(np.abs(T.f64(out)[0, h] - o) <= bound)
    assert np.all(T.f64(out)[1] == 0)
    np.testing.assert_allclose(T.f64(lse)[1], np.log(9), rtol=1e-6)


def _wide(s, n):
    rng = np.random.default_rng(5 + ord(n[0]))
    return (s * np.exp2(rng.integers(-12, 5, s.shape))).astype(np.float32).astype(float)


def _odd(s, n):
    rng = np.random.default_rng(7 + ord(n[0]))
    return (s * rng.uniform(0.3, 3.0, s.shape)).astype(np.float32).astype(float)


def _tiny(s, n):
    return np.maximum(s * 2.0 ** -100, 2.0 ** -126)


@pytest.mark.parametrize("scales", [_wide, _odd, _tiny])
def test_decode8_scales(scales):
    """Scales that differ between the blocks of a tile, that are no powers of two, that are next to nothing."""
    case = C.Case(2, 16, 128, 48, 400, [400, 129], seed=3, scales=scales)
    q, cache, b_k, b_v, n, _ = case.cuda()
    out, lse, _ = lrkv.decode8(q, cache, b_k, b_v, n)
    case.check(out, lse)


@pytest.mark.parametrize("q_scale", [0.0, 2.0 ** -90, 1e-3, 30.0])
@pytest.mark.parametrize("scale", [0.0, 0.02])
def test_decode8_query_sizes(q_scale, scale):
    case = C.Case(2, 8, 64, 32, 300, [300, 129], seed=4, q_scale=q_scale)
    q, cache, b_k, b_v, n, _ = case.cuda()
    out, lse, _ = lrkv.decode8(q, cache, b_k, b_v, n, scale=scale)
    case.check(out, lse, scale=scale or None)


def test_decode8_of_a_query_that_is_not_finite_spoils_its_head_alone():
    case = C.Case(2, 16, 64, 32, 300, [300, 129], seed=6)
    q, cache, b_k, b_v, n, _ = case.cuda()
    want, want_lse, _ = lrkv.decode8(q, cache, b_k, b_v, n)
    q[0, 3, 5], q[1, 9, 0] = float("nan"), float("inf")
    out, lse, _ = lrkv.decode8(q, cache, b_k, b_v, n)
    bad = torch.zeros(2, 16, dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[1, 9] = True
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])


def test_decode8_bounds():
    """Lengths past the capacity are clamped, entries that name no page read as zero rows; both are reported."""
    case = C.Case(3, 8, 64, 32, 256, [256, 130, 0], seed=8)
    q, cache, b_k, b_v, n, _ = case.cuda()
    out, lse, ws = lrkv.decode8(q, cache, b_k, b_v, torch.tensor([300, 130, -5], dtype=torch.int32).cuda())
    case.check(out, lse)
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_ERR_DEVICE_BOUNDS
    out, lse, ws = lrkv.decode8(q, cache, b_k, b_v, n, ws=ws)
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    for page in (16, 64, 128):
        q, cache, b_k, b_v, n, table = case.cuda(page)
        keep = np.ones((3, 256), dtype=bool)
        for b, j, v in ((0, 1, -1), (1, 0, cache.k_s.shape[0])):
            table[b, j] = v
            keep[b, j * page:(j + 1) * page] = False
        out, lse, ws = lrkv.decode8(q, cache, b_k, b_v, n, block_table=table)
        case.check(out, lse, keep=keep)
        assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("offset", [0, 2, 4, 6, 8])
def test_decode8_bases_at_any_address_that_is_allowed(offset):
    """Elements into a larger buffer: the wide reads of the bases start where they can."""
    for r in (28, 32, 26):
        case = C.Case(1, 8, 64, r, 200, [177], seed=9)
        q, cache, b_k, b_v, n, _ = case.cuda()

        def moved(t):
            buf = torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
            buf[offset:offset + t.numel()] = t.flatten()
            return buf[offset:offset + t.numel()].view(t.shape)

        out, lse, _ = lrkv.decode8(q, cache, moved(b_k), moved(b_v), n)
        case.check(out, lse)


QUANTIZES = [
    # B, H, d_h, r, max_len, page, n_new, start, new_lens, dtype
    (2, 8, 64, 28, 64, 0, 40, [0, 5], None, "bf16"),
    (3, 16, 128, 48, 128, 32, 33, [1, 90, 16], [33, 33, 1], "bf16"),
    (3, 16, 128, 56, 96, 16, 1, [0, 15, 95], None, "bf16"),         # the token of a decode step
    (2, 5, 80, 16, 37, 0, 37, [0, 0], [37, 0], "f32"),              # a sequence that brings nothing
    (2, 8, 256, 62, 50, 0, 20, [3, 30], None, "f32"),
    (1, 256, 16, 64, 48, 0, 20, [7], None, "bf16"),                 # several slabs of heads
    (2, 8, 64, 2, 40, 0, 25, [9, 14], None, "bf16"),
    (2, 3, 48, 0, 64, 64, 50, [2, 0], [9, 50], "bf16"),
    (1, 8, 16, 30, 33, 0, 33, [0], None, "bf16"),
]


def _empty(lead, H, dh, r):
    """A cache that holds a pattern everywhere."""
    cache = lrkv.empty_cache8(*lead, H, dh, r)
    gen = torch.Generator().manual_seed(3)
    for n in lrkv.Cache8.NAMES:
        t = getattr(cache, n)
        if t is None:
            continue
        if n.endswith("scale"):
            t.copy_(torch.exp2(torch.randint(-12, -4, t.shape, generator=gen).float()))
        else:
            t.view(torch.uint8).copy_(torch.randint(0, 0x7f, t.shape, generator=gen, dtype=torch.uint8))
    return cache


@pytest.mark.parametrize("shape", QUANTIZES)
def test_quantize(shape):
    B, H, dh, r, L, page, n_new, start, new, dtype = shape
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator().manual_seed(L)
    rows = {}
    for n in ("k_s", "v_s", "z_k", "z_v"):
        x = torch.randn(B, n_new, *((H, r) if n[0] == "z" else (1, dh)), generator=gen)
        x *= torch.exp2(torch.randint(-20, 20, (B, n_new, x.shape[2], 1), generator=gen).float())
        x[0, 0, 0, :1], x[-1, -1, -1, -1:] = float("inf"), float("nan")
        rows[n] = x.to(dt)
    table, lead = None, (B, L)
    if page:
        pages = B * (L // page) + 2
        table = torch.randperm(pages, generator=gen)[:B * (L // page)].view(B, -1).int()
        lead = (pages, page)
    cache = _empty(lead, H, dh, r)
    before = {n: None if getattr(cache, n) is None else getattr(cache, n).clone() for n in C.NAMES}
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    arg = {n: (x[:, :, 0] if n[1] == "_" and n[2] == "s" else x).contiguous().cuda() for n, x in rows.items()}
    lrkv.quantize(arg["k_s"], arg["v_s"], arg["z_k"] if r else None, arg["z_v"] if r else None,
                  torch.tensor(start, dtype=torch.int32).cuda(), cache,
                  new_lens=None if new is None else torch.tensor(new, dtype=torch.int32).cuda(),
                  block_table=None if table is None else table.cuda(), ws=ws)
    torch.cuda.synchronize()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    for n in ("k_s", "v_s") + (("z_k", "z_v") if r else ()):
        heads, width = rows[n].shape[2:]
        v0 = before[n].double().cpu().numpy().reshape(lead + (heads, width))
        s0 = before[n + "_scale"].double().cpu().numpy().reshape(lead[0], -1, heads)
        want_v, want_s = v0.copy(), s0.copy()
        for b in range(B):
            # the sequence's logical rows, and back
            at = ([(b, i) for i in range(L)] if table is None
                  else [(int(table[b, i // page]), i % page) for i in range(L)])
            lo = [x for x, _ in at], [y for _, y in at]
            blk = lo[0][::16], [y // 16 for y in lo[1][::16]]
            v, s = O.quantize_reference(v0[lo], s0[blk], T.f64(rows[n][b]), start[b],
                                        n_new if new is None else new[b])
            want_v[lo], want_s[blk] = v, s
        np.testing.assert_array_equal(getattr(cache, n).double().cpu().numpy().reshape(want_v.shape), want_v, err_msg=n)
        np.testing.assert_array_equal(getattr(cache, n + "_scale").double().cpu().numpy().reshape(want_s.shape), want_s,
                                      err_msg=n)


def test_quantize_token_by_token():
    """Forty tokens one at a time, some of them outliers: scales grow inside begun blocks."""
    B, H, dh, r, L = 2, 8, 64, 28, 64
    gen = torch.Generator().manual_seed(2)
    rows = {n: torch.randn(B, 40, *((H, r) if n[0] == "z" else (1, dh)), generator=gen) for n in ("k_s", "v_s", "z_k", "z_v")}
    for x in rows.values():
        x *= torch.where(torch.rand(B, 40, x.shape[2], 1, generator=gen) < 0.2, 16.0, 1.0)
    rows = {n: x.bfloat16() for n, x in rows.items()}
    cache = _empty((B, L), H, dh, r)
    ref = {n: [[getattr(cache, n)[b].double().cpu().numpy().reshape(L, *rows[n].shape[2:]),
                getattr(cache, n + "_scale")[b].double().cpu().numpy().reshape(4, -1)] for b in range(B)] for n in rows}
    start = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    for t in range(40):
        one = {n: (x[:, t:t + 1, 0] if n[2] == "s" else x[:, t:t + 1]).contiguous().cuda() for n, x in rows.items()}
        lrkv.quantize(*[one[n] for n in rows], start + t, cache)
        for n in rows:
            for b in range(B):
                ref[n][b] = list(O.quantize_reference(*ref[n][b], T.f64(rows[n][b, t:t + 1]), (0, 9)[b] + t, 1))
    for n in rows:
        for b in range(B):
            np.testing.assert_array_equal(getattr(cache, n)[b].double().cpu().numpy().reshape(ref[n][b][0].shape), ref[n][b][0])
            np.testing.assert_array_equal(getattr(cache, n + "_scale")[b].double().cpu().numpy().reshape(4, -1), ref[n][b][1])


def test_quantize_skips_and_reports_rows_that_have_no_place():
    B, H, dh, r, L, page = 5, 8, 64, 32, 96, 32
    gen = torch.Generator().manual_seed(4)
    rows = [torch.randn(B, 40, *((H, r) if z else (dh,)), generator=gen).bfloat16().cuda() for z in (0, 0, 1, 1)]
    start = torch.tensor([-7, 80, 10, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).cuda()
    new = torch.tensor([40, 40, 40, 40, 40], dtype=torch.int32).cuda()
    table = torch.arange(B * 3, dtype=torch.int32).view(B, 3)
    table[2, 1] = 99
    for paged in (False, True):
        lead = (B * 3, page) if paged else (B, L)
        cache, plain = _empty(lead, H, dh, r), _empty(lead, H, dh, r)
        ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
        lrkv.quantize(*rows, start, cache, new_lens=new, block_table=table.cuda() if paged else None, ws=ws)
        assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_ERR_DEVICE_BOUNDS
        for n, x in zip(("k_s", "v_s", "z_k", "z_v"), rows):
            heads, width = (H, r) if n[0] == "z" else (1, dh)
            v0 = getattr(plain, n).double().cpu().numpy().reshape(B, L, heads, width)
            s0 = getattr(plain, n + "_scale").double().cpu().numpy().reshape(B, L // 16, heads)
            want = [v0.copy(), s0.copy()]
            x = T.f64(x).reshape(B, 40, heads, width)
            want[0][0], want[1][0] = O.quantize_reference(v0[0], s0[0], x[0, 7:], 0, 33)
            want[0][1], want[1][1] = O.quantize_reference(v0[1], s0[1], x[1], 80, 16)
            want[0][2], want[1][2] = O.quantize_reference(v0[2], s0[2], x[2], 10, 40)
            if paged:   # rows 32 .. 49 have no page
                want[0][2, 32:64], want[1][2, 2:4] = v0[2, 32:64], s0[2, 2:4]
            np.testing.assert_array_equal(getattr(cache, n).double().cpu().numpy().reshape(want[0].shape), want[0])
            np.testing.assert_array_equal(getattr(cache, n + "_scale").double().cpu().numpy().reshape(want[1].shape), want[1])
    # new_lens outside [0, n]
    cache, plain = _empty((B, L), H, dh, r), _empty((B, L), H, dh, r)
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    lrkv.quantize(*rows, zero, cache, new_lens=torch.tensor([-1, 41, 0, 3, 40], dtype=torch.int32).cuda(), ws=ws)
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_ERR_DEVICE_BOUNDS
    v0, s0 = (getattr(plain, n).double().cpu().numpy().reshape(B, -1, 1, w) for n, w in (("v_s", dh), ("v_s_scale", 1)))
    for b, k in enumerate([0, 40, 0, 3, 40]):
        v, s = O.quantize_reference(v0[b], s0[b, :, :, 0], T.f64(rows[1])[b][:, None], 0, k)
        np.testing.assert_array_equal(cache.v_s[b].double().cpu().numpy(), v[:, 0])
        np.testing.assert_array_equal(cache.v_s_scale[b].double().cpu().numpy(), s[:, 0])
