"""The pages of a paged cache against the oracle, which goes through them one at
a time: forks, extensions with copies on write, compaction; tables, lengths,
references and every byte of the pools."""
import numpy as np
import pytest
import torch

import _cache8_util as C
from _lib_util import ensure_built
from compressed_cache_decode_gb300 import inputs, lrkv
from oracle import lrkv_oracle as O
from test_canary_gpu import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    lrkv.load()


def _state(rng, B, blocks, page, pages, share=0.5, full=False):
    """A consistent table: sequences with pages of their own, others forked from them; some pages held outside."""
    table, lens, refs = np.full((B, blocks), -1), np.zeros(B, dtype=np.int64), np.zeros(pages, dtype=np.int64)
    free = list(rng.permutation(pages))
    for b in range(B):
        if b and rng.random() < share:
            p = int(rng.integers(0, b))
            lens[b] = lens[p] if rng.random() < 0.7 else rng.integers(0, lens[p] + 1)
            table[b, :-(-lens[b] // page)] = table[p, :-(-lens[b] // page)]
        else:
            lens[b] = rng.integers(0, blocks * page + 1) if not full else blocks * page
            lens[b] = min(lens[b], len(free) * page)
            for j in range(-(-lens[b] // page)):
                table[b, j] = free.pop()
        for j in range(-(-lens[b] // page)):
            refs[table[b, j]] += 1
    for p in rng.permutation(pages)[:pages // 10]:
        refs[p] += 1
    return table, lens, refs


def _cuda(*arrays):
    return [torch.from_numpy(np.asarray(a).astype(np.int32)).cuda() for a in arrays]


def _same(got, want, what=""):
    np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(want), err_msg=what)


SHAPES = [
    # B, blocks, page, pages
    (1, 1, 16, 1), (1, 1, 16, 7), (5, 4, 16, 40), (64, 16, 64, 700), (33, 7, 128, 97), (256, 40, 256, 4000),
    (4096, 3, 16, 9000), (3, 2000, 16, 5000), (17, 300, 32, 100001),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(shape, in_place):
    B, blocks, page, pages = shape
    rng = np.random.default_rng(B + blocks)
    for parents, keeps in ((True, True), (True, False), (False, True), (False, False)):
        table, lens, refs = _state(rng, B, blocks, page, pages)
        parent = rng.integers(-1, B, B) if parents else None
        keep = rng.integers(0, blocks * page + 9, B) if keeps else None
        want = O.pages_fork_reference(table, lens, refs, page, parent, keep)
        t, l, r = _cuda(table, lens, refs)
        outs = {} if in_place else dict(table_out=torch.full_like(t, 77), lens_out=torch.full_like(l, 77),
                                        refs_out=torch.full_like(r, 77))
        got = lrkv.pages_fork(t, l, r, page, parent=None if parent is None else _cuda(parent)[0],
                              keep=None if keep is None else _cuda(keep)[0], **outs)
        assert lrkv.lrkv_read_device_status(got[3]) == lrkv.LRKV_OK
        for g, w in zip(got, want):
            _same(g, w)
        if not in_place:
            for a, b in zip((t, l, r), (table, lens, refs)):
                _same(a, b)


def _pools(pages, page, gen):
    """Pools of every kind: 16-byte rows, scales of blocks, odd words, wide rows."""
    some = lambda *s, dtype: torch.randint(0, 255, s, generator=gen, device="cuda", dtype=torch.uint8).view(dtype)
    return [some(pages, page, 2 * 48, dtype=torch.bfloat16), some(pages, page // 16, 4, dtype=torch.float32),
            some(pages, page, 5, 4, dtype=torch.int32), some(pages, page, 4 * 37, dtype=torch.float32),
            some(pages, 1, 16, dtype=torch.int32), some(pages, page, 2048 + 16, dtype=torch.uint8)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_extend(shape, in_place):
    B, blocks, page, pages = shape
    rng = np.random.default_rng(B * 3 + blocks)
    gen = torch.Generator(device="cuda").manual_seed(B)
    shortages = 0
    for grow in (1, page // 2 + 3, 3 * page, 0):
        table, lens, refs = _state(rng, B, blocks, page, max(1, pages * 2 // 3))
        refs = np.concatenate([refs, np.zeros(pages - len(refs), dtype=np.int64)])
        new = np.minimum(lens + rng.integers(0, grow + 1, B), blocks * page) - rng.integers(0, 2, B)
        new = np.maximum(new, 0)
        want = O.pages_extend_reference(table, lens, refs, page, new)
        shortages += want[4] > 0
        t, l, r, n = _cuda(table, lens, refs, new)
        pools = _pools(pages, page, gen) if pages * page < 1 << 18 else []
        kept = [p.clone() for p in pools]
        missing = torch.full((1,), 77, dtype=torch.int32, device="cuda")
        outs = {} if in_place else dict(table_out=torch.full_like(t, 77), lens_out=torch.full_like(l, 77),
                                        refs_out=torch.full_like(r, 77))
        got = lrkv.pages_extend(pools, t, l, r, page, n, missing=missing, **outs)
        assert lrkv.lrkv_read_device_status(got[3]) == (lrkv.LRKV_ERR_NO_PAGES if want[4] else lrkv.LRKV_OK)
        for g, w in zip(got[:3], want):
            _same(g, w)
        _same(missing, [want[4]])
        for p, before in zip(pools, kept):
            each = page // p.shape[1]
            for frm, to, rows in want[3]:
                before[to, :-(-rows // each)] = before[frm, :-(-rows // each)]
            assert torch.equal(p.view(torch.uint8), before.view(torch.uint8))
    if pages == 97:
        assert shortages   # (a pool that does not hold everything)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(shape, in_place):
    B, blocks, page, pages = shape
    rng = np.random.default_rng(B * 5 + blocks)
    gen = torch.Generator(device="cuda").manual_seed(B)
    for share in (0.0, 0.8):
        table, lens, refs = _state(rng, B, blocks, page, pages, share)
        want = O.pages_compact_reference(table, lens, refs, page)
        t, l, r = _cuda(table, lens, refs)
        pools = _pools(pages, page, gen) if pages * page < 1 << 18 else []
        kept = [p.clone() for p in pools]
        moved, live = torch.full_like(r, 77), torch.full((1,), 77, dtype=torch.int32, device="cuda")
        outs = {} if in_place else dict(table_out=torch.full_like(t, 77), refs_out=torch.full_like(r, 77))
        got = lrkv.pages_compact(pools, t, l, r, page, moved=moved, live=live, **outs)
        assert lrkv.lrkv_read_device_status(got[2]) == lrkv.LRKV_OK
        _same(got[0], want[0])
        _same(got[1], want[1])
        _same(moved, want[2])
        _same(live, [want[3]])
        for p, before in zip(pools, kept):
            for frm, to in want[4]:
                before[to] = before[frm]
            assert torch.equal(p.view(torch.uint8), before.view(torch.uint8))


@pytest.mark.parametrize("refs", [[0] * 5, [1] * 5, [0, 0, 0, 0, 3], [2, 0, 0, 0, 0]])
def test_compact_of_nothing_and_of_everything(refs):
    t, l, r = _cuda([[-1, -1]], [0], refs)
    want = O.pages_compact_reference([[-1, -1]], [0], refs, 16)
    got = lrkv.pages_compact([], t, l, r, 16, moved=(m := torch.zeros_like(r)))
    _same(got[0], want[0])
    _same(got[1], want[1])
    _same(m, want[2])


def test_what_does_not_fit_is_clamped_left_out_and_reported():
    page, bad = 16, lrkv.LRKV_ERR_DEVICE_BOUNDS
    # an entry in use that names no page stays, and counts nowhere
    for v in (-1, 6, 2 ** 30):
        t, l, r = _cuda([[0, v], [2, 3]], [32, 20], [1, 0, 1, 1, 0, 0])
        got = lrkv.pages_fork(t, l, r, page, parent=_cuda([0, 0])[0])
        assert lrkv.lrkv_read_device_status(got[3]) == bad
        _same(got[0], [[0, v], [0, v]])
        _same(got[2], [2, 0, 0, 0, 0, 0])
        t, l, r = _cuda([[0, v], [2, 3]], [20, 20], [1, 0, 1, 1, 0, 0])
        got = lrkv.pages_extend([], t, l, r, page, _cuda([25, 20])[0])
        assert lrkv.lrkv_read_device_status(got[3]) == bad
        _same(got[0], [[0, v], [2, 3]])
        _same(got[1], [25, 20])
        t, l, r = _cuda([[0, v], [2, 3]], [20, 20], [1, 0, 1, 1, 0, 0])
        got = lrkv.pages_compact([], t, l, r, page)
        assert lrkv.lrkv_read_device_status(got[2]) == bad
        _same(got[0], [[0, v], [2, 1]])
    # an entry that names a free page
    t, l, r = _cuda([[0, 4], [2, 3]], [20, 20], [1, 0, 1, 1, 0, 0])
    got = lrkv.pages_compact([], t, l, r, page)
    assert lrkv.lrkv_read_device_status(got[2]) == bad
    _same(got[0], [[0, 4], [2, 1]])
    # parents, lengths to keep and lengths out of range
    t, l, r = _cuda([[0, 1], [2, 3], [4, -1]], [32, 17, 9], [1, 1, 1, 1, 1])
    got = lrkv.pages_fork(t, l, r, page, parent=_cuda([3, 1, -2])[0], keep=_cuda([9, -1, 9])[0])
    assert lrkv.lrkv_read_device_status(got[3]) == bad
    _same(got[0], -np.ones((3, 2)))
    _same(got[1], [0, 0, 0])
    _same(got[2], [0] * 5)
    t, l, r = _cuda([[0, 1], [2, 3], [4, -1]], [2 ** 31 - 1, -5, 9], [1, 1, 0, 0, 1])
    got = lrkv.pages_fork(t, l, r, page)
    assert lrkv.lrkv_read_device_status(got[3]) == bad
    _same(got[1], [32, 0, 9])
    _same(got[0], [[0, 1], [-1, -1], [4, -1]])
    t, l, r = _cuda([[0, 1], [-1, -1]], [20, 0], [1, 1, 0, 0])
    got = lrkv.pages_extend([], t, l, r, page, _cuda([2 ** 31 - 1, 40])[0])
    assert lrkv.lrkv_read_device_status(got[3]) == bad
    _same(got[1], [32, 32])
    _same(got[0], [[0, 1], [2, 3]])
    # references below zero are free
    t, l, r = _cuda([[1, -1]], [16], [-3, 1, 0])
    got = lrkv.pages_extend([], t, l, r, page, _cuda([17])[0])
    assert lrkv.lrkv_read_device_status(got[3]) == lrkv.LRKV_OK
    _same(got[0], [[1, 0]])
    _same(got[2], [1, 1, 0])


def test_guards_and_one_workspace_for_calls_that_follow_each_other():
    B, blocks, page, pages = 30, 9, 32, 400
    rng = np.random.default_rng(3)
    table, lens, refs = _state(rng, B, blocks, page, pages - 60)
    refs = np.concatenate([refs, np.zeros(60, dtype=np.int64)])
    i32 = lambda *s: Guarded(s, torch.int32)
    t, l, r = _cuda(table, lens, refs)
    size = lrkv._size_of("lrkv_pages_workspace_size", B, blocks, pages)
    ws, to, lo, ro = i32(size // 4), i32(B, blocks), i32(B), i32(pages)
    pool, moved, live, missing = Guarded((pages, page, 24), torch.float32), i32(pages), i32(1), i32(1)
    pool.t.zero_()
    w = ws.t.view(torch.uint8)
    lrkv.pages_fork(t, l, r, page, parent=_cuda(np.arange(B) // 2)[0], table_out=to.t, lens_out=lo.t, refs_out=ro.t, ws=w)
    want = O.pages_fork_reference(table, lens, refs, page, np.arange(B) // 2, None)
    for g, x in zip((to, lo, ro), want):
        g.check(True)
        _same(g.t, x)
    new = np.minimum(want[1] + 5, blocks * page)
    lrkv.pages_extend([pool.t], to.t, lo.t, ro.t, page, _cuda(new)[0], missing=missing.t, ws=w)
    want = O.pages_extend_reference(*want, page, new)
    for g, x in zip((to, lo, ro), want):
        _same(g.t, x)
    _same(missing.t, [want[4]])
    lrkv.pages_compact([pool.t], to.t, lo.t, ro.t, page, moved=moved.t, live=live.t, ws=w)
    want = O.pages_compact_reference(*want[:3], page)
    _same(to.t, want[0])
    _same(ro.t, want[1])
    for g in (ws, to, lo, ro, pool, moved, live, missing):
        g.check()


def test_a_serving_run_over_an_8_bit_pool():
    """Prompts, samples of one prompt, decode steps, an end, a compaction: every step's attention against the oracle
    over each sequence's own rows.  The step is captured once and replayed."""
    B, H, dh, r, page, blocks = 4, 8, 64, 28, 32, 6
    pages = 20
    gen = torch.Generator().manual_seed(1)
    cache = lrkv.empty_cache8(pages, page, H, dh, r)
    for t in cache.pools():
        t.view(torch.uint8).fill_(0x7f)
    table = torch.full((B, blocks), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    b_k, b_v = ((torch.randn(H, dh, r, generator=gen) / 5).bfloat16() for _ in range(2))
    widths = ((1, dh), (1, dh), (H, r), (H, r))
    draw = lambda n: [torch.randn(B, n, *((H, r) if z else (dh,)), generator=gen).bfloat16() for z in (0, 0, 1, 1)]

    class Held:
        """What a sequence's pages hold: the four tensors' numbers and scales, and its length."""

        def __init__(self, other=None, n=0):
            self.t = ([[v.copy(), s.copy()] for v, s in other.t] if other else
                      [[np.zeros((blocks * page, h, w)), np.zeros((blocks * page // 16, h))] for h, w in widths])
            self.n = other.n if other else n

        def add(self, rows):
            for k, (h, w) in enumerate(widths):
                x = rows[k].double().numpy().reshape(-1, h, w)
                self.t[k] = list(O.quantize_reference(*self.t[k], x, self.n, len(x)))
            self.n += len(rows[0])

    held = [Held() for _ in range(B)]

    def check(q, out, lse):
        for b in range(B):
            if held[b].n == 0:
                assert torch.all(out[b] == 0) and torch.all(torch.isinf(lse[b]))
                continue
            ks, vs, zk, zv = (O.cache8_rows(v, s)[:held[b].n] for v, s in held[b].t)
            o, l = O.decode_reference(q[b:b + 1], ks[None, :, 0], vs[None, :, 0], zk[None], zv[None], b_k, b_v,
                                      np.array([len(ks)]))
            # as in _cache8_util: scores whose magnitudes sum to 60 at most, 176 additions; values of at most 8
            assert np.abs(lse[b].cpu().double().numpy() - l[0]).max() <= 2 * C.U * 176 * 60
            assert np.abs(out[b].cpu().double().numpy() - o[0]).max() <= 4 * C.U * (176 * 60 + 300) * 8

    rows = [x.cuda() for x in draw(1)]
    q = torch.zeros(B, H, dh, dtype=torch.bfloat16, device="cuda")
    grow = torch.ones(B, dtype=torch.int32, device="cuda")
    ws = lrkv.pages_workspace(B, blocks, pages)
    dws = lrkv.decode8_workspace(lrkv.make_dims(B, H, dh, r, blocks * page, torch.bfloat16))
    qws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(B, H, dh, device="cuda"), torch.empty(B, H, device="cuda")
    start, target = torch.zeros_like(lens), torch.zeros_like(lens)

    def step():
        start.copy_(lens)
        torch.add(lens, grow, out=target)
        lrkv.pages_extend(cache.pools(), table, lens, refs, page, target, ws=ws)
        lrkv.quantize(*rows, start, cache, new_lens=grow, block_table=table, ws=qws)
        lrkv.decode8(q, cache, bk, bv, lens, block_table=table, out=out, lse=lse, ws=dws)

    bk, bv = b_k.cuda(), b_v.cuda()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    state = (table, lens, refs)
    keep = [t.clone() for t in state]
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for t, k in zip(state, keep):
        t.copy_(k)
    # two prompts of different lengths, then samples of the first one
    prompt, n = draw(45), [45, 20, 0, 0]
    lrkv.pages_extend(cache.pools(), table, lens, refs, page, torch.tensor(n, dtype=torch.int32).cuda(), ws=ws)
    lrkv.quantize(*[x.cuda() for x in prompt], torch.zeros_like(lens), cache, new_lens=lens, block_table=table)
    for b in (0, 1):
        held[b].add([x[b, :n[b]] for x in prompt])
    lrkv.pages_fork(table, lens, refs, page, parent=torch.tensor([0, 1, 0, 0], dtype=torch.int32).cuda(), ws=ws)
    held[2], held[3] = Held(held[0]), Held(held[0])
    assert sorted(refs.cpu().tolist(), reverse=True)[:3] == [3, 3, 1]

    for k in range(24):
        new = draw(1)
        for x, y in zip(rows, new):
            x.copy_(y)
        fresh_q = torch.randn(B, H, dh, generator=gen).bfloat16()
        q.copy_(fresh_q)
        graph.replay()
        torch.cuda.synchronize()
        assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
        assert lrkv.lrkv_read_device_status(dws) == lrkv.LRKV_OK and lrkv.lrkv_read_device_status(qws) == lrkv.LRKV_OK
        for b in range(B):
            if grow[b]:
                held[b].add([x[b] for x in new])
        if k % 4 == 3 or k == 0:
            check(fresh_q, out, lse)
        if k == 9:     # a sample ends, another goes on from the first
            lrkv.pages_fork(table, lens, refs, page, parent=torch.tensor([0, 1, -1, 0], dtype=torch.int32).cuda(), ws=ws)
            held[2], held[3] = Held(), Held(held[0])
            grow[2] = 0
        if k == 14:    # a prompt is cut back to a place inside a page, and the pool compacted
            cut = torch.tensor([100, 25, 0, 100], dtype=torch.int32).cuda()
            lrkv.pages_fork(table, lens, refs, page, keep=cut, ws=ws)
            held[1].n = 25
            live = torch.zeros(1, dtype=torch.int32, device="cuda")
            lrkv.pages_compact(cache.pools(), table, lens, refs, page, live=live, ws=ws)
            n_live = int(live)
            assert (refs[:n_live] > 0).all() and (refs[n_live:] == 0).all()
            for t in cache.pools():   # nothing past the live pages is needed
                t.view(torch.uint8)[n_live:].fill_(0x7f)
    used = set()
    for b in range(B):
        used |= set(table[b, :-(-int(lens[b]) // page)].tolist())
    assert used == set(torch.nonzero(refs).flatten().tolist())


def test_a_decode_right_after_a_call_without_pools_sees_its_table():
    """lrkv_decode8 reads tables and lengths as soon as the launch before it lets it start."""
    B, H, dh, r, page, blocks = 64, 8, 64, 16, 16, 64
    pages = B * blocks
    cache = lrkv.empty_cache8(pages, page, H, dh, r)
    for t in cache.pools():
        t.view(torch.uint8).zero_()
    q = torch.ones(B, H, dh, dtype=torch.bfloat16, device="cuda")
    b = torch.ones(H, dh, r, dtype=torch.bfloat16, device="cuda")
    ws, dws = lrkv.pages_workspace(B, blocks, pages), None
    for n in (1000, 16, 513, 1, 1024):
        table = torch.full((B, blocks), -1, dtype=torch.int32, device="cuda")
        lens, refs = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
        lrkv.pages_extend([], table, lens, refs, page, torch.full_like(lens, n), ws=ws)
        out, lse, dws = lrkv.decode8(q, cache, b, b, lens, block_table=table, ws=dws)
        assert lrkv.lrkv_read_device_status(dws) == lrkv.LRKV_OK
        assert (lse.double().cpu() - np.log(n)).abs().max() <= 1e-6 and torch.all(out == 0)


def test_bf16_pages_forked_extended_and_appended():
    """The same over a bf16 pool: append_paged and decode_paged on pages that the calls handed out."""
    B, H, dh, r, page, blocks, d = 2, 16, 64, 32, 32, 4, 128
    pages = 9
    gen = torch.Generator().manual_seed(2)
    bf = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()
    pools = [torch.full((pages, page, *t), float("nan"), dtype=torch.bfloat16, device="cuda")
             for t in ((dh,), (dh,), (H, r), (H, r))]
    w = [bf(dh, d), bf(dh, d), bf(H * r, d), bf(H * r, d)]
    w = [x / d ** 0.5 for x in w]
    b_k, b_v, q = bf(H, dh, r) / 5, bf(H, dh, r) / 5, bf(B, H, dh)
    table = torch.full((B, blocks), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    plain = [torch.zeros(B, blocks * page, *p.shape[2:], dtype=torch.bfloat16, device="cuda") for p in pools]

    def grow(n, x):
        start = lens.clone()
        lrkv.pages_extend(pools, table, lens, refs, page, lens + n)
        lrkv.append_paged(x, *w, start, table, *pools, H)
        lrkv.append(x, *w, start, *plain)

    x = bf(1, 50, d)
    grow(torch.tensor([50, 0], dtype=torch.int32, device="cuda"), torch.cat([x, x]).contiguous())
    lrkv.pages_fork(table, lens, refs, page, parent=torch.zeros(B, dtype=torch.int32, device="cuda"))
    for p in plain:
        p[1] = p[0]
    for _ in range(20):
        grow(torch.ones(B, dtype=torch.int32, device="cuda"), bf(B, 1, d))
    out, lse, ws = lrkv.decode_paged(q, *pools, b_k, b_v, table, lens)
    want, want_lse = lrkv.decode(q, *plain, b_k, b_v, lens)
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    # the same rows in another split: fp32 sums of 70 rows in another order, probabilities in bf16 (2^-8 each)
    assert (out - want).abs().max() <= 2.0 ** -7 * want.abs().max() and (lse - want_lse).abs().max() <= 1e-5
    assert int(refs.sum()) == 6 and int((refs > 0).sum()) == 5 and table[0, 0] == table[1, 0]
