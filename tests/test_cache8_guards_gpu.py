"""Around the 8-bit cache's calls: guard regions on what they write, other
streams, captured graphs replayed on other contents, two calls at once, waits
that run out."""
import numpy as np
import pytest
import torch

import _cache8_util as C
from _lib_util import ensure_built
from compressed_cache_decode_gb300 import lrkv
from test_budget_timeouts_gpu import _give_up_and_recover
from test_canary_gpu import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    lrkv.load()


def _case(seed=1, lens=(400, 217)):
    return C.Case(2, 16, 128, 48, 400, lens, seed=seed)


def test_guards():
    case = _case()
    q, cache, b_k, b_v, n, _ = case.cuda()
    dims = lrkv.make_dims(2, 16, 128, 48, 400, torch.bfloat16)
    size = lrkv._size_of("lrkv_decode8_workspace_size", lrkv.ctypes.byref(dims))
    out, lse = Guarded((2, 16, 128), torch.float32), Guarded((2, 16), torch.float32)
    ws = Guarded((size // 4,), torch.float32)
    lrkv.decode8(q, cache, b_k, b_v, n, out=out.t, lse=lse.t, ws=ws.t.view(-1).view(torch.uint8))
    out.check(True, "out")
    lse.check(True, "lse")
    ws.check(False, "ws")
    case.check(out.t, lse.t)
    # the cache inside guards, filled by quantize to its last row
    rows = [torch.randn(2, 400, *((16, 48) if z else (128,)), device="cuda").bfloat16() for z in (0, 0, 1, 1)]
    guarded = {}
    for name in C.NAMES:
        t = getattr(cache, name)
        scale = name.endswith("scale")
        guarded[name] = Guarded(t.shape if scale else (t.numel() // 2,), torch.float32 if scale else torch.bfloat16)
    held = {k: g.t if k.endswith("scale") else g.t.view(torch.float8_e4m3fn).view(getattr(cache, k).shape)
            for k, g in guarded.items()}
    lrkv.quantize(*rows, torch.zeros(2, dtype=torch.int32, device="cuda"), lrkv.Cache8(**held))
    for name, g in guarded.items():
        g.check(name.endswith("scale"), name)


def test_other_streams_and_two_calls_at_once():
    """Each call on a stream of its own, with inputs written there just before and a workspace of its own."""
    cases = [_case(s, l) for s, l in ((1, (400, 217)), (2, (399, 0)))]
    state = [c.cuda() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(3):
        got = []
        for (q, cache, b_k, b_v, n, _), st in zip(state, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                torch.cuda._sleep(2000000)
                late = torch.empty_like(q)
                late.copy_(q)
            got.append(lrkv.decode8(late, cache, b_k, b_v, n, stream=st))
    torch.cuda.synchronize()
    for case, (out, lse, ws) in zip(cases, got):
        assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
        case.check(out, lse)


def test_a_captured_step_replayed_on_other_contents():
    """quantize and decode8 of a step in one graph; a second graph on the same workspace; replays by turns."""
    B, H, dh, r, L = 2, 16, 128, 48, 400
    case = _case(3, (300, 170))
    q, cache, b_k, b_v, n, _ = case.cuda(garbage=False)
    gen = torch.Generator().manual_seed(5)
    rows = [torch.zeros(B, 1, *((H, r) if z else (dh,)), dtype=torch.bfloat16, device="cuda") for z in (0, 0, 1, 1)]
    ws = lrkv.decode8_workspace(lrkv.make_dims(B, H, dh, r, L, torch.bfloat16))
    out, lse = torch.empty(B, H, dh, device="cuda"), torch.empty(B, H, device="cuda")
    other = torch.empty_like(out), torch.empty_like(lse)
    start = n.clone()

    def step(o):
        lrkv.quantize(*rows, start, cache)
        start.add_(1)
        lrkv.decode8(q, cache, b_k, b_v, start, out=o[0], lse=o[1], ws=ws)

    eager = [t.clone() for t in cache.pools()]
    graphs = []
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step((out, lse))
        for o in ((out, lse), other):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                step(o)
            graphs.append(g)
    torch.cuda.synchronize()
    for t, e in zip(cache.pools(), eager):
        t.view(torch.uint8).copy_(e.view(torch.uint8))
    start.copy_(n)
    new = [[torch.randn(x.shape, generator=gen).bfloat16() for x in rows] for _ in range(6)]
    results = []
    for k, step_rows in enumerate(new):
        for x, y in zip(rows, step_rows):
            x.copy_(y)
        graphs[k % 2].replay()
        torch.cuda.synchronize()
        results.append([t.clone() for t in ((out, lse), other)[k % 2]])
    # the same steps, call by call
    for t, e in zip(cache.pools(), eager):
        t.view(torch.uint8).copy_(e.view(torch.uint8))
    start.copy_(n)
    for step_rows, want in zip(new, results):
        for x, y in zip(rows, step_rows):
            x.copy_(y)
        step((out, lse))
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("captured", [False, True])
def test_calls_that_write_what_a_decode_still_reads(captured):
    """A decode, then rows quantized over its cache, its lengths cut to nothing, its pages moved: none of them waits
    on the host, each waits for the decode."""
    B, H, dh, r, L, page = 4, 16, 128, 48, 8192, 256
    lens = (8192, 8000, 5000, 8192)
    case = C.Case(B, H, dh, r, L, lens, seed=11)
    q, cache, b_k, b_v, n, table = case.cuda(page, seed=3, garbage=False)
    pages = cache.k_s.shape[0]
    refs = torch.zeros(pages, dtype=torch.int32)
    for b, k in enumerate(lens):
        refs[table[b, :-(-k // page)].cpu().long()] += 1
    refs = refs.cuda()
    dims = lrkv.make_dims(B, H, dh, r, L, torch.bfloat16)
    ws, pws = lrkv.decode8_workspace(dims), lrkv.pages_workspace(B, L // page, pages)
    rows = [torch.zeros(B, 64, *((H, r) if z else (dh,)), dtype=torch.bfloat16, device="cuda") for z in (0, 0, 1, 1)]
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    outs = [torch.empty(B, H, dh, device="cuda") for _ in range(4)]
    first, other = (torch.empty(B, H, device="cuda") for _ in range(2))

    def decode(o):
        lrkv.decode8(q, cache, b_k, b_v, n, block_table=table, out=o, lse=first if o is outs[0] else other, ws=ws)

    def run():
        decode(outs[0])
        lrkv.pages_compact(cache.pools(), table, n, refs, page, ws=pws)
        decode(outs[1])
        lrkv.quantize(*rows, zero, cache, block_table=table)   # the first rows to zeros
        decode(outs[2])
        lrkv.pages_fork(table, n, refs, page, keep=zero, ws=pws)
        decode(outs[3])

    state = [*cache.pools(), table, n, refs]
    saved = [t.clone() for t in state]

    def restore():
        for t, x in zip(state, saved):
            t.view(torch.uint8).copy_(x.view(torch.uint8))

    run()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    case.check(want[0], first, pairs={(b, 3 * b) for b in range(B)})
    assert torch.equal(want[0], want[1]) and not torch.equal(want[1], want[2]) and not want[3].any()
    restore()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        run = g.replay
    for _ in range(5):
        restore()
        for o in outs:
            o.fill_(7)
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("heads, head_dim, rank, page", [(32, 128, 48, 0), (16, 64, 28, 0), (8, 256, 64, 64)])
def test_waits_that_run_out(heads, head_dim, rank, page, monkeypatch):
    B, L = 2, 32768
    gen = torch.Generator().manual_seed(1)
    lead = (B * L // page, page) if page else (B, L)
    cache = lrkv.empty_cache8(*lead, heads, head_dim, rank)
    for t in cache.pools():
        if t.dtype == torch.float32:
            t.fill_(2.0 ** -8)
        else:
            t.view(torch.uint8).random_(0, 0x70)
    table = torch.randperm(lead[0], generator=gen).view(B, -1).int().cuda() if page else None
    q = torch.randn(B, heads, head_dim, generator=gen).bfloat16().cuda()
    b_k, b_v = (torch.randn(heads, head_dim, rank, generator=gen).bfloat16().cuda() for _ in range(2))
    lens = torch.tensor([L, 20001], dtype=torch.int32).cuda()
    ws = lrkv.decode8_workspace(lrkv.make_dims(B, heads, head_dim, rank, L, torch.bfloat16))

    def run():
        return lrkv.decode8(q, cache, b_k, b_v, lens, block_table=table, ws=ws)[:2]

    _give_up_and_recover(run, ws, monkeypatch)


def test_the_same_every_time():
    case = C.Case(6, 32, 128, 56, 4096, [4096, 1000, 3333, 17, 0, 2049], seed=2)
    q, cache, b_k, b_v, n, _ = case.cuda()
    want = lrkv.decode8(q, cache, b_k, b_v, n)[:2]
    for _ in range(20):
        got = lrkv.decode8(q, cache, b_k, b_v, n)[:2]
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_accuracy_is_that_of_fp32():
    """N(0, 1) rows: the outputs' error, 2-norm over 2-norm.  A score is a sum of 176 products of which each
    addition is off by about 2^-25 of a partial sum of a few units: 2^-25 sqrt(176) 4 ~ 2^-19.3 at most of a
    probability, half of it on average, and an output averages hundreds of rows' independent errors."""
    case = C.Case(2, 8, 128, 48, 3000, [3000, 1500], seed=7)
    q, cache, b_k, b_v, n, _ = case.cuda()
    out, _, _ = lrkv.decode8(q, cache, b_k, b_v, n)
    want = np.array([[case.reference(b, h)[0] for h in range(8)] for b in range(2)])
    got = out.double().cpu().numpy()
    assert np.linalg.norm(got - want) <= 2.0 ** -20 * np.linalg.norm(want)
