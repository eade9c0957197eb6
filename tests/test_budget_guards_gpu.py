"""Around the calls that keep a cache inside a token budget: guard regions on
every buffer they write, a captured graph of them replayed on other contents,
two calls at once, waits that run out, prompt windows of every tile shape and
over many items per SM, evictions of long rows and from long sequences."""
import pytest
import torch

import _budget_util as T
import test_budget_gpu as base
from _lib_util import ensure_built
from compressed_cache_decode_gb300 import inputs, lrkv
from test_canary_gpu import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    lrkv.load()


# windows of one tile of 16, 32, 64 and 128 queries and the next sizes, heads
# that fill a tile's columns and that leave some; ranks of one to four steps
WINDOWS = [
    # B, H, d_h, r, max_len, lengths, q_len, window, page, normed
    (1, 8, 128, 64, 300, [300], 20, 16, 0, False),
    (2, 8, 64, 8, 600, [600, 129], 40, 17, 0, False),
    (1, 12, 128, 24, 520, [513], 33, 33, 0, True),       # four heads of a group of twelve
    (2, 6, 128, 48, 320, [300, 257], 65, 64, 32, False),
    (1, 5, 64, 64, 400, [400], 66, 65, 0, False),        # one head to a tile
    (1, 3, 128, 64, 448, [390], 128, 128, 64, False),
    (1, 3, 128, 40, 400, [390], 140, 129, 0, False),     # two tiles
    (2, 32, 128, 0, 300, [300, 40], 20, 20, 0, False),   # one tile, no latents
    (3, 8, 64, 64, 20000, [20000, 128, 16385], 32, 32, 0, False),   # several items per SM, one and two halves
    (2, 8, 128, 64, 30016, [30011, 29313], 4, 4, 16, False),        # the same, pages of 16
]


@pytest.mark.parametrize("shape", WINDOWS)
def test_prefill_weights_of_every_tile_shape(shape):
    base.test_prefill_weights(shape)


EVICTIONS = [
    # B, H, d_h, r, max_len, lengths, budget, sink, recent, dtype, axes
    (2, 64, 128, 64, 40, [40, 33], 12, 1, 2, "f32", 2),          # rows of 33 KB, moved in two parts
    (1, 256, 64, 64, 24, [24], 10, 0, 3, "f32", 0),              # rows of 128 KB, moved in five
    (3, 1, 8, 0, 5000, [5000, 4097, 2], 4096, 4, 16, "bf16", 0),  # rows of 32 bytes, no latents
    (1, 1, 64, 8, 700000, [699999], 1000, 0, 10, "bf16", 0),     # 16 CTAs, more rows each than keys they keep
    (80, 1, 16, 8, 42000, [42000 - 523 * b for b in range(80)], 40, 1, 9, "bf16", 1),  # the same, a CTA each
]


@pytest.mark.parametrize("shape", EVICTIONS)
@pytest.mark.parametrize("ordered", [False, True])
@pytest.mark.parametrize("page", [0, 1])
def test_evict_long_rows_and_long_sequences(shape, ordered, page):
    base.test_evict(shape, ordered, page)


def _state(B=2, H=8, dh=128, r=48, Lm=400, lens=(400, 217), seed=5):
    d = T.cuda(inputs.random_decode_case(seed=seed, batch=B, heads=H, head_dim=dh, rank=r, max_len=Lm, dtype="bf16",
                                         lens=list(lens)))
    return d, [d[k] for k in T.NAMES]


def _bytes(n):
    return Guarded(((n + 1) // 2,), torch.bfloat16)


def test_guards_around_what_the_calls_write():
    B, H, dh, r, Lm, axes = 2, 8, 128, 48, 400, 3
    d, q = _state(B, H, dh, r, Lm)
    dims = lrkv.make_dims(B, H, dh, r, Lm, torch.bfloat16)
    table = lrkv.rope_table(500, dh)
    pos = T.random_positions(B, Lm, axes, 500, 3).cuda()
    size = {c: lrkv._size_of(f"lrkv_{c}_workspace_size", lrkv.ctypes.byref(dims))
            for c in ("decode_weighted", "decode_rope_axes")}

    def outputs():
        return (Guarded((B, H, dh), torch.float32), Guarded((B, H), torch.float32),
                Guarded((B, Lm), torch.float32, fill=torch.zeros(B, Lm)))

    def check(what, ws, *full, partial=()):
        for i, g in enumerate(full):
            g.check(True, f"{what} {i}")
        for i, g in enumerate(partial):
            g.check(False, f"{what} {i}")
        ws.check(False, f"{what} workspace")

    out, lse, w = outputs()
    ws = _bytes(size["decode_weighted"])
    lrkv.decode_weighted(*q, w.t, out=out.t, lse=lse.t, ws=ws.t.view(torch.uint8))
    check("decode_weighted", ws, out, lse, w)

    out, lse, w = outputs()
    ws = _bytes(size["decode_rope_axes"])
    lrkv.decode_rope_axes(*q[:7], table, pos, [16, 24, 24], q[7], weights=w.t, out=out.t, lse=lse.t,
                          ws=ws.t.view(torch.uint8))
    check("decode_rope_axes", ws, out, lse, w)

    for window in (30, 150):                                 # one tile, two tiles
        prompt = T.cuda(inputs.random_prefill_case(seed=2, batch=B, q_len=200, heads=H, head_dim=dh, rank=r,
                                                   max_len=Lm, lens=[400, 217]))
        w = Guarded((B, Lm), torch.float32, fill=torch.zeros(B, Lm))
        ws = _bytes(lrkv._size_of("lrkv_prefill_weights_workspace_size", lrkv.ctypes.byref(dims), window))
        lrkv.prefill_weights(prompt["q"], prompt["k_s"], prompt["z_k"], prompt["b_k"],
                             torch.full((B, H, 200), 6.0, device="cuda"), prompt["seq_lens"], w.t, window=window,
                             ws=ws.t.view(torch.uint8))
        check("prefill_weights", ws, w)

    x = torch.randn(B, 7, H, dh, device="cuda").bfloat16()
    turned = Guarded((B, 7, H, dh), torch.bfloat16)
    ws = Guarded((4,), torch.int32, fill=torch.zeros(4, dtype=torch.int32))
    lrkv.rope_rotate(x, pos[:, :7].contiguous(), table, [16, 24, 24], out=turned.t,
                     ws=ws.t.view(torch.uint8))
    check("rope_rotate", ws, turned)

    budget = 100
    cache = {k: Guarded(tuple(d[k].shape), torch.bfloat16, fill=d[k]) for k in ("k_s", "v_s", "z_k", "z_v")}
    guarded = dict(weights=Guarded((B, Lm), torch.float32, fill=torch.rand(B, Lm)),
                   order=Guarded((B, Lm), torch.int32, fill=torch.arange(Lm, dtype=torch.int32).repeat(B, 1)),
                   key_scale=Guarded((B, H, Lm), torch.float32, fill=torch.rand(B, H, Lm)),
                   positions=Guarded((B, Lm, axes), torch.int32, fill=pos))
    lens = Guarded((B,), torch.int32, fill=d["seq_lens"])
    kept = Guarded((B, budget), torch.int32)
    ws = _bytes(lrkv._size_of("lrkv_evict_workspace_size", B, Lm, budget))
    rest = {k: g.t[:, budget:].clone() for k, g in cache.items()}
    lrkv.evict(*[cache[k].t for k in ("k_s", "v_s", "z_k", "z_v")], guarded["weights"].t, lens.t, budget, sink=3,
               recent=9, kept=kept.t, ws=ws.t.view(torch.uint8),
               **{k: g.t for k, g in guarded.items() if k != "weights"})
    check("evict", ws, lens, kept, *guarded.values(), partial=cache.values())
    for k, g in cache.items():
        assert torch.equal(g.t[:, budget:], rest[k]), k      # rows past the new length are as they were


def test_a_captured_run_of_the_calls_on_other_contents():
    """Every call once in one graph; replayed after its buffers were given other
    contents and other lengths it gives what the calls give one by one."""
    B, H, dh, r, Lm, budget, sections = 2, 8, 128, 64, 300, 120, [20, 44]
    table = lrkv.rope_table(900, dh)
    pos = T.random_positions(B, Lm, 2, 900, 1).cuda()

    def fresh(seed, lens):
        d, _ = _state(B, H, dh, r, Lm, lens, seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        d["x"] = torch.randn(B, 40, H, dh, generator=gen, device="cuda").bfloat16()
        d["weights"] = torch.rand(B, Lm, generator=gen, device="cuda")
        d["positions"] = pos.clone()
        d["kept"] = torch.zeros((B, budget), dtype=torch.int32, device="cuda")
        d["out"], d["lse"] = torch.zeros((B, H, dh), device="cuda"), torch.zeros((B, H), device="cuda")
        d["lse_q"] = torch.full((B, H, 40), 7.0, device="cuda")
        d["turned"] = torch.zeros_like(d["x"])
        return d

    dims = lrkv.make_dims(B, H, dh, r, Lm, torch.bfloat16)
    spaces = (lrkv.prefill_weights_workspace(dims, 40), lrkv.decode_weighted_workspace(dims),
              lrkv.evict_workspace(B, Lm, budget), lrkv.decode_rope_axes_workspace(dims))

    def run(d):
        cache = [d[k] for k in ("k_s", "v_s", "z_k", "z_v", "b_k", "b_v")]
        lrkv.rope_rotate(d["x"], d["positions"][:, :40].contiguous(), table, sections, out=d["turned"])
        lrkv.prefill_weights(d["turned"], d["k_s"], d["z_k"], d["b_k"], d["lse_q"], d["seq_lens"], d["weights"],
                             ws=spaces[0])
        lrkv.decode_weighted(d["q"], *cache, d["seq_lens"], d["weights"], out=d["out"], lse=d["lse"], ws=spaces[1])
        lrkv.evict(*cache[:4], d["weights"], d["seq_lens"], budget, recent=4, positions=d["positions"],
                   kept=d["kept"], ws=spaces[2])
        lrkv.decode_rope_axes(d["q"], *cache, table, d["positions"], sections, d["seq_lens"], weights=d["weights"],
                              out=d["out"], lse=d["lse"], ws=spaces[3])

    static = fresh(1, (300, 150))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(static)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(static)
    for seed, lens in ((2, (300, 150)), (3, (77, 299)), (4, (40, 121))):
        other = fresh(seed, lens)
        for k in static:
            static[k].copy_(other[k])
        graph.replay()
        torch.cuda.synchronize()
        for ws in spaces:
            assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
        run(other)
        torch.cuda.synchronize()
        for k in static:
            assert torch.equal(static[k], other[k]), (seed, k)


def test_two_calls_at_once():
    """On two streams with a workspace each, beside one another: the bits of the
    calls one after another."""
    cases = [_state(2, 16, 128, 64, 6000, (6000, 4000), s) for s in (1, 2)]
    prompts = [T.cuda(inputs.random_prefill_case(seed=s, batch=2, q_len=64, heads=16, head_dim=128, rank=64,
                                                 max_len=6000, lens=[6000, 4000])) for s in (3, 4)]
    table = lrkv.rope_table(6000, 128)
    pos = T.random_positions(2, 6000, 2, 6000, 3).cuda()
    lse = torch.full((2, 16, 64), 8.0, device="cuda")
    dims = lrkv.make_dims(2, 16, 128, 64, 6000, torch.bfloat16)
    spaces = [(lrkv.decode_weighted_workspace(dims), lrkv.prefill_weights_workspace(dims, 64),
               lrkv.decode_rope_axes_workspace(dims), lrkv.evict_workspace(2, 6000, 1000)) for _ in cases]

    def run(i, stream):
        d, q = cases[i]
        p = prompts[i]
        lens = d["seq_lens"].clone()
        cache = [d[k].clone() for k in ("k_s", "v_s", "z_k", "z_v")]
        w = torch.zeros((2, 6000), device="cuda")
        a = lrkv.decode_weighted(*q, w, ws=spaces[i][0], stream=stream)
        lrkv.prefill_weights(p["q"], p["k_s"], p["z_k"], p["b_k"], lse, p["seq_lens"], w, ws=spaces[i][1],
                             stream=stream)
        x = lrkv.decode_rope_axes(*q[:7], table, pos, [32, 32], q[7], weights=w, ws=spaces[i][2], stream=stream)
        lrkv.evict(*cache, w, lens, 1000, recent=10, ws=spaces[i][3], stream=stream)
        return [a[0], a[1], x[0], x[1], w, lens, *cache]

    alone = []
    for i in range(2):
        alone.append(run(i, None))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        both = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                both.append(run(i, s))
        torch.cuda.synchronize()
        for got, want in zip(both, alone):
            for g, t in zip(got, want):
                assert torch.equal(g, t)


@pytest.mark.parametrize("call", ["decode_weighted", "decode_rope_axes"])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_recovers(call, monkeypatch):
    """The bound of the waits cut to one cycle (caches larger than L2, so that
    copies are in flight): reported in the status word, and the next call on the
    same workspace is whole."""
    B, H, dh, r, Lm = 2, 32, 128, 48, 32768
    d, q = _state(B, H, dh, r, Lm, (32768, 20000))
    dims = lrkv.make_dims(B, H, dh, r, Lm, torch.bfloat16)
    ws = getattr(lrkv, call + "_workspace")(dims)
    table = lrkv.rope_table(Lm, dh)
    pos = torch.arange(Lm, dtype=torch.int32, device="cuda").expand(B, Lm)[..., None].contiguous()

    def run():
        w = torch.zeros((B, Lm), device="cuda")
        got = (lrkv.decode_weighted(*q, w, ws=ws) if call == "decode_weighted" else
               lrkv.decode_rope_axes(*q[:7], table, pos, [64], q[7], weights=w, ws=ws))
        torch.cuda.synchronize()
        return got

    want = run()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    torch.empty(512 << 20, dtype=torch.uint8, device="cuda").fill_(1)
    monkeypatch.setenv("LRKV_WAIT_LIMIT_CYCLES", "1")
    run()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_ERR_TIMEOUT
    monkeypatch.delenv("LRKV_WAIT_LIMIT_CYCLES")
    got = run()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    for g, t in zip(got[:3], want[:3]):
        assert torch.equal(g, t)
