"""The calls that keep a cache inside a token budget, on the GPU, against the
64-bit oracle: weights of a decode step and of a prompt's queries, eviction,
rotation with several axes, the decode whose rows carry positions, and a run
of them together."""
import math

import numpy as np
import pytest
import torch

import _budget_util as T
from _lib_util import ensure_built
from compressed_cache_decode_gb300 import inputs, lrkv
from oracle import lrkv_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    lrkv.load()


def _sync(ws=None, want=lrkv.LRKV_OK):
    torch.cuda.synchronize()
    if ws is not None:
        assert lrkv.lrkv_read_device_status(ws) == want


def _check_decode(case, got, prior, decay, key_scale=None, positions=None, sections=None, out_buffer=None):
    """out, lse and weights of a weighted decode against the oracle; rows past
    the lengths as `out_buffer` had them."""
    out, lse, weights = (t.detach().cpu().double().numpy() for t in got)
    B, H, dh = case["q"].shape
    scale = 1 / math.sqrt(dh)
    ref_o, ref_l, fresh = O.decode_weights_reference(*[case[k] for k in T.NAMES], key_scale=key_scale,
                                                     positions=positions, sections=sections)
    for b in range(B):
        L = int(case["seq_lens"][b])
        bound = np.zeros(L)
        for h in range(H):
            if L == 0:
                assert np.all(out[b, h] == 0) and lse[b, h] == -np.inf
                continue
            eo, el, ew = T.decode_bounds(case, b, h, scale, key_scale, positions, sections)
            assert np.all(np.abs(out[b, h] - ref_o[b, h]) <= eo), (b, h)
            assert abs(lse[b, h] - ref_l[b, h]) <= el, (b, h)
            bound += ew
        if L:
            want = O.accumulate_weights(fresh[b], prior[b], decay, L, 1)
            bound += (H + 2) * T.U * np.abs(want) + 1e-37
            assert np.all(np.abs(weights[b, :L] - want) <= bound), b
        assert np.array_equal(weights[b, L:], out_buffer[b, L:].double().numpy(), equal_nan=True)


DECODES = [
    # B, H, d_h, r, max_len, lengths
    (1, 16, 64, 28, 64, [1]),                       # one token
    (3, 16, 64, 28, 320, [300, 0, 77]),             # an empty sequence
    (2, 32, 128, 48, 512, [511, 129]),              # two row tiles
    (5, 18, 64, 8, 97, [1, 2, 3, 97, 65]),          # a partial row tile, odd capacity
    (2, 16, 128, 64, 200, [200, 17]),
    (2, 16, 128, 0, 130, [130, 5]),                 # no latents
    (1, 32, 128, 56, 5000, [4999]),                 # split over many CTAs
    (2, 16, 64, 20, 150, [150, 33]),                # a rank without its own instantiation
    (40, 16, 64, 32, 48, [(7 * b) % 48 for b in range(40)]),
]


@pytest.mark.parametrize("shape", DECODES)
@pytest.mark.parametrize("decay", [1.0, 0.75])
def test_decode_weighted(shape, decay):
    B, H, dh, r, Lm, lens = shape
    case = inputs.random_decode_case(seed=B + r, batch=B, heads=H, head_dim=dh, rank=r, max_len=Lm, dtype="bf16",
                                     lens=lens)
    prior = T.random_prior((B, Lm), 5)
    for b, L in enumerate(lens):
        prior[b, max(L - 1, 0):] = math.nan   # the new row's slot and the rows past it may hold anything
        for k in ("k_s", "v_s", "z_k", "z_v"):
            case[k][b, L:] = math.nan
    buffer = torch.full((B, Lm), -3.0)
    d = T.cuda(case)
    weights_out = buffer.cuda()
    out, lse, w, ws = lrkv.decode_weighted(*[d[k] for k in T.NAMES], prior.cuda(), decay=decay,
                                           weights_out=weights_out)
    _sync(ws)
    assert w is weights_out
    _check_decode(case, (out, lse, w), prior, decay, out_buffer=buffer)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("normed", [False, True])
def test_decode_weighted_paged_normed_in_place(page, normed):
    B, H, dh, r, Lm, lens = 3, 32, 128, 48, 256, [256, 1, 130]
    case = inputs.random_decode_case(seed=9, batch=B, heads=H, head_dim=dh, rank=r, max_len=Lm, dtype="bf16",
                                     lens=lens)
    pg = T.cuda(T.paged(case, page, 4))
    scales = torch.rand((B, H, Lm), generator=torch.Generator().manual_seed(2)) + 0.5 if normed else None
    prior = T.random_prior((B, Lm), 6)
    w = prior.clone().cuda()
    out, lse, w2, ws = lrkv.decode_weighted(*[pg[k] for k in T.NAMES], w, decay=1.0,
                                            key_scale=None if scales is None else scales.cuda(),
                                            block_table=pg["block_table"])
    _sync(ws)
    assert w2 is w
    _check_decode(case, (out, lse, w), prior, 1.0, key_scale=scales, out_buffer=prior)


def test_decode_weighted_without_earlier_weights_and_with_bad_lengths():
    B, H, dh, r, Lm = 2, 16, 64, 28, 64
    case = inputs.random_decode_case(seed=1, batch=B, heads=H, head_dim=dh, rank=r, max_len=Lm, dtype="bf16",
                                     lens=[64, 40])
    d = T.cuda(case)
    buffer = torch.full((B, Lm), 7.0)
    out, lse, w, ws = lrkv.decode_weighted(*[d[k] for k in T.NAMES], None, decay=0.0, weights_out=buffer.cuda())
    _sync(ws)
    _check_decode(case, (out, lse, w), torch.full((B, Lm), math.nan), 0.0, out_buffer=buffer)
    d["seq_lens"] = torch.tensor([65, 40], dtype=torch.int32, device="cuda")   # clamped to the capacity
    out2, lse2, w2, ws = lrkv.decode_weighted(*[d[k] for k in T.NAMES], None, decay=0.0, weights_out=buffer.cuda())
    _sync(ws, lrkv.LRKV_ERR_DEVICE_BOUNDS)
    assert torch.equal(w2, w) and torch.equal(out2, out)


def test_decode_weighted_flags_a_page_outside_the_pool():
    B, H, dh, r, Lm = 2, 16, 64, 28, 64
    case = inputs.random_decode_case(seed=1, batch=B, heads=H, head_dim=dh, rank=r, max_len=Lm, dtype="bf16",
                                     lens=[64, 40])
    pg = T.paged(case, 16, 4)
    pg["block_table"][0, 1] = 10 ** 6
    d = T.cuda(pg)
    out, lse, w, ws = lrkv.decode_weighted(*[d[k] for k in T.NAMES], None, decay=0.0,
                                           block_table=d["block_table"])
    _sync(ws, lrkv.LRKV_ERR_DEVICE_BOUNDS)
    assert abs(float(w[1, :40].sum()) - H) < 1e-3    # the other sequence is whole


# ------------------------------------------------------------------ prompt --

PROMPTS = [
    # B, H, d_h, r, max_len, lengths, q_len, window, page, normed
    (1, 4, 64, 16, 40, [40], 1, 1, 0, False),             # one query, heads side by side
    (2, 8, 128, 64, 400, [400, 131], 100, 32, 0, False),  # four heads to a tile
    (1, 2, 128, 64, 700, [700], 700, 700, 0, False),      # every query, several tiles, diagonal
    (2, 3, 64, 8, 300, [299, 150], 150, 37, 0, False),    # odd heads and window, rank 8
    (1, 1, 64, 24, 129, [129], 5, 5, 0, False),           # one head
    (3, 4, 128, 56, 512, [512, 257, 130], 129, 129, 16, False),  # pages within a key tile
    (2, 4, 128, 48, 512, [400, 128], 128, 100, 256, True),
    (1, 6, 128, 0, 260, [260], 260, 200, 0, True),        # no latents
    (1, 16, 128, 64, 3000, [2900], 64, 64, 0, False),     # more items than SMs
]


@pytest.mark.parametrize("shape", PROMPTS)
def test_prefill_weights(shape):
    B, H, dh, r, Lm, lens, Tq, window, page, normed = shape
    case = inputs.random_prefill_case(seed=Lm + r, batch=B, q_len=Tq, heads=H, head_dim=dh, rank=r, max_len=Lm,
                                      lens=lens)
    for b, L in enumerate(lens):
        for k in ("k_s", "z_k"):
            case[k][b, L:] = math.nan
    scales = torch.rand((B, H, Lm), generator=torch.Generator().manual_seed(2)) + 0.5 if normed else None
    scale = 1 / math.sqrt(dh)
    lse = np.zeros((B, H, Tq))
    rows = {}
    for b, L in enumerate(lens):
        for h in range(H):
            s = O.row_scores(case["q"][b, :, h], case["k_s"][b, :L], case["z_k"][b, :L], case["b_k"], h, scale,
                             None if scales is None else scales[b, h, :L])
            s = np.where(np.arange(L)[None] <= L - Tq + np.arange(Tq)[:, None], s, -np.inf)
            m = s.max(1)
            lse[b, h] = m + np.log(np.exp(s - m[:, None]).sum(1))
            rows[b, h] = s
    lse[0, 0, Tq - 1] = -np.inf if Tq > 1 else lse[0, 0, Tq - 1]   # a query that saw nothing gives nothing
    lse32 = torch.tensor(lse).float()
    prior, decay = T.random_prior((B, Lm), 8), 0.5
    buffer = torch.full((B, Lm), -3.0)
    d = T.cuda(T.paged(case, page, 3) if page else case)
    for b, L in enumerate(lens):
        prior[b, L - Tq:] = math.nan
    w, ws = lrkv.prefill_weights(d["q"], d["k_s"], d["z_k"], d["b_k"], lse32.cuda(), d["seq_lens"], prior.cuda(),
                                 window=window, decay=decay, weights_out=buffer.cuda(),
                                 key_scale=None if scales is None else scales.cuda(),
                                 block_table=d.get("block_table"))
    _sync(ws)
    fresh = O.prefill_weights_reference(case["q"], case["k_s"], case["z_k"], case["b_k"], lse32, case["seq_lens"],
                                        window, key_scale=scales)
    w = w.cpu().double().numpy()
    for b, L in enumerate(lens):
        bound = np.zeros(L)
        for h in range(H):
            ks = None if scales is None else scales[b, h, :L]
            err = T.score_error(case["q"][b, Tq - window:, h], case["k_s"][b, :L], case["z_k"][b, :L], case["b_k"],
                                h, scale, ks)
            given = T.f64(lse32[b, h, Tq - window:])
            s = np.where(np.isneginf(given)[:, None], -np.inf, rows[b, h][Tq - window:])
            bound += T.weight_bound(s, np.where(np.isneginf(given), 0.0, given), err)[0]
        want = O.accumulate_weights(fresh[b], prior[b], decay, L, Tq)
        bound += (H * (window / 128 + 1) + 32) * T.U * np.abs(want) + 1e-37
        assert np.all(np.abs(w[b, :L] - want) <= bound), (b, np.max(np.abs(w[b, :L] - want) / bound))
        assert np.array_equal(w[b, L:], buffer[b, L:].double().numpy())


def test_prefill_weights_take_the_prefill_s_lse():
    """prefill, then its weights: every query's weights sum to one per head."""
    B, Tq, H, Lm = 2, 130, 4, 300
    case = inputs.random_prefill_case(seed=2, batch=B, q_len=Tq, heads=H, head_dim=128, rank=64, max_len=Lm,
                                      lens=[300, 180])
    d = T.cuda(case)
    _, lse, _ = lrkv.prefill(*[d[k] for k in T.NAMES])
    w, ws = lrkv.prefill_weights(d["q"], d["k_s"], d["z_k"], d["b_k"], lse, d["seq_lens"], None, decay=0.0)
    _sync(ws)
    for b, L in enumerate([300, 180]):
        # lse within the prefill's 2e-3 of the exact one
        assert abs(float(w[b, :L].double().sum()) - H * Tq) <= H * Tq * 2.1e-3
        assert float(w[b, L:].abs().max()) == 0 if L < Lm else True


def test_prefill_weights_flag_lengths_and_pages():
    case = inputs.random_prefill_case(seed=2, batch=2, q_len=20, heads=2, head_dim=64, rank=16, max_len=64,
                                      lens=[64, 64])
    d = T.cuda(T.paged(case, 16, 1))
    lse = torch.zeros((2, 2, 20), device="cuda")
    args = (d["q"], d["k_s"], d["z_k"], d["b_k"], lse)
    lens = torch.tensor([64, 7], dtype=torch.int32, device="cuda")   # shorter than its queries
    _, ws = lrkv.prefill_weights(*args, lens, None, decay=0.0, block_table=d["block_table"])
    _sync(ws, lrkv.LRKV_ERR_DEVICE_BOUNDS)
    table = d["block_table"].clone()
    table[1, 2] = -5
    _, ws = lrkv.prefill_weights(*args, d["seq_lens"], None, decay=0.0, block_table=table)
    _sync(ws, lrkv.LRKV_ERR_DEVICE_BOUNDS)
    _, ws = lrkv.prefill_weights(*args, d["seq_lens"], None, decay=0.0, block_table=d["block_table"])
    _sync(ws)


# ---------------------------------------------------------------- eviction --

def _evict_case(B, H, dh, r, Lm, lens, dtype, seed, axes, ties=True):
    gen = torch.Generator().manual_seed(seed)
    case = inputs.random_decode_case(seed=seed, batch=B, heads=H, head_dim=dh, rank=r, max_len=Lm, dtype=dtype,
                                     lens=lens)
    w = torch.rand((B, Lm), generator=gen)
    if ties:
        w = (w * 6).floor()
    w[torch.rand((B, Lm), generator=gen) < 0.05] = math.nan
    w[torch.rand((B, Lm), generator=gen) < 0.05] = math.inf
    w[torch.rand((B, Lm), generator=gen) < 0.05] = -0.0
    w[torch.rand((B, Lm), generator=gen) < 0.02] = -math.inf
    case["weights"] = w
    case["order"] = torch.stack([torch.randperm(Lm, generator=gen) for _ in range(B)]).to(torch.int32) * 2
    case["key_scale"] = torch.rand((B, H, Lm), generator=gen)
    case["positions"] = T.random_positions(B, Lm, axes, 100, seed) if axes else None
    return case


EVICTS = [
    # B, H, d_h, r, max_len, lengths, budget, sink, recent, dtype, axes
    (1, 4, 16, 4, 8, [1], 1, 0, 0, "f32", 0),
    (3, 8, 64, 16, 64, [64, 0, 33], 32, 2, 5, "bf16", 3),        # shorter than, and at, the budget
    (4, 16, 64, 28, 100, [100, 99, 31, 2], 30, 0, 0, "bf16", 1),
    (2, 8, 128, 32, 300, [300, 257], 256, 4, 100, "f32", 4),     # few moves
    (2, 2, 64, 8, 2000, [2000, 1777], 7, 3, 4, "bf16", 2),       # the held rows alone
    (5, 4, 64, 8, 1025, [1025, 1024, 1023, 513, 1], 512, 1, 0, "bf16", 0),
    (1, 2, 64, 8, 20001, [20001], 5000, 5, 300, "bf16", 3),      # a cluster of CTAs
    (1, 2, 64, 8, 70003, [70003], 70002, 0, 1, "bf16", 0),       # one row goes
    (1, 1, 64, 8, 400000, [399999], 1000, 0, 10, "bf16", 0),     # keys read again, not kept
]


@pytest.mark.parametrize("shape", EVICTS)
@pytest.mark.parametrize("ordered", [False, True])
@pytest.mark.parametrize("page", [0, 1])
def test_evict(shape, ordered, page):
    B, H, dh, r, Lm, lens, budget, sink, recent, dtype, axes = shape
    if page:
        page = next((p for p in (64, 16, 4) if Lm % p == 0), 0)
        if not page:
            pytest.skip("capacity not a multiple of a page")
    case = _evict_case(B, H, dh, r, Lm, lens, dtype, seed=Lm + budget, axes=axes)
    d = T.cuda(T.paged(case, page, 3) if page else case)
    order = case["order"] if ordered else None
    outs = dict(weights_out=torch.full((B, Lm), -7.0), order_out=torch.full((B, Lm), -7, dtype=torch.int32),
                new_lens=torch.full((B,), -7, dtype=torch.int32),
                kept=torch.full((B, budget), -7, dtype=torch.int32))
    outs = T.cuda(outs)
    before = {k: d[k].clone() for k in ("k_s", "v_s", "z_k", "z_v", "key_scale", "weights", "order", "seq_lens")}
    new_lens, weights_out, order_out, ws = lrkv.evict(
        d["k_s"], d["v_s"], d["z_k"], d["z_v"], d["weights"], d["seq_lens"], budget, sink=sink, recent=recent,
        order=d["order"] if ordered else None, key_scale=d["key_scale"], positions=d["positions"],
        block_table=d.get("block_table"), **outs)
    _sync(ws)
    for k in ("weights", "order", "seq_lens"):
        assert torch.equal(d[k].view(torch.int32), before[k].view(torch.int32)), k   # inputs are left alone
    table = d["block_table"].cpu().numpy() if page else None

    def place(b, t):
        return (b, t) if not page else (int(table[b, t // page]), t % page)

    want = {k: before[k].cpu().clone() for k in ("k_s", "v_s", "z_k", "z_v")}
    ks, pos = case["key_scale"].clone(), None if not axes else case["positions"].clone()
    for b, L in enumerate(lens):
        src = O.evict_reference(case["weights"][b].numpy(), L, budget, sink, recent,
                                None if order is None else order[b].numpy())
        n = len(src)
        assert int(new_lens[b]) == n == min(L, budget)
        assert outs["kept"][b, :n].tolist() == src.tolist()
        assert outs["kept"][b, n:].tolist() == [-1] * (budget - n)
        index = torch.from_numpy(src)
        assert np.array_equal(weights_out[b, :n].cpu().numpy(), case["weights"][b, index].numpy(), equal_nan=True)
        assert torch.all(weights_out[b, n:] == -7) and torch.all(order_out[b, n:] == -7)
        age = order[b] if ordered else torch.arange(Lm, dtype=torch.int32)
        assert torch.equal(order_out[b, :n].cpu(), age[index])
        for i, j in enumerate(src):
            if i != j:
                for k in want:
                    want[k][place(b, i)] = before[k][place(b, int(j))].cpu()
        ks[b][:, :n] = case["key_scale"][b][:, index]
        if axes:
            pos[b, :n] = case["positions"][b, index]
    bits = torch.int32 if dtype == "f32" else torch.int16
    for k in want:   # bit for bit, unwritten rows (NaN) included
        assert torch.equal(d[k].cpu().view(bits), want[k].view(bits)), k
    assert torch.equal(d["key_scale"].cpu(), ks)
    if axes:
        assert torch.equal(d["positions"].cpu(), pos)


def test_evict_in_place_and_again():
    """Weights, order and lengths updated in place; a second call at the budget
    changes nothing; a held set larger than the budget competes by weight."""
    B, Lm, budget = 3, 500, 100
    case = _evict_case(B, 4, 64, 16, Lm, [500, 320, 60], "bf16", 5, 0)
    case["order"][2] = 7    # equal ages: every row of this sequence is held
    d = T.cuda(case)
    lrkv.evict(d["k_s"], d["v_s"], d["z_k"], d["z_v"], d["weights"], d["seq_lens"], budget, recent=10,
               order=d["order"])
    _sync()
    for b, L in enumerate([500, 320, 60]):
        src = O.evict_reference(case["weights"][b].numpy(), L, budget, 0, 10, case["order"][b].numpy())
        n = len(src)
        assert int(d["seq_lens"][b]) == n
        assert np.array_equal(d["weights"][b, :n].cpu().numpy(), case["weights"][b, src].numpy(), equal_nan=True)
        assert torch.equal(d["order"][b, :n].cpu(), case["order"][b, src])
        assert torch.equal(d["k_s"][b, :n].cpu(), case["k_s"][b, src])
        assert torch.equal(d["z_v"][b, n:].cpu(), case["z_v"][b, n:])
    before = {k: v.clone() for k, v in d.items() if isinstance(v, torch.Tensor)}
    lrkv.evict(d["k_s"], d["v_s"], d["z_k"], d["z_v"], d["weights"], d["seq_lens"], budget, recent=10,
               order=d["order"])
    _sync()
    for k, v in before.items():
        assert torch.equal(v.view(torch.int8), d[k].view(torch.int8)), k


def test_evict_held_rows_above_the_budget_compete_by_weight():
    case = _evict_case(1, 4, 64, 16, 200, [200], "bf16", 6, 0)
    case["order"][:] = 3
    d = T.cuda(case)
    kept = torch.empty((1, 50), dtype=torch.int32, device="cuda")
    lrkv.evict(d["k_s"], d["v_s"], d["z_k"], d["z_v"], d["weights"], d["seq_lens"], 50, recent=1, order=d["order"],
               kept=kept)
    _sync()
    assert kept[0].tolist() == O.evict_reference(case["weights"][0].numpy(), 200, 50, 0, 1,
                                                 case["order"][0].numpy()).tolist()


def test_evict_without_latents():
    case = _evict_case(2, 4, 64, 0, 90, [90, 80], "bf16", 7, 0)
    d = T.cuda(case)
    lrkv.evict(d["k_s"], d["v_s"], None, None, d["weights"], d["seq_lens"], 40)
    _sync()
    for b, L in enumerate([90, 80]):
        src = O.evict_reference(case["weights"][b].numpy(), L, 40)
        assert torch.equal(d["v_s"][b, :40].cpu(), case["v_s"][b, src])


def test_evict_flags_pages_and_lengths():
    case = _evict_case(2, 4, 64, 16, 64, [64, 64], "bf16", 8, 0)
    case["weights"][:] = torch.arange(64.0)            # the last rows move into the first
    pg = T.paged(case, 16, 2)
    pg["block_table"][0, 3] = 10 ** 6
    d = T.cuda(pg)
    kept = torch.empty((2, 32), dtype=torch.int32, device="cuda")
    _, _, _, ws = lrkv.evict(d["k_s"], d["v_s"], d["z_k"], d["z_v"], d["weights"], d["seq_lens"], 32,
                             block_table=d["block_table"], kept=kept)
    _sync(ws, lrkv.LRKV_ERR_DEVICE_BOUNDS)
    assert kept[0].tolist() == list(range(32, 64)) == kept[1].tolist()
    page = pg["block_table"]
    assert torch.equal(d["k_s"][page[1, 1]].cpu(), pg["k_s"][page[1, 3]])      # moved
    assert torch.equal(d["k_s"][page[0, 1]].cpu(), pg["k_s"][page[0, 1]])      # its page is missing: left
    lens = torch.tensor([-1, 70], dtype=torch.int32, device="cuda")
    c = T.cuda(case)
    new, _, _, ws = lrkv.evict(c["k_s"], c["v_s"], c["z_k"], c["z_v"], c["weights"], lens, 32)
    _sync(ws, lrkv.LRKV_ERR_DEVICE_BOUNDS)
    assert new.tolist() == [0, 32]


# ---------------------------------------------------------------- rotation --

@pytest.mark.parametrize("shape", [(1, 1, 1, 64, [32]), (2, 7, 3, 80, [10, 15, 15]), (3, 33, 16, 128, [16, 24, 24]),
                                   (2, 5, 8, 32, [4, 0, 6, 6]), (1, 300, 32, 128, [0, 64]), (1, 2, 300, 256, [128])])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_rotate(shape, dtype):
    B, n, H, dh, sections = shape
    gen = torch.Generator().manual_seed(n)
    x = torch.randn((B, n, H, dh), generator=gen).to(dtype)
    pos = T.random_positions(B, n, len(sections), 70000, 1)
    table = lrkv.rope_table(70000, dh)
    xd, pd = x.cuda(), pos.cuda()
    out = lrkv.rope_rotate(xd, pd, table, sections)
    _sync()
    assert torch.equal(xd.cpu(), x)
    ref = np.stack([np.stack([O.rope_rotate_axes(x[b, :, h], pos[b], sections) for h in range(H)], 1)
                    for b in range(B)])
    mag = np.abs(T.f64(x)).reshape(B, n, H, dh // 2, 2).sum(-1).repeat(2, -1)
    # cos, sin and two products and a sum in fp32 (4 u of the pair), one rounding
    half = 2.0 ** -8 if dtype == torch.bfloat16 else T.U
    bound = 4 * T.U * mag * (1 + half) + half * np.abs(ref)
    assert np.all(np.abs(T.f64(out) - ref) <= bound)
    lrkv.rope_rotate(xd, pd, table, sections, out=xd)   # in place
    _sync()
    assert torch.equal(xd, out)


def test_rope_rotate_flags_positions():
    table = lrkv.rope_table(10, 64)
    x = torch.randn((1, 3, 2, 64), generator=torch.Generator().manual_seed(0)).cuda()
    pos = torch.tensor([[[0], [10], [-1]]], dtype=torch.int32, device="cuda")
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    out = lrkv.rope_rotate(x, pos, table, [32], ws=ws)
    _sync(ws, lrkv.LRKV_ERR_DEVICE_BOUNDS)
    clamped = torch.tensor([[[0], [9], [0]]], dtype=torch.int32, device="cuda")
    ws.zero_()
    assert torch.equal(out, lrkv.rope_rotate(x, clamped, table, [32], ws=ws))
    _sync(ws)


ROPES = [
    # B, H, d_h, r, max_len, lengths, sections
    (1, 8, 64, 16, 16, [1], [32]),
    (3, 16, 64, 32, 300, [300, 0, 37], [8, 12, 12]),
    (2, 8, 128, 48, 257, [257, 130], [16, 24, 24]),
    (2, 16, 128, 64, 200, [199, 65], [0, 40, 20, 4]),
    (1, 8, 64, 48, 3001, [3001], [5, 27]),
    (20, 8, 128, 32, 40, [(11 * b) % 41 for b in range(20)], [63, 1]),
]


@pytest.mark.parametrize("shape", ROPES)
@pytest.mark.parametrize("weighted", [False, True])
def test_decode_rope_axes(shape, weighted):
    B, H, dh, r, Lm, lens, sections = shape
    case = inputs.random_decode_case(seed=Lm, batch=B, heads=H, head_dim=dh, rank=r, max_len=Lm, dtype="bf16",
                                     lens=lens)
    pos = T.random_positions(B, Lm, len(sections), 5000, 3)
    dev = pos.clone()
    prior = T.random_prior((B, Lm), 4)
    for b, L in enumerate(lens):
        dev[b, L:] = -10 ** 9          # rows past the length are not read
        prior[b, max(L - 1, 0):] = math.nan
        for k in ("k_s", "v_s", "z_k", "z_v"):
            case[k][b, L:] = math.nan
    table = lrkv.rope_table(5000, dh)
    buffer = torch.full((B, Lm), -3.0)
    d = T.cuda(case)
    q = [d[k] for k in T.NAMES]
    out, lse, w, ws = lrkv.decode_rope_axes(*q[:7], table, dev.cuda(), sections, q[7],
                                            weights=prior.cuda() if weighted else None, decay=0.5,
                                            weights_out=buffer.cuda() if weighted else None)
    _sync(ws)
    if not weighted:
        assert w is None
        fresh = O.decode_weights_reference(*[case[k] for k in T.NAMES], positions=pos, sections=sections)[2]
        w = buffer.clone()
        for b, L in enumerate(lens):
            w[b, :L] = torch.from_numpy(O.accumulate_weights(fresh[b], prior[b], 0.5, L, 1)) if L else w[b, :L]
    _check_decode(case, (out, lse, w), prior, 0.5, positions=pos, sections=sections, out_buffer=buffer)


def test_decode_rope_axes_with_row_positions_is_decode_rope():
    """One axis whose positions are the row indices: the same decode."""
    B, H, dh, r, Lm = 2, 8, 128, 48, 300
    d = T.cuda(inputs.random_decode_case(seed=8, batch=B, heads=H, head_dim=dh, rank=r, max_len=Lm, dtype="bf16",
                                         lens=[300, 150]))
    table = lrkv.rope_table(Lm, dh)
    q = [d[k] for k in T.NAMES]
    out, lse = lrkv.decode_rope(*q[:7], table, q[7])
    pos = torch.arange(Lm, dtype=torch.int32, device="cuda").expand(B, Lm)[..., None].contiguous()
    out2, lse2, _, ws = lrkv.decode_rope_axes(*q[:7], table, pos, [dh // 2], q[7])
    _sync(ws)
    assert float((out - out2).abs().max()) < 1e-4 and float((lse - lse2).abs().max()) < 1e-5


def test_decode_rope_axes_flags_positions():
    B, H, dh, r, Lm = 1, 8, 64, 16, 40
    d = T.cuda(inputs.random_decode_case(seed=8, batch=B, heads=H, head_dim=dh, rank=r, max_len=Lm, dtype="bf16",
                                         lens=[40]))
    table = lrkv.rope_table(100, dh)
    pos = torch.zeros((B, Lm, 2), dtype=torch.int32, device="cuda")
    pos[0, 7, 1] = 100
    q = [d[k] for k in T.NAMES]
    out, _, _, ws = lrkv.decode_rope_axes(*q[:7], table, pos, [16, 16], q[7])
    _sync(ws, lrkv.LRKV_ERR_DEVICE_BOUNDS)
    pos[0, 7, 1] = 99
    out2, _, _, ws = lrkv.decode_rope_axes(*q[:7], table, pos, [16, 16], q[7])
    _sync(ws)
    assert torch.equal(out, out2)


# ---------------------------------------------------------------- together --

@pytest.mark.parametrize("captured", [False, True])
def test_a_cache_kept_inside_its_budget(captured):
    """Prompt, its weights, eviction, then decode steps that append a token,
    attend, accumulate and evict, against the oracle on the host; eager, and
    with the steps as one captured graph replayed."""
    B, H, dh, r, Lm, Tq, budget, sink, recent, steps = 2, 4, 128, 64, 256, 150, 96, 2, 8, 3
    gen = torch.Generator().manual_seed(11)
    case = inputs.random_prefill_case(seed=12, batch=B, q_len=Tq, heads=H, head_dim=dh, rank=r, max_len=Lm,
                                      lens=[200, 150])
    d = T.cuda(case)
    lens = d["seq_lens"].clone()
    weights = torch.full((B, Lm), math.nan, device="cuda")
    weights[:, :50] = 0.25                                  # what earlier calls gave the 50 rows before the chunk
    order = torch.arange(Lm, dtype=torch.int32, device="cuda").repeat(B, 1)
    _, lse, _ = lrkv.prefill(*[d[k] for k in T.NAMES])
    lrkv.prefill_weights(d["q"], d["k_s"], d["z_k"], d["b_k"], lse, lens, weights, window=32)
    lrkv.evict(d["k_s"], d["v_s"], d["z_k"], d["z_v"], weights, lens, budget, sink=sink, recent=recent, order=order)
    _sync()
    # the host's copy of the state, followed by the oracle step by step
    host = {k: d[k].cpu() for k in ("k_s", "v_s", "z_k", "z_v")}
    host_w, host_o = weights.cpu().double().numpy().copy(), order.cpu().numpy().copy()
    assert lens.tolist() == [96, 96]
    kept = set(host_o[0, :96].tolist())
    assert {0, 1} | set(range(192, 200)) <= kept

    new = {k: torch.randn((steps,) + s, generator=gen).bfloat16() for k, s in
           dict(k_s=(B, dh), v_s=(B, dh), z_k=(B, H, r), z_v=(B, H, r), q=(B, H, dh)).items()}
    feed = {k: torch.zeros_like(v[0]).cuda() for k, v in new.items()}
    ids = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    out, lse1 = torch.empty((B, H, dh), device="cuda"), torch.empty((B, H), device="cuda")
    dims = lrkv.make_dims(B, H, dh, r, Lm, torch.bfloat16)
    ws1, ws2 = lrkv.decode_weighted_workspace(dims), lrkv.evict_workspace(B, Lm, budget)

    def step():
        at = lens.long()
        rows = torch.arange(B, device="cuda")
        for k in ("k_s", "v_s", "z_k", "z_v"):
            d[k][rows, at] = feed[k]
        order.scatter_(1, at[:, None], ids)
        lens.add_(1)
        lrkv.decode_weighted(feed["q"], d["k_s"], d["v_s"], d["z_k"], d["z_v"], d["b_k"], d["b_v"], lens, weights,
                             decay=0.9, out=out, lse=lse1, ws=ws1)
        lrkv.evict(d["k_s"], d["v_s"], d["z_k"], d["z_v"], weights, lens, budget, sink=sink, recent=recent,
                   order=order, ws=ws2)

    graph = None
    if captured:
        side = torch.cuda.Stream()
        saved = {k: v.clone() for k, v in d.items()}
        saved_state = [t.clone() for t in (lens, weights, order)]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                          # set-up outside the capture
        torch.cuda.current_stream().wait_stream(side)
        for k in d:
            d[k].copy_(saved[k])
        for t, s in zip((lens, weights, order), saved_state):
            t.copy_(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    seen = [200, 150]
    host_lens = [96, 96]
    for i in range(steps):
        for k in feed:
            feed[k].copy_(new[k][i])
        ids.copy_(torch.tensor([[seen[0] + i], [seen[1] + i]], dtype=torch.int32))
        graph.replay() if captured else step()
        _sync(ws1)
        _sync(ws2)
        c = dict(q=new["q"][i], b_k=case["b_k"], b_v=case["b_v"], seq_lens=torch.tensor(host_lens) + 1, **host)
        for b in range(B):
            for k in ("k_s", "v_s", "z_k", "z_v"):
                host[k][b, host_lens[b]] = new[k][i, b]
            host_o[b, host_lens[b]] = seen[b] + i
        ref_o, ref_l, fresh = O.decode_weights_reference(*[c[k] for k in T.NAMES])
        for b in range(B):
            L = host_lens[b] + 1
            for h in range(H):
                eo, el, _ = T.decode_bounds(c, b, h, 1 / math.sqrt(dh))
                assert np.all(np.abs(T.f64(out[b, h]) - ref_o[b, h]) <= eo)
                assert abs(float(lse1[b, h]) - ref_l[b, h]) <= el
            w = O.accumulate_weights(fresh[b], host_w[b], 0.9, L, 1)
            src = O.evict_reference(w, L, budget, sink, recent, host_o[b])
            n = len(src)
            assert int(lens[b]) == n
            # the device chose by its own fp32 weights: follow its choice where two rows are within their errors
            assert order[b, :n].tolist() == host_o[b, src].tolist()
            np.testing.assert_allclose(weights[b, :n].cpu().double().numpy(), w[src], rtol=2e-5, atol=1e-9)
            host_w[b, :n] = w[src]
            host_o[b, :n] = host_o[b, src]
            for k in ("k_s", "v_s", "z_k", "z_v"):
                host[k][b, :n] = host[k][b, src].clone()
                assert torch.equal(d[k][b, :n].cpu(), host[k][b, :n]), k
            host_lens[b] = n


def test_calls_take_their_stream_and_repeat_bit_for_bit():
    """On another stream, twice: the same bits (no atomics in the sums)."""
    B, H, dh, r, Lm = 2, 16, 128, 64, 2000
    d = T.cuda(inputs.random_decode_case(seed=8, batch=B, heads=H, head_dim=dh, rank=r, max_len=Lm, dtype="bf16",
                                         lens=[2000, 1500]))
    prompt = T.cuda(inputs.random_prefill_case(seed=2, batch=B, q_len=200, heads=H, head_dim=dh, rank=r, max_len=Lm,
                                               lens=[2000, 1500]))
    lse = torch.full((B, H, 200), 8.0, device="cuda")
    table = lrkv.rope_table(Lm, dh)
    pos = T.random_positions(B, Lm, 3, Lm, 3).cuda()
    torch.cuda.synchronize()
    got = []
    for stream in (torch.cuda.Stream(), torch.cuda.Stream(), None):
        a = lrkv.decode_weighted(*[d[k] for k in T.NAMES], None, decay=0.0, stream=stream,
                                 weights_out=torch.zeros((B, Lm), device="cuda"))
        torch.cuda.synchronize()
        p = lrkv.prefill_weights(prompt["q"], prompt["k_s"], prompt["z_k"], prompt["b_k"], lse, prompt["seq_lens"],
                                 None, decay=0.0, weights_out=torch.zeros((B, Lm), device="cuda"), stream=stream)
        torch.cuda.synchronize()
        x = lrkv.decode_rope_axes(*[d[k] for k in T.NAMES[:7]], table, pos, [16, 24, 24], d["seq_lens"], decay=0.0,
                                  weights_out=torch.zeros((B, Lm), device="cuda"), stream=stream)
        torch.cuda.synchronize()
        got.append([a[0], a[1], a[2], p[0], x[0], x[1], x[2]])
    for other in got[1:]:
        for s, t in zip(got[0], other):
            assert torch.equal(s, t)
