"""Values at the edge of what the header allows, in the calls that keep a cache
inside a token budget."""
import math

import numpy as np
import pytest
import torch

import _budget_util as T
from _lib_util import ensure_built
from compressed_cache_decode_gb300 import inputs, lrkv
from oracle import lrkv_oracle as O

pytestmark = pytest.mark.gpu
LAST = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    lrkv.load()


@pytest.mark.parametrize("L, budget", [(60, 20), (5000, 900), (20001, 5000)])
@pytest.mark.parametrize("sink, recent", [(0, 3), (2, 1), (0, 0)])
def test_evict_up_to_the_largest_age(L, budget, sink, recent):
    """Ages that end at 2^31 - 1: `newest` is 2^31, and the newest rows are held."""
    case = inputs.random_decode_case(seed=L, batch=2, heads=2, head_dim=64, rank=8, max_len=L, dtype="bf16",
                                     lens=[L, L - 1])
    gen = torch.Generator().manual_seed(L)
    order = torch.stack([torch.randperm(L, generator=gen) for _ in range(2)]).to(torch.int32)
    for b in range(2):
        top = order[b] >= order[b, :L - b].max() - 5
        order[b, top] += LAST - int(order[b, :L - b].max())      # six ages end at the largest one
        order[b, L - b:] = LAST                                  # (rows past the length may hold anything)
    weights = torch.rand((2, L), generator=gen)
    weights[order > LAST - 10] = 0                               # the newest rows go unless they are held
    d = T.cuda(case)
    kept = torch.empty((2, budget), dtype=torch.int32, device="cuda")
    _, _, _, ws = lrkv.evict(d["k_s"], d["v_s"], d["z_k"], d["z_v"], weights.cuda(), d["seq_lens"], budget, sink=sink,
                             recent=recent, order=order.cuda(), kept=kept)
    torch.cuda.synchronize()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    for b in range(2):
        n = L - b
        want = O.evict_reference(weights[b].numpy(), n, budget, sink, recent, order[b].numpy())
        assert kept[b].tolist() == want.tolist()
        assert int((order[b, want] > LAST - recent).sum()) == recent


@pytest.mark.parametrize("heads, q_len, window", [(8, 40, 32), (8, 40, 17), (3, 40, 5), (4, 300, 300), (5, 290, 130)])
@pytest.mark.parametrize("rank", [16, 0])
def test_prefill_weights_of_queries_that_are_padding(heads, q_len, window, rank):
    """A query with lse -inf gives nothing, whatever it holds: the weights of the
    others are those of a call on zeros in its place."""
    B, dh, L, lens = 2, 64, 700, [700, 430]
    case = inputs.random_prefill_case(seed=heads + window, batch=B, q_len=q_len, heads=heads, head_dim=dh, rank=rank,
                                      max_len=L, lens=lens)
    gen = torch.Generator().manual_seed(window)
    lse = torch.rand((B, heads, q_len), generator=gen) + 6
    pad = torch.rand((B, q_len), generator=gen) < 0.3
    pad[:, -1] = True
    lse[pad[:, None, :].expand(B, heads, q_len)] = -math.inf
    case["q"][pad] = 0
    d = T.cuda(case)

    def run(q):
        w, ws = lrkv.prefill_weights(q, d["k_s"], d["z_k"], d["b_k"], lse.cuda(), d["seq_lens"], None, window=window,
                                     decay=0.0)
        torch.cuda.synchronize()
        assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
        return w

    want = run(d["q"])
    assert torch.isfinite(want).all() and float(want.max()) > 0
    for fill in (math.nan, math.inf):
        q = d["q"].clone()
        q[pad.cuda()] = fill
        assert torch.equal(run(q), want)


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_a_budget_kept_where_rows_are_within_their_errors(seed):
    """Steps of decode_weighted and evict followed on the host by the device's own
    choice: every dropped row weighs no more than every kept one that is not held,
    within the errors of their weights (equal keys make many rows that near), and
    what is kept is whole."""
    B, H, dh, r, L, budget, sink, recent, steps, decay = 2, 8, 64, 16, 80, 48, 2, 6, 12, 0.9
    gen = torch.Generator().manual_seed(seed)
    case = inputs.random_decode_case(seed=seed, batch=B, heads=H, head_dim=dh, rank=r, max_len=L, dtype="bf16",
                                     lens=[budget] * B)
    for k in ("k_s", "z_k"):                                  # three keys for all rows: ties up to the arithmetic
        case[k][:] = case[k][:, torch.arange(L) % 3]
    d = T.cuda(case)
    host = {k: case[k].clone() for k in ("k_s", "v_s", "z_k", "z_v")}
    w = np.zeros((B, L))
    error = np.zeros((B, L))
    number = np.tile(np.arange(L), (B, 1))                    # the row's token
    order = torch.arange(L, dtype=torch.int32).repeat(B, 1).cuda()
    weights, lens = torch.zeros((B, L), device="cuda"), d["seq_lens"]
    for step in range(steps):
        n = budget + 1
        new = {k: torch.randn((B,) + tuple(host[k].shape[2:]), generator=gen).bfloat16() for k in ("v_s", "z_v")}
        new.update({k: host[k][:, step % 3].clone() for k in ("k_s", "z_k")})
        q = torch.randn((B, H, dh), generator=gen).bfloat16()
        for k in host:
            host[k][:, budget] = new[k]
            d[k][:, budget] = new[k].cuda()
        number[:, budget] = L + step
        order[:, budget] = L + step
        lens.fill_(n)
        kept = torch.empty((B, budget), dtype=torch.int32, device="cuda")
        lrkv.decode_weighted(q.cuda(), d["k_s"], d["v_s"], d["z_k"], d["z_v"], d["b_k"], d["b_v"], lens, weights,
                             decay=decay)
        got = T.f64(weights)
        lrkv.evict(d["k_s"], d["v_s"], d["z_k"], d["z_v"], weights, lens, budget, sink=sink, recent=recent,
                   order=order, kept=kept)
        torch.cuda.synchronize()
        c = dict(q=q, b_k=case["b_k"], b_v=case["b_v"], seq_lens=torch.tensor([n] * B), **host)
        fresh = O.decode_weights_reference(*[c[k] for k in T.NAMES])[2]
        for b in range(B):
            w[b, :n] = O.accumulate_weights(fresh[b], w[b], decay, n, 1)
            error[b, :budget] *= decay
            error[b, budget] = 0
            # (the sum over the heads, the decay as fp32 and its product)
            error[b, :n] += sum(T.decode_bounds(c, b, h, 1 / math.sqrt(dh))[2] for h in range(H))
            error[b, :n] += (H + 4) * T.U * w[b, :n]
            assert np.all(np.abs(got[b, :n] - w[b, :n]) <= error[b, :n])
            source = kept[b].cpu().numpy()
            stays = np.zeros(n, bool)
            stays[source] = True
            assert len(set(source.tolist())) == budget
            held = (number[b, :n] < sink) | (number[b, :n] >= number[b, :n].max() + 1 - recent)
            assert np.all(stays[held])
            top, bottom = w[b, :n] + error[b, :n], w[b, :n] - error[b, :n]
            assert bottom[~stays].max() <= top[stays & ~held].min()
            w[b, :budget], error[b, :budget], number[b, :budget] = w[b, source], error[b, source], number[b, source]
            assert order[b, :budget].tolist() == number[b, :budget].tolist()
            for k in host:
                host[k][b, :budget] = host[k][b, source].clone()
                assert torch.equal(d[k][b, :budget].cpu(), host[k][b, :budget]), k
