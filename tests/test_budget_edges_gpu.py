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
