"""Waits that run out in the calls that keep a cache inside a token budget.

With the bound of the waits cut short (LRKV_WAIT_LIMIT_CYCLES; caches larger
than L2 and L2 flushed, so that copies are under way) a call gives up
somewhere: at one cycle at its first waits, at larger bounds in the middle of its
work, with some warps gone on and others not.  It must end, wait at the full
bound for every copy and MMA that it issued, and say so in its status word; the
next call on the same workspace is whole."""
import math

import pytest
import torch

import _budget_util as T
from _lib_util import ensure_built
from compressed_cache_decode_gb300 import inputs, lrkv

pytestmark = pytest.mark.gpu

LIMITS = [1, 300, 1000, 2000, 4000, 10000]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    lrkv.load()


def _give_up_and_recover(run, ws, monkeypatch):
    """run() under every limit and whole again after each; its results as a list."""
    want = run()
    torch.cuda.synchronize()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    flush = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    seen = []
    for limit in LIMITS:
        flush.fill_(1)
        monkeypatch.setenv("LRKV_WAIT_LIMIT_CYCLES", str(limit))
        run()
        torch.cuda.synchronize()
        seen.append(lrkv.lrkv_read_device_status(ws))
        monkeypatch.delenv("LRKV_WAIT_LIMIT_CYCLES")
        got = run()
        torch.cuda.synchronize()
        assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
        for g, t in zip(got, want):
            assert torch.equal(g, t), limit
    assert seen[0] == lrkv.LRKV_ERR_TIMEOUT
    assert set(seen) <= {lrkv.LRKV_OK, lrkv.LRKV_ERR_TIMEOUT}


def _decode_case(B=2, H=32, dh=128, r=48, Lm=32768, lens=(32768, 20000)):
    d = T.cuda(inputs.random_decode_case(seed=5, batch=B, heads=H, head_dim=dh, rank=r, max_len=Lm, dtype="bf16",
                                         lens=list(lens)))
    return d, lrkv.make_dims(B, H, dh, r, Lm, torch.bfloat16)


@pytest.mark.parametrize("heads, head_dim, rank", [(32, 128, 48), (16, 64, 64)])
def test_decode_rope_axes(heads, head_dim, rank, monkeypatch):
    d, dims = _decode_case(H=heads, dh=head_dim, r=rank)
    ws = lrkv.decode_rope_axes_workspace(dims)
    table = lrkv.rope_table(32768, head_dim)
    pos = torch.arange(32768, dtype=torch.int32, device="cuda").expand(2, 32768)[..., None].contiguous()

    def run():
        w = torch.zeros((2, 32768), device="cuda")
        return lrkv.decode_rope_axes(*[d[k] for k in T.NAMES[:7]], table, pos, [head_dim // 2], d["seq_lens"],
                                     weights=w, ws=ws)[:3]

    _give_up_and_recover(run, ws, monkeypatch)


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("heads, head_dim, rank, q_len, window", [
    (32, 128, 48, 32, 32),      # a window of one tile
    (16, 64, 64, 40, 7),
    (32, 128, 48, 300, 300),    # of several
    (16, 64, 64, 200, 130),
])
def test_prefill_weights(heads, head_dim, rank, q_len, window, padded, monkeypatch):
    d = T.cuda(inputs.random_prefill_case(seed=2, batch=2, q_len=q_len, heads=heads, head_dim=head_dim, rank=rank,
                                          max_len=32768, lens=[32768, 20000]))
    dims = lrkv.make_dims(2, heads, head_dim, rank, 32768, torch.bfloat16)
    ws = lrkv.prefill_weights_workspace(dims, window)
    lse = torch.full((2, heads, q_len), 8.0, device="cuda")
    if padded:
        lse[..., ::3] = -math.inf

    def run():
        w = torch.zeros((2, 32768), device="cuda")
        return lrkv.prefill_weights(d["q"], d["k_s"], d["z_k"], d["b_k"], lse, d["seq_lens"], w, window=window,
                                    ws=ws)[:1]

    _give_up_and_recover(run, ws, monkeypatch)


@pytest.mark.parametrize("heads, head_dim, rank, dtype", [(32, 128, 48, "bf16"), (64, 128, 64, "f32")])
def test_evict(heads, head_dim, rank, dtype, monkeypatch):
    """Rows of one part and of two; every run on a fresh copy of the cache."""
    L, budget = (32768, 16000) if dtype == "bf16" else (6000, 3000)
    case = T.cuda(inputs.random_decode_case(seed=5, batch=2, heads=heads, head_dim=head_dim, rank=rank, max_len=L,
                                            dtype=dtype, lens=[L, L - 1000]))
    case["weights"] = torch.rand((2, L), generator=torch.Generator().manual_seed(1)).cuda()
    names = ("k_s", "v_s", "z_k", "z_v", "weights", "seq_lens")
    ws = lrkv.evict_workspace(2, L, budget)
    flush = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")

    def run():
        state = [case[k].clone() for k in names]
        flush.fill_(1)
        lrkv.evict(*state, budget, sink=2, recent=10, ws=ws)
        return state

    _give_up_and_recover(run, ws, monkeypatch)
