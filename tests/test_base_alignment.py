"""Bases b_k, b_v at addresses the decode's wide reads cannot start from.

The bf16 scan copies B^K in bulk (16 bytes) or, when the row tile's bases do not
fit its ring, reads it 8 bytes at a time; the narrow merge reads short rows of
B^V as 32-bit words.  A base that lies elsewhere is refused on the host, before
anything is enqueued (the addresses are fakes that are never dereferenced); one
that its path can read is not."""
import ctypes

import pytest
import torch

from _lib_util import ensure_built
from compressed_cache_decode_gb300 import inputs, lrkv

FAKE = 1 << 20
BAD, SPACE = lrkv.LRKV_ERR_INVALID_ARG, lrkv.LRKV_ERR_WORKSPACE   # (a workspace of no bytes ends a good call)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def decode(d, bk, bv):
    return lrkv.load().lrkv_decode(d, FAKE, FAKE, FAKE, FAKE, FAKE, bk, bv, FAKE, FAKE, FAKE, FAKE, 0, None)


def paged(d, bk, bv):
    return lrkv.load().lrkv_decode_paged(d, 64, 8, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, bk, bv, FAKE, FAKE, FAKE, FAKE,
                                         0, None)


def normed(d, bk, bv):
    return lrkv.load().lrkv_decode_normed(d, FAKE, FAKE, FAKE, FAKE, FAKE, bk, bv, FAKE, FAKE, FAKE, FAKE, FAKE, 0,
                                          None)


def weighted(d, bk, bv):
    return lrkv.load().lrkv_decode_weighted(d, FAKE, 0, 0, None, FAKE, FAKE, FAKE, FAKE, bk, bv, None, FAKE, 1.0, FAKE,
                                            FAKE, FAKE, FAKE, FAKE, 0, None)


def step(d, bk, bv):
    return lrkv.load().lrkv_decode_step(d, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, bk, bv, FAKE,
                                        FAKE, FAKE, FAKE, 0, None)


def step_paged(d, bk, bv):
    return lrkv.load().lrkv_decode_step_paged(d, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 64, 8, FAKE, FAKE, FAKE, FAKE,
                                              FAKE, bk, bv, FAKE, FAKE, FAKE, FAKE, 0, None)


CALLS = [decode, paged, normed, weighted, step, step_paged]
BULK = dict(head_dim=64, rank=32)      # 64 KB of bases a row tile: in the ring
WIDE = dict(head_dim=128, rank=64)     # 256 KB: read 8 bytes at a time


def dims(head_dim, rank, dtype="bf16"):
    return ctypes.byref(lrkv.make_dims(2, 16, head_dim, rank, 256, dtype))


@pytest.fixture
def plans(monkeypatch):
    monkeypatch.setenv("LRKV_SM_COUNT", "152")     # plans without a device
    return monkeypatch


@pytest.mark.parametrize("call", CALLS)
def test_bases_where_a_wide_read_cannot_start_are_refused(plans, call):
    for bk in (FAKE + 2, FAKE + 4, FAKE + 8):
        assert call(dims(**BULK), bk, FAKE) == BAD
    for bk in (FAKE + 2, FAKE + 4):
        assert call(dims(**WIDE), bk, FAKE) == BAD
    assert call(dims(**WIDE), FAKE + 8, FAKE) == SPACE
    assert call(dims(**BULK), FAKE, FAKE + 1) == BAD
    assert call(dims(**BULK), FAKE, FAKE + 2) == SPACE          # the wide merge falls back to elements
    assert call(dims(**BULK), FAKE, FAKE) == SPACE
    plans.setenv("LRKV_DECODE_WIDE_MERGE", "0")                 # the narrow merge
    assert call(dims(**BULK), FAKE, FAKE + 2) == BAD
    assert call(dims(**BULK), FAKE, FAKE + 4) == SPACE
    assert call(dims(**WIDE), FAKE, FAKE + 2) == SPACE          # its long rows: elements


def test_single_elements_need_no_more_than_theirs(plans):
    assert decode(dims(32, 64), FAKE + 2, FAKE + 2) == SPACE    # bf16 outside the streaming scan
    assert decode(dims(64, 32, "f32"), FAKE + 4, FAKE + 4) == SPACE
    assert decode(dims(64, 32, "f32"), FAKE + 2, FAKE) == BAD
    assert decode(dims(64, 32, "f32"), FAKE, FAKE + 2) == BAD


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [BULK, WIDE])
def test_bases_8_bytes_off_decode_the_same_or_are_refused(shape):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    case = inputs.random_decode_case(seed=4, batch=2, heads=16, max_len=200, dtype="bf16", lens=[200, 77], **shape)
    d = {k: v.cuda() for k, v in case.items()}
    args = [d[k] for k in ("q", "k_s", "v_s", "z_k", "z_v", "b_k", "b_v", "seq_lens")]
    off = [torch.empty(b.numel() + 4, dtype=b.dtype, device="cuda")[4:].view(b.shape).copy_(b) for b in args[5:7]]
    assert all(b.data_ptr() % 16 == 8 for b in off)
    w = torch.zeros((2, 200), device="cuda")
    want = lrkv.decode(*args), lrkv.decode_weighted(*args, w.clone())
    if shape is BULK:
        with pytest.raises(lrkv.LRKVError):
            lrkv.decode(*args[:5], *off, args[7])
        with pytest.raises(lrkv.LRKVError):
            lrkv.decode_weighted(*args[:5], *off, args[7], w.clone())
        return
    got = lrkv.decode(*args[:5], *off, args[7]), lrkv.decode_weighted(*args[:5], *off, args[7], w.clone())
    torch.cuda.synchronize()
    for a, b in ((got[0], want[0]), (got[1][:3], want[1][:3])):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
