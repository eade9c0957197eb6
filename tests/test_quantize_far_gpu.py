"""Rows near the last number that an int holds, and past it."""
import pytest
import torch

from _lib_util import ensure_built
from compressed_cache_decode_gb300 import lrkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    lrkv.load()


@pytest.mark.parametrize("before_end, n, kept", [(0, 40, 0), (5, 40, 5), (16, 33, 16), (21, 700, 21), (-15, 17, 0)])
def test_quantize_at_the_end_of_the_longest_table(before_end, n, kept):
    """A table of 2^27 - 1 pages of 16 rows: the blocks past it begin at row 2^31 and further on."""
    page, dh, pages = 16, 16, 3
    blocks = 2 ** 27 - 1
    table = torch.full((1, blocks), -1, dtype=torch.int32, device="cuda")
    table[0, -2:] = torch.tensor([2, 1], dtype=torch.int32)
    cache = lrkv.empty_cache8(pages, page, 8, dh, 0)
    for t in cache.pools():
        t.fill_(1.0) if t.dtype == torch.float32 else t.view(torch.uint8).fill_(0x55)
    rows = torch.full((1, n, dh), 2.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    start = blocks * page - before_end
    lrkv.quantize(rows, rows, None, None, torch.tensor([start], dtype=torch.int32).cuda(), cache, block_table=table, ws=ws)
    torch.cuda.synchronize()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_ERR_DEVICE_BOUNDS
    # 2 / 2^-7 = 256: 0x78; blocks that were begun before keep their scale of 1: 2 = 0x40
    want = torch.full((pages * page, dh), 0x55, dtype=torch.uint8)
    scale = torch.ones(pages)
    for k, p in ((0, 1), (1, 2)):       # the last page of the table, the one before it
        lo, hi = max(0, page * (k + 1) - before_end), min(page, page * (k + 1) - before_end + kept)
        if lo < hi:
            begun = lo > 0
            want[p * page + lo:p * page + hi] = 0x40 if begun else 0x78
            scale[p] = 1.0 if begun else 2.0 ** -7
    assert torch.equal(cache.k_s.view(torch.uint8).cpu().view(-1, dh), want)
    assert torch.equal(cache.v_s.view(torch.uint8).cpu().view(-1, dh), want)
    assert torch.equal(cache.k_s_scale.cpu().flatten(), scale) and torch.equal(cache.v_s_scale.cpu().flatten(), scale)
