"""Cache8 keeps what it was made with: its calls use addresses that were taken once."""
import ctypes
import gc

import pytest
import torch

from compressed_cache_decode_gb300 import lrkv

B, H, DH, R, L = 2, 16, 64, 32, 48
E4M3 = torch.float8_e4m3fn


@pytest.fixture
def parts(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    return dict(k_s=torch.zeros(B, L, DH, dtype=E4M3), v_s=torch.zeros(B, L, DH, dtype=E4M3),
                z_k=torch.zeros(B, L, H, R, dtype=E4M3), z_v=torch.zeros(B, L, H, R, dtype=E4M3),
                k_s_scale=torch.ones(B, 3), v_s_scale=torch.ones(B, 3), z_k_scale=torch.ones(B, 3, H),
                z_v_scale=torch.ones(B, 3, H))


def held(cache):
    return ctypes.cast(ctypes.pointer(cache.ref._obj), ctypes.POINTER(ctypes.c_void_p * 8)).contents[:]


def test_attributes_cannot_be_exchanged(parts):
    cache = lrkv.Cache8(**parts)
    want = [t.data_ptr() for t in parts.values()]
    assert held(cache) == want
    for name in (*lrkv.Cache8.NAMES, "device", "shape", "ref", "at", "held", "other"):
        with pytest.raises(AttributeError):
            setattr(cache, name, parts["k_s"].clone())
        with pytest.raises(AttributeError):
            delattr(cache, name)
    assert held(cache) == want and all(a is b for a, b in zip(cache.pools(), parts.values()))
    assert cache.device == 0 and cache.shape == (B, L, H, DH, R)


def test_memory_exchanged_under_a_tensor_is_kept_and_noticed(parts):
    cache = lrkv.Cache8(**parts)
    old = parts["v_s"].view(torch.uint8).fill_(7).data_ptr()
    parts["v_s"].set_(torch.zeros(B, L, DH, dtype=E4M3))
    gc.collect()
    with pytest.raises(ValueError):
        cache.pools()
    # the bytes that the calls' addresses name are still there
    assert held(cache)[1] == old
    assert bytes((ctypes.c_ubyte * (B * L * DH)).from_address(old)) == b"\x07" * (B * L * DH)


def test_a_cache_without_latents(parts):
    cache = lrkv.Cache8(**dict(parts, z_k=None, z_v=None, z_k_scale=None, z_v_scale=None))
    assert len(cache.pools()) == 4 and held(cache)[2] is None and cache.shape == (B, L, 0, DH, 0)


def test_a_table_of_more_rows_than_an_int_holds(monkeypatch):
    """2^32 + 2^20 rows a sequence would reach the library as 2^20."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    rows = torch.zeros(1, 1 << 20, 16, dtype=E4M3)
    scales = torch.ones(1, 1 << 16)
    cache = lrkv.Cache8(rows, rows, None, None, scales, scales, None, None)
    for blocks, fits in ((2047, True), (2048, False), (4097, False)):
        table = torch.zeros(2, blocks, dtype=torch.int32)
        if fits:
            assert cache.rows(table, 2, 1, 16, 0, 0) == (blocks << 20, 1 << 20, 1)
            continue
        with pytest.raises(ValueError, match="more than"):
            lrkv.decode8(torch.zeros(2, 1, 16).bfloat16(), cache, None, None, torch.ones(2, dtype=torch.int32),
                         block_table=table)
        with pytest.raises(ValueError, match="more than"):
            new = torch.zeros(2, 1, 16).bfloat16()
            lrkv.quantize(new, new, None, None, torch.ones(2, dtype=torch.int32), cache, block_table=table)
