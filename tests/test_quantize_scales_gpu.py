"""Rows stored in blocks of an 8-bit cache that have a caller's own scales."""
import numpy as np
import pytest
import torch

import _budget_util as T
import _cache8_util as C
from _lib_util import ensure_built
from compressed_cache_decode_gb300 import lrkv
from oracle import lrkv_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    lrkv.load()


def _ties(rng, n):
    """Numbers halfway between two e4m3 numbers."""
    return (2 * rng.integers(8, 16, n) + 1) * 2.0 ** rng.integers(-6, 4, n)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("grow", [False, True])
@pytest.mark.parametrize("small", [0, -100])
def test_quantize_into_blocks_with_scales_of_the_caller(dtype, grow, small):
    """Scales that are no powers of two, chosen so that quotients lie next to ties: of the new rows where they keep the
    block's scale, of the earlier rows where a new one makes it grow.  To the bit."""
    B, H, dh, r, L, start, n_new = 3, 16, 64, 28, 48, 7, 20
    rng = np.random.default_rng(11 + grow)
    held, rows = {}, {}
    for n in ("k_s", "v_s", "z_k", "z_v"):
        heads, width = (H, r) if n[0] == "z" else (1, dh)
        v = O.e4m3_round(rng.uniform(-448, 448, (B, L, heads, width)))
        s = rng.uniform(1, 2, (B, 3, heads)) * 2.0 ** small
        x = T.f64(torch.from_numpy(rng.uniform(-200, 200, (B, n_new, heads, width)) * 2.0 ** small).to(dtype))
        ties = _ties(rng, (B, heads))
        if grow:     # e4m3 f, a power of two scale to come: before = tie scale / f, rounded
            f = np.full((B, heads), 13.0 * 2.0 ** 4)
            v[:, 2, :, 0] = f
            top = 448 * 2.0 ** (small + 3)
            x[:, 1, :, 1] = top
            s[:, 0] = np.float32(np.where(ties < f, ties, ties / 16) * 2.0 ** (small + 3) / f)
        else:        # x, its scale = x / tie, rounded
            one = T.f64(torch.from_numpy(rng.uniform(50, 100, (B, heads)) * 2.0 ** small).to(dtype))
            x[:, 0, :, 0] = one
            s[:, 0] = np.float32(one / ties)
            x = np.clip(x, -400 * s[:, :1, :, None], 400 * s[:, :1, :, None])
            x = T.f64(torch.from_numpy(x).to(dtype))
        x[0, 3, 0, 2], x[1, 4, 0, 3] = np.inf, np.nan
        held[n], held[n + "_scale"], rows[n] = v, np.float32(s).astype(float), x
    flat = lambda n, t: t[:, :, 0] if n[2] == "s" else t
    tensors = {}
    for n in ("k_s", "v_s", "z_k", "z_v"):
        tensors[n] = flat(n, C.to8(held[n])).contiguous().cuda()
        tensors[n + "_scale"] = flat(n, torch.from_numpy(held[n + "_scale"]).float()).contiguous().cuda()
    arg = [flat(n, torch.from_numpy(rows[n]).to(dtype)).contiguous().cuda() for n in rows]
    lrkv.quantize(*arg, torch.full((B,), start, dtype=torch.int32).cuda(), lrkv.Cache8(**tensors))
    torch.cuda.synchronize()
    for n in rows:
        for b in range(B):
            v, s = O.quantize_reference(held[n][b], held[n + "_scale"][b], rows[n][b], start, n_new)
            assert (s[0] > held[n + "_scale"][b, 0]).all() == grow or not grow, n
            np.testing.assert_array_equal(T.f64(tensors[n + "_scale"][b]).reshape(s.shape), s, err_msg=n)
            np.testing.assert_array_equal(tensors[n][b].double().cpu().numpy().reshape(v.shape), v, err_msg=n)
