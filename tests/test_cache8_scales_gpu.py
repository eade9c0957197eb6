"""A decode over an 8-bit cache with scales that lrkv_quantize does not make: any
finite positive ones.

Bound of a decode's outputs, beside that of _cache8_util (u = 2^-24).  A
probability times its block's scale enters the value products over a power of
two, so that the largest of its tile lies in (1, 2^8): six e4m3 parts of it are off by
2^-24 of itself and, where it is small, by 2^-30, which is at most as much of the
tile's largest product.  Its exponent (x = log2 of the probability, plus
two whole numbers) is rounded twice: 2 u (|x| + 64) of it at most, as scales
that matter beside each other are within 2^64.  What is below the smallest normal
number is off by 2^-149 for every addition.
"""
import numpy as np
import pytest
import torch

import _budget_util as T
import _cache8_util as C
from _lib_util import ensure_built
from compressed_cache_decode_gb300 import lrkv

pytestmark = pytest.mark.gpu

U = T.U


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    lrkv.load()


def _check(case, out, lse):
    out, lse = T.f64(out), T.f64(lse)
    for b in range(case.B):
        L = case.lens[b]
        for h in range(case.H):
            _, want, _, lse_err = case.reference(b, h)
            assert abs(lse[b, h] - want) <= lse_err, (b, h)
            q, Bk, Bv = T.f64(case.c["q"][b, h]), T.f64(case.c["b_k"])[h], T.f64(case.c["b_v"])[h]
            ks, vs = case.rows("k_s")[b, :L, 0], case.rows("v_s")[b, :L, 0]
            zk, zv = (case.rows(n)[b, :L, h] for n in ("z_k", "z_v"))
            scale = case.dh ** -0.5
            s = scale * ((ks + zk @ Bk.T) @ q)
            p = np.abs(q) @ np.abs(Bk)
            qk, pz = np.abs(ks) @ np.abs(q), np.abs(zk) @ p
            err = (2 * U * (case.dh + 3 * case.r + 24) * (qk + pz) + 2.0 ** -24 * pz
                   + 2.0 ** -29 * np.abs(q).max() * np.abs(ks).sum(1) + 2.0 ** -37 * p.max() * np.abs(zk).sum(1)) * scale
            w, a = T.weight_bound(s[None], np.array([want]), err[None])
            a = a[0]
            x = (s - s.max()) / np.log(2)
            lift = np.abs(Bv).sum(1)
            mag = np.abs(vs) + np.abs(zv) @ np.abs(Bv).T
            floor = np.zeros(case.dh)
            for t in range(0, L, 128):
                rows = slice(t, min(L, t + 128))
                blocks = np.arange(rows.start, rows.stop) // 16
                top = [(a[rows] * case.scales[n][b, blocks, k]).max() for n, k in (("v_s", 0), ("z_v", h))]
                floor += 2.0 ** -30 * len(blocks) * 448 * (top[0] + top[1] * lift)
            bound = (w + a * (2.0 ** -24 + 2 * U * (L + 128) + 2 * U * (np.abs(x) + 64))) @ mag + floor
            bound += 2.0 ** -149 * (L + 200) * (1 + lift)
            off = np.abs(out[b, h] - a @ (vs + zv @ Bv.T))
            assert np.all(off <= bound), (b, h, off.max(), bound[np.argmax(off - bound)], np.abs(mag).max())


def _run(case, page=0):
    q, cache, b_k, b_v, n, table = case.cuda(page)
    out, lse, ws = lrkv.decode8(q, cache, b_k, b_v, n, block_table=table)
    torch.cuda.synchronize()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    _check(case, out, lse)
    return out


def _small_values(case, at, seed=0):
    """The values' numbers of blocks `at` become multiples of 2^-9 up to 2^-7."""
    rng = np.random.default_rng(seed)
    for n in ("v_s", "z_v"):
        v = case.values[n]
        for j in at:
            part = v[:, 16 * j:16 * j + 16]
            part[...] = rng.integers(-4, 5, part.shape) * 2.0 ** -9


@pytest.mark.parametrize("scale", [2.0 ** 127, 1.75 * 2.0 ** 127, 2.0 ** 126])
@pytest.mark.parametrize("everywhere", [False, True])
def test_decode8_of_the_largest_value_scales(scale, everywhere):
    at = range(25) if everywhere else (3, 24)
    case = C.Case(2, 12, 64, 32, 400, [400, 129], seed=3,
                  scales=lambda s, n: np.where(np.isin(np.arange(25), at)[None, :, None], scale, s) if n[0] + n[2] in
                  ("vs", "zv") else s)
    _small_values(case, at)
    out = _run(case)
    assert torch.isfinite(out).all() and out.abs().max() > 2.0 ** 100


@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -127, 1.5 * 2.0 ** -128, 2.0 ** -130, 2.0 ** -140])
def test_decode8_of_the_smallest_value_scales(scale):
    case = C.Case(2, 12, 64, 32, 400, [400, 129], seed=4,
                  scales=lambda s, n: np.full_like(s, scale) if n[0] + n[2] in ("vs", "zv") else s)
    out = _run(case, 16 if scale < 2.0 ** -128 else 0)
    assert out.any()


@pytest.mark.parametrize("bits", [5, 7, 14, 20, 30, 36, 60, 90])
@pytest.mark.parametrize("far", [0, 2])
@pytest.mark.parametrize("rows", [16, 128])
def test_decode8_of_weight_on_blocks_of_small_scale(bits, far, rows):
    """Every other block (or tile) has value scales 2^bits above its neighbours' and scores further below than that."""
    B, H, dh, r, L = 2, 12, 64, 32, 400
    case = C.Case(B, H, dh, r, L, [400, 129], seed=5)
    low = np.arange(L) // rows % 2 == 1
    for b in range(B):
        for h in range(H):
            p = T.f64(case.c["q"][b, h]) @ T.f64(case.c["b_k"])[h]
            case.values["z_k"][b, :, h] = np.sign(p)[None] * np.where(low, -1.0, 1.0)[:, None]
            # a score of (bits ln 2) / 2 + far on one side, its negative on the other
            case.scales["z_k"][b, :, h] = np.float32((bits * np.log(2) / 2 + far) * np.sqrt(dh) / np.abs(p).sum())
    for n in ("v_s", "z_v"):
        case.scales[n] = np.where(low[::16][None, :, None], 2.0 ** bits, 1.0) * np.ones_like(case.scales[n])
    _run(case, 16 if far else 0)


def test_decode8_of_scores_that_are_minus_infinity():
    """A tile whose scores leave fp32's range downwards has no weight."""
    case = C.Case(1, 8, 64, 32, 256, [256], seed=6)
    case.c["q"][0] = case.c["q"][0, :1]
    case.values["k_s"][0, 128:] = -448 * np.sign(T.f64(case.c["q"][0, 0]))[None, None]
    case.scales["k_s"][0, 8:] = 2.0 ** 127
    q, cache, b_k, b_v, n, _ = case.cuda()
    out, lse, _ = lrkv.decode8(q, cache, b_k, b_v, n)
    want, want_lse, _ = lrkv.decode8(q, cache, b_k, b_v, torch.full_like(n, 128))
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and torch.isfinite(out).all()
