"""The fp32 accuracy of the decodes that accumulate weights, on inputs whose
arithmetic has so few rounding steps that fewer bits anywhere show.

Bounds over sums of d_h or L terms admit more than two bf16 parts of an operand
leave (2^-16).  Here nearly all terms are zero, so additions that round are few:

- SCORES: one row's key meets the query in one shared and one latent product, s =
  scale (q_i k_i + p_c z_c) near 32, every other row's score is 0: lse is that
  score to e^-30.  p_c = q_i B_ic + q_j B_jc needs 24 bits.
- PROBABILITIES: small scores, and every value column and latent is non-zero in
  one row: out_d = a_j v_jd / l.
- SUMS: every score 0, so every probability 1; the values' sum over the first tile
  is 1 and over each later tile 1.992 2^-24, just under one step of fp32 at 1: an fp32
  addition rounds it to that step, a sum cut short of rounding loses it.

u = 2^-24 is half a step of fp32; products of two bf16 numbers are exact; a step
of the tensor cores may truncate, 2 u.  The planted mistakes (two bf16 parts of p,
of the probabilities, of the shared key; one accumulator, cut short, for all
tiles) are made in the oracle's arithmetic on the CPU and miss the bounds."""
import math

import numpy as np
import pytest
import torch

import _budget_util as T
from _lib_util import ensure_built
from compressed_cache_decode_gb300 import lrkv
from oracle import lrkv_oracle as O

U = T.U
SHAPES = [(16, 128, 64), (32, 128, 48), (16, 64, 28), (16, 64, 20)]     # heads, d_h, rank; the last: no own instance
ROPE_SHAPES = [(16, 128, 64), (8, 64, 16)]


def bf(x):
    return torch.as_tensor(x, dtype=torch.float64).bfloat16()


def parts(x, n):
    """x as the sum of n bf16 parts."""
    x = torch.as_tensor(x, dtype=torch.float64)
    total = torch.zeros_like(x)
    for _ in range(n):
        total += bf(x - total).double()
    return total.numpy()


def cut(x):
    """x cut to the 24 bits of fp32."""
    m, e = math.frexp(x)
    return math.ldexp(math.trunc(m * 2 ** 24), e - 24)


def empty_case(B, L, H, dh, r, lens):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    return dict(q=z(B, H, dh), k_s=z(B, L, dh), v_s=z(B, L, dh), z_k=z(B, L, H, r), z_v=z(B, L, H, r), b_k=z(H, dh, r),
                b_v=z(H, dh, r), seq_lens=torch.tensor(lens, dtype=torch.int32))


# ------------------------------------------------------------------ scores --

def score_case(H, dh, r, rope=False):
    gen = torch.Generator().manual_seed(H + dh + r)
    draw = lambda *s: bf(1 + torch.rand(s, generator=gen, dtype=torch.float64))
    lens = [1, 2, 15, 16, 17, 40, 63, 64, 65, 128, 129, 300, 31, 200, 299, 77]
    B, L = len(lens), 300
    c = empty_case(B, L, H, dh, r, lens)
    i, j = 2, dh - 6                                 # (even: first elements of their pairs)
    row = torch.tensor([int(torch.randint(0, n, (1,), generator=gen)) for n in lens])
    lat = torch.randint(0, r, (B,), generator=gen)
    # s near 2 * 12 + 1 * 8: most of it where the mistakes would be, the latents' part or (rope) the shared one
    c["q"][:, :, i] = draw(B, H)
    c["b_k"][:, i] = draw(H, r)
    if not rope:
        c["q"][:, :, j] = bf(draw(B, H).double() * 2 ** -9)
        c["b_k"][:, j] = draw(H, r)
    for b in range(B):
        c["k_s"][b, row[b], i] = bf(draw(1).double() * (12 if rope else 2))
        c["z_k"][b, row[b], :, lat[b]] = bf(draw(H).double() * (2 if rope else 8))
    c["v_s"][:, :, 0] = 1
    if not rope:
        return c, row, lat, (i, j), None
    pos = torch.randint(1, 2000, (B, L, 1), generator=gen, dtype=torch.int32)
    while np.any(rotation(c, pos, row, i) < 0.5):    # (a turned key that faces the query)
        pos[:] = torch.randint(1, 2000, (B, L, 1), generator=gen, dtype=torch.int32).where(
            torch.from_numpy(rotation(c, pos, row, i) < 0.5)[:, None, None], pos)
    return c, row, lat, (i, j), pos


def rotation(case, pos, row, i):
    """cos of the turn of pair i / 2 at the chosen rows."""
    dh = case["q"].shape[2]
    theta = O.rope_frequencies(dh, 10000.0)[i // 2]
    return np.cos(T.f64(pos)[np.arange(len(row)), row.numpy(), 0] * theta)


def score_parts(case, row, lat, dims):
    """(q_i k_i, p_c, z_c) of the chosen rows, [B, H] each."""
    i, j = dims
    B = len(row)
    q, bk = T.f64(case["q"]), T.f64(case["b_k"])
    p = q[:, :, i] * bk[:, i, :][:, lat].T + q[:, :, j] * bk[:, j, :][:, lat].T
    k = T.f64(case["k_s"])[np.arange(B), row, i]
    z = T.f64(case["z_k"])[np.arange(B), row][np.arange(B), :, lat]
    return q[:, :, i] * k[:, None], p, z


def lse_of(s, lens):
    """log(e^s + (L - 1) e^0)."""
    return np.logaddexp(s, np.log(np.maximum(lens.double().numpy()[:, None] - 1, 1e-300)))


def lse_bound(terms, s, steps):
    """`steps` roundings of u each of a score whose terms' magnitudes add up to
    `terms`; lse = (m + log2 l) ln 2 with l next to 1: four roundings of numbers
    below |s| + 4, two of log2 e."""
    return steps * U * terms + 8 * U * (np.abs(s) + 4)


# p: one rounding, and what three parts leave, 2^-24; high, low and third part's products and the shared one, and
# the sums of the four accumulators: 8 steps of 2 u; the scale in the log2 domain and its product, 2
SCORE_STEPS = 2 + 16 + 2
# the shared element joined to the rebuilt one, cos, its product, two sums over pairs, the difference of the two
# sums, three sums of a thread's lanes, the two halves' sum, the scale in the log2 domain and its product
ROPE_STEPS = 1 + 1 + 1 + 2 + 1 + 3 + 1 + 2


@pytest.mark.parametrize("shape", SHAPES)
def test_two_parts_of_p_would_show(shape):
    case, row, lat, dims, _ = score_case(*shape)
    qk, p, z = score_parts(case, row, lat, dims)
    s = qk + p * z
    assert np.all((s > 10) & (s < 140))
    bound = lse_bound(np.abs(qk) + np.abs(p * z), s, SCORE_STEPS)
    want = lse_of(s, case["seq_lens"])
    for n, fits in ((3, True), (2, False)):
        off = np.abs(lse_of(qk + parts(p, n) * z, case["seq_lens"]) - want)
        assert np.all(off <= bound) == fits
    ref = O.decode_weights_reference(*[case[k] for k in T.NAMES], scale=1.0)[1]
    np.testing.assert_allclose(ref, want, rtol=1e-12)


@pytest.mark.parametrize("shape", ROPE_SHAPES)
def test_two_parts_of_the_shared_key_would_show(shape):
    case, row, lat, dims, pos = score_case(*shape, rope=True)
    qk, p, z = score_parts(case, row, lat, dims)
    turn = rotation(case, pos, row, dims[0])[:, None]
    s = (qk + p * z) * turn
    bound = lse_bound((np.abs(qk) + np.abs(p * z)) * np.abs(turn), s, ROPE_STEPS)
    k = T.f64(case["k_s"])[np.arange(len(row)), row, dims[0]][:, None]
    q = T.f64(case["q"])[:, :, dims[0]]
    off = np.abs(q * parts(k * turn, 2) + p * z * turn - s)
    assert np.any(off > bound)
    ref = O.decode_weights_reference(*[case[x] for x in T.NAMES], scale=1.0, positions=pos,
                                     sections=[shape[1] // 2])[1]
    np.testing.assert_allclose(ref, lse_of(s, case["seq_lens"]), rtol=1e-10)


# ----------------------------------------------------------- probabilities --

def value_case(H, dh, r, L=12):
    """One non-zero row for each value column of the lower half of the head
    dimension and for each latent; latent c is output column dh / 2 + c."""
    gen = torch.Generator().manual_seed(H + dh + r)
    draw = lambda *s: bf(1 + torch.rand(s, generator=gen, dtype=torch.float64))
    B = 6
    c = empty_case(B, L, H, dh, r, [L] * B)
    c["q"][:, :, 0] = draw(B, H)
    c["k_s"][:, :, 0] = bf(torch.rand((B, L), generator=gen, dtype=torch.float64) / 4 - 0.125)
    for d in range(dh // 2):
        c["v_s"][torch.arange(B), (torch.arange(B) + d) % L, d] = draw(B)
    n = min(r, dh // 2)
    for k in range(n):
        c["z_v"][torch.arange(B), (torch.arange(B) + k) % L, :, k] = draw(B, H)
        c["b_v"][:, dh // 2 + k, k] = 1
    return c


def value_reference(case, n_parts=None):
    """(out, the rows' probabilities at each output) in 64 bits, the probabilities
    relative to the largest in n_parts bf16 parts."""
    q, k = T.f64(case["q"])[:, :, 0], T.f64(case["k_s"])[:, :, 0]
    s = q[:, :, None] * k[:, None, :]                                   # [B, H, L]
    p = np.exp(s - s.max(-1, keepdims=True))
    used = p if n_parts is None else parts(p, n_parts)
    a = used / p.sum(-1, keepdims=True)
    out = np.einsum("bhl,bld->bhd", a, T.f64(case["v_s"]))
    return out + np.einsum("bhl,blhc,hdc->bhd", a, T.f64(case["z_v"]), T.f64(case["b_v"])), s


def value_bound(out, s, L, steps):
    """Relative: the score (`steps` u of a |s| <= 1/4) in the exponent, twice (the
    row's and the largest); the exponential's two steps and its argument's roundings
    (6 u of |s| + 1 in all), in p and in l; l's sum over the rows and the merge
    (L + 8); three parts' products, 2 u each, and what they leave; the merge of the
    partials, the division and the lift (8)."""
    m = np.abs(s).max()
    return np.abs(out) * U * (2 * steps * m + 2 * 6 * (m + 1) + 2 * 4 + L + 8 + 6 + 1 + 8)


@pytest.mark.parametrize("shape", SHAPES + ROPE_SHAPES)
def test_two_parts_of_the_probabilities_would_show(shape):
    case = value_case(*shape)
    want, s = value_reference(case)
    bound = value_bound(want, s, 12, SCORE_STEPS if shape in SHAPES else ROPE_STEPS)
    assert np.abs(s).max() <= 0.25 and np.all(want >= 0)
    assert np.all(np.abs(value_reference(case, 3)[0] - want) <= bound)
    half = want.shape[2] // 2
    off = np.abs(value_reference(case, 2)[0] - want) > bound
    assert off[:, :, :half].any() and off[:, :, half:].any()           # shared columns and latents
    np.testing.assert_allclose(O.decode_weights_reference(*[case[k] for k in T.NAMES], scale=1.0)[0], want, rtol=1e-12)


# -------------------------------------------------------------------- sums --

STEP = 1.9921875 * 2.0 ** -24


def sum_case(H, dh, r, rows, head, tiles):
    """`tiles` tiles of `rows` rows for each of head / rows streams: the first head
    rows' values add up to 1 a tile, each later tile's to STEP."""
    L = head * tiles
    c = empty_case(1, L, H, dh, r, [L])
    for k in ("v_s", "z_v"):
        c[k][:, :head] = 1 / rows
        c[k][:, head:] = STEP / rows
    c["v_s"][..., dh // 2:] = 0
    for k in range(min(r, dh // 2)):
        c["b_v"][:, dh // 2 + k, k] = 1
    streams = head // rows
    want = (streams + STEP * streams * (tiles - 1)) / L
    cols = dh // 2 + min(r, dh // 2)
    # a tile's sum is exact; one addition of u of a running sum in [1, 2) per tile, 16 for the merge and the lift
    return c, want, cols, want * U * (tiles + 16)


def test_one_accumulator_cut_short_would_show():
    for rows, tiles in ((16, 256), (128, 256)):
        total = rounded = 1.0
        for _ in range(tiles - 1):
            total = cut(total + STEP)                                  # (a tile's steps one by one: the same)
            rounded = float(np.float32(rounded + STEP))
        want = 1 + STEP * (tiles - 1)
        assert abs(total - want) > want * U * (tiles + 16) >= 10 * abs(rounded - want)


# ------------------------------------------------------------------ on the GPU --

@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    lrkv.load()


def _run(case, rope_positions=None, scale=1.0):
    """(out, lse, weights) of decode_weighted, or of decode_rope_axes with one
    axis, in 64 bits on the host."""
    d = T.cuda(case)
    B, L = d["k_s"].shape[:2]
    w = torch.zeros((B, L), device="cuda")
    if rope_positions is None:
        out, lse, w, ws = lrkv.decode_weighted(*[d[k] for k in T.NAMES], w, scale=scale)
    else:
        dh = d["q"].shape[2]
        table = lrkv.rope_table(2000, dh)
        out, lse, w, ws = lrkv.decode_rope_axes(*[d[k] for k in T.NAMES[:7]], table, rope_positions.cuda(), [dh // 2],
                                                d["seq_lens"], weights=w, scale=scale)
    torch.cuda.synchronize()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    return T.f64(out), T.f64(lse), T.f64(w)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
def test_scores_of_few_terms(shape, lib):
    case, row, lat, dims, _ = score_case(*shape)
    qk, p, z = score_parts(case, row, lat, dims)
    s = qk + p * z
    out, lse, w = _run(case)
    off = np.abs(lse - lse_of(s, case["seq_lens"]))
    assert np.all(off <= lse_bound(np.abs(qk) + np.abs(p * z), s, SCORE_STEPS)), off.max()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", ROPE_SHAPES)
def test_turned_scores_of_few_terms(shape, lib):
    case, row, lat, dims, pos = score_case(*shape, rope=True)
    qk, p, z = score_parts(case, row, lat, dims)
    turn = rotation(case, pos, row, dims[0])[:, None]
    s = (qk + p * z) * turn
    out, lse, w = _run(case, pos)
    off = np.abs(lse - lse_of(s, case["seq_lens"]))
    assert np.all(off <= lse_bound((np.abs(qk) + np.abs(p * z)) * np.abs(turn), s, ROPE_STEPS)), off.max()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES + ROPE_SHAPES)
def test_probabilities_keep_their_bits(shape, lib):
    case = value_case(*shape)
    want, s = value_reference(case)
    pos = None if shape in SHAPES else torch.zeros((6, 12, 1), dtype=torch.int32)
    out = _run(case, pos)[0]
    off = np.abs(out - want)
    assert np.all(off <= value_bound(want, s, 12, SCORE_STEPS if pos is None else ROPE_STEPS)), off.max()


@pytest.mark.gpu
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("shape", [(16, 128, 64), (16, 64, 20), (8, 64, 16)])
def test_sums_over_many_tiles(shape, rope, lib, monkeypatch):
    """One CTA for a head group's whole history: 256 tiles in each running sum."""
    H, dh, r = shape
    if rope and r % 16:
        pytest.skip("not a rank of the rope decode")
    if not rope and H < 16:
        pytest.skip("covered by sixteen heads")
    monkeypatch.setenv("LRKV_SM_COUNT", "1")
    rows, head = (128, 128) if rope else (16, 64)          # (the scan's warp pairs take every fourth tile)
    case, want, cols, bound = sum_case(H, dh, r, rows, head, 256)
    out, lse, w = _run(case, torch.zeros((1, head * 256, 1), dtype=torch.int32) if rope else None)
    assert np.all(np.abs(out[0, :, :cols] - want) <= bound), np.abs(out[0, :, :cols] / want - 1).max()
    assert np.all(out[0, :, cols:] == 0)
    assert np.all(np.abs(lse - math.log(head * 256)) <= 8 * U * 16)
    # each row's weight: H equal probabilities of 1 / L
    assert np.all(np.abs(w * (head * 256) / H - 1) <= U * (8 * 16 + H))
