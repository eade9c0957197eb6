"""Pins of the oracle's weight accumulation, eviction and multi-axis rotation:
closed forms, the existing pinned functions as special cases, invariances, and
planted mistakes that the pins catch."""
import math

import numpy as np
import pytest
import torch

from compressed_cache_decode_gb300 import inputs
from oracle import lrkv_oracle as O


def _case(lens=(9, 4), heads=4, dim=16, rank=8, max_len=9, seed=0):
    return inputs.random_decode_case(seed=seed, batch=len(lens), heads=heads, head_dim=dim, rank=rank,
                                     max_len=max_len, dtype="bf16", lens=list(lens))


def test_decode_weights_agree_with_the_pinned_decode_and_sum_to_the_heads():
    c = _case()
    args = [c[k] for k in ("q", "k_s", "v_s", "z_k", "z_v", "b_k", "b_v", "seq_lens")]
    out, lse, fresh = O.decode_weights_reference(*args)
    ref_o, ref_l = O.decode_reference(*args)
    np.testing.assert_allclose(out, ref_o, rtol=0, atol=1e-12)
    np.testing.assert_allclose(lse, ref_l, rtol=0, atol=1e-12)
    for f, L in zip(fresh, c["seq_lens"].tolist()):
        assert f.shape == (L,) and abs(f.sum() - 4) < 1e-12   # each head's weights sum to one


def test_decode_weights_of_a_zero_query_are_uniform():
    c = _case()
    c["q"] = torch.zeros_like(c["q"])
    fresh = O.decode_weights_reference(*[c[k] for k in ("q", "k_s", "v_s", "z_k", "z_v", "b_k", "b_v",
                                                        "seq_lens")])[2]
    for f, L in zip(fresh, c["seq_lens"].tolist()):
        np.testing.assert_allclose(f, 4 / L, rtol=1e-12)


def test_prefill_weights_of_one_query_are_the_decode_weights():
    c = _case()
    _, lse, fresh = O.decode_weights_reference(*[c[k] for k in ("q", "k_s", "v_s", "z_k", "z_v", "b_k", "b_v",
                                                                "seq_lens")])
    got = O.prefill_weights_reference(c["q"][:, None], c["k_s"], c["z_k"], c["b_k"], lse[:, :, None],
                                      c["seq_lens"], 1)
    for a, b in zip(got, fresh):
        np.testing.assert_allclose(a, b, rtol=1e-12)


def test_prefill_weights_count_every_query_of_the_window_once():
    c = inputs.random_prefill_case(seed=3, batch=2, q_len=5, heads=3, head_dim=16, rank=8, max_len=9, lens=[9, 5])
    _, lse = O.prefill_reference(*[c[k] for k in ("q", "k_s", "v_s", "z_k", "z_v", "b_k", "b_v", "seq_lens")])
    for window in (1, 3, 5):
        fresh = O.prefill_weights_reference(c["q"], c["k_s"], c["z_k"], c["b_k"], lse, c["seq_lens"], window)
        for f in fresh:
            assert abs(f.sum() - 3 * window) < 1e-10
    # the newest row is seen by the newest query alone
    whole = O.prefill_weights_reference(c["q"], c["k_s"], c["z_k"], c["b_k"], lse, c["seq_lens"], 5)
    last = O.prefill_weights_reference(c["q"], c["k_s"], c["z_k"], c["b_k"], lse, c["seq_lens"], 1)
    assert whole[0][-1] == pytest.approx(last[0][-1], rel=1e-12)


def test_accumulation_skips_the_new_rows():
    got = O.accumulate_weights([1.0, 1.0, 1.0], [2.0, 4.0, math.nan], 0.5, 3, 1)
    np.testing.assert_array_equal(got, [2.0, 3.0, 1.0])
    np.testing.assert_array_equal(O.accumulate_weights([1.0, 2.0], [math.nan] * 2, 0.0, 2, 1), [1.0, 2.0])


@pytest.mark.parametrize("seed", range(6))
def test_evict_keeps_the_best_set_and_moves_no_row_twice(seed):
    rng = np.random.default_rng(seed)
    L, budget, sink, recent = 20, 8, 2, 3
    w = rng.integers(0, 4, L).astype(np.float64)   # ties
    src = O.evict_reference(w, L, budget, sink, recent)
    assert len(set(src)) == budget and {0, 1, 17, 18, 19} <= set(src)
    free = [j for j in range(L) if 2 <= j < 17]
    kept = [j for j in free if j in src]
    gone = [j for j in free if j not in src]
    assert len(kept) == budget - 5
    # every kept one beats every dropped one, by weight or by index
    assert all((-w[a], a) < (-w[b], b) for a in kept for b in gone)
    # rows below the budget stay; the others come from behind it, upwards
    moved = [j for i, j in enumerate(src) if j != i]
    assert all(j >= budget for j in moved) and moved == sorted(moved)


def test_evict_hand_case_order_and_nan():
    w = [5.0, math.nan, 1.0, 7.0, 1.0, -math.inf, 0.0, -0.0]
    assert O.evict_reference(w, 8, 4).tolist() == [0, 4, 2, 3]       # 7, 5, then the two ones
    assert O.evict_reference(w, 8, 6).tolist() == [0, 6, 2, 3, 4, 7]  # zeros of either sign tie
    assert O.evict_reference(w, 8, 7).tolist() == [0, 1, 2, 3, 4, 7, 6]  # NaN ties with -inf: lower row
    assert O.evict_reference(w, 3, 4).tolist() == [0, 1, 2]          # nothing to drop
    # ages in any order: row 3 is the oldest token, rows 4 and 5 the newest two
    age = [30, 10, 20, 0, 70, 60, 50, 40]
    assert O.evict_reference(np.zeros(8), 8, 3, sink=1, recent=11, order=age).tolist() == [3, 4, 5]
    # more held rows than the budget: they compete by weight
    assert O.evict_reference([0, 0, 0, 9, 1, 2, 0, 0], 8, 2, sink=0, recent=11, order=age).tolist() == [4, 5]
    assert O.evict_reference([0, 0, 0, 9, 1, 2, 0, 0], 8, 1, sink=0, recent=11, order=age).tolist() == [5]


def test_rotation_with_one_axis_is_the_pinned_rotation():
    rng = np.random.default_rng(1)
    X = rng.standard_normal((7, 16))
    pos = np.array([[0], [5], [3], [3], [100], [2], [9]])
    np.testing.assert_allclose(O.rope_rotate_axes(X, pos, [8]),
                               O.rope_rotate_rows(X, pos[:, 0], O.rope_frequencies(16)), atol=1e-13)


def test_rotation_with_equal_axes_is_the_rotation_with_one():
    rng = np.random.default_rng(2)
    X, p = rng.standard_normal((5, 16)), rng.integers(0, 50, (5, 1))
    np.testing.assert_allclose(O.rope_rotate_axes(X, np.repeat(p, 3, 1), [2, 3, 3]),
                               O.rope_rotate_axes(X, p, [8]), atol=1e-13)


def test_scores_depend_on_position_differences_per_axis():
    rng = np.random.default_rng(3)
    K, q = rng.standard_normal((6, 16)), rng.standard_normal((1, 16))
    pk, pq = rng.integers(0, 30, (6, 2)), rng.integers(0, 30, (1, 2))
    base = O.rope_rotate_axes(q, pq, [3, 5]) @ O.rope_rotate_axes(K, pk, [3, 5]).T
    shift = np.array([[11, 4]])
    moved = O.rope_rotate_axes(q, pq + shift, [3, 5]) @ O.rope_rotate_axes(K, pk + shift, [3, 5]).T
    np.testing.assert_allclose(moved, base, atol=1e-12)
    # a mistake the pin catches: the axes swapped on the keys only
    wrong = O.rope_rotate_axes(q, pq + shift, [3, 5]) @ O.rope_rotate_axes(K, (pk + shift)[:, ::-1], [3, 5]).T
    assert np.max(np.abs(wrong - base)) > 1e-3


def test_decode_with_row_positions_is_the_pinned_rope_decode():
    c = _case()
    args = [c[k] for k in ("q", "k_s", "v_s", "z_k", "z_v", "b_k", "b_v", "seq_lens")]
    pos = np.tile(np.arange(9)[None, :, None], (2, 1, 1))
    out, lse, _ = O.decode_weights_reference(*args, positions=pos, sections=[8])
    ref_o, ref_l = O.decode_reference_rope(*args)
    np.testing.assert_allclose(out, ref_o, atol=1e-12)
    np.testing.assert_allclose(lse, ref_l, atol=1e-12)


def test_decode_does_not_depend_on_the_order_of_the_rows():
    """What eviction relies on: rows permuted with their positions attend alike."""
    c = _case(lens=(9, 9))
    pos = np.random.default_rng(4).integers(0, 40, (2, 9, 3))
    names = ("q", "k_s", "v_s", "z_k", "z_v", "b_k", "b_v", "seq_lens")
    out, lse, fresh = O.decode_weights_reference(*[c[k] for k in names], positions=pos, sections=[2, 3, 3])
    perm = torch.randperm(9, generator=torch.Generator().manual_seed(1))
    d = dict(c, **{k: c[k][:, perm] for k in ("k_s", "v_s", "z_k", "z_v")})
    out2, lse2, fresh2 = O.decode_weights_reference(*[d[k] for k in names], positions=pos[:, perm.numpy()],
                                                    sections=[2, 3, 3])
    np.testing.assert_allclose(out2, out, atol=1e-12)
    np.testing.assert_allclose(lse2, lse, atol=1e-12)
    np.testing.assert_allclose(fresh2[0], fresh[0][perm.numpy()], atol=1e-12)
