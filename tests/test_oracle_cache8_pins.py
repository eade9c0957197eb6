"""Pins of the oracle's 8-bit cache and page functions: every e4m3 number, hand
calculations, invariances, and planted mistakes that the pins catch."""
import math

import numpy as np
import pytest
import torch

from oracle import lrkv_oracle as O


def _all_e4m3():
    """The 256 e4m3 numbers from the format: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    out = []
    for byte in range(256):
        s, e, m = byte >> 7, byte >> 3 & 15, byte & 7
        v = math.nan if e == 15 and m == 7 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out.append(-v if s else v)
    return np.array(out)


def test_e4m3_numbers_round_to_themselves_and_agree_with_the_format():
    v = _all_e4m3()
    torch_v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(v, torch_v)
    np.testing.assert_array_equal(O.e4m3_round(v), v)


def test_e4m3_rounds_to_the_nearest_and_ties_to_even():
    v = np.unique(_all_e4m3()[np.isfinite(_all_e4m3())])
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 8, 4000)])
    got = O.e4m3_round(x)
    near = v[np.abs(x[:, None] - v[None, :]).argmin(axis=1)]
    assert np.all(np.abs(got - x) <= np.abs(near - x))
    # halfway between neighbours: the even mantissa
    np.testing.assert_array_equal(O.e4m3_round([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10]),
                                  [1.0, 1.25, 0.0, 2.0 ** -8])
    np.testing.assert_array_equal(O.e4m3_round([449.0, 1e30, np.inf, -np.inf]), [448, 448, 448, -448])
    assert np.isnan(O.e4m3_round([np.nan]))[0]


def test_the_scale_is_the_smallest_power_of_two_that_holds_the_largest_number():
    for amax, s in [(448.0, 1.0), (448.0001, 2.0), (0.875, 2.0 ** -9), (224.0, 0.5), (1.0, 2.0 ** -8), (0.0, 2.0 ** -126)]:
        assert O.scale_for(amax) == s
        assert amax <= 448 * s and (s == 2.0 ** -126 or amax > 448 * s / 2)


def test_quantize_by_hand():
    """Two rows into an empty block, then a third that needs a larger scale."""
    values, scales = np.zeros((16, 1, 2)), np.full((1, 1), 7.0)
    values, scales = O.quantize_reference(values, scales, [[[0.875, 0.1]], [[-0.5, 0.0]]], 0, 2)
    assert scales[0, 0] == 2.0 ** -9                       # 0.875 = 448 / 512; the 7 was another's
    # 0.1 * 512 = 51.2 -> 52 (steps of 4 from 32 to 64)
    np.testing.assert_array_equal(values[:2, 0], [[448, 52], [-256, 0]])
    values, scales = O.quantize_reference(values, scales, [[[3.0, 0.001]]], 2, 1)
    assert scales[0, 0] == 2.0 ** -7                       # 448 / 128 = 3.5 >= 3
    np.testing.assert_array_equal(values[:3, 0], [[112, 13], [-64, 0], [384, 0.125]])
    values, scales = O.quantize_reference(values, scales, [[[0.25, 0.25]]], 3, 1)
    assert scales[0, 0] == 2.0 ** -7                       # the block keeps its scale
    np.testing.assert_array_equal(values[3, 0], [32, 32])


def test_quantize_is_off_by_a_sixteenth_at_most_and_row_by_row_equals_at_once_where_no_scale_grows():
    rng = np.random.default_rng(1)
    rows = rng.standard_normal((37, 3, 8))
    rows[0] = 30.0                                          # the first row of a block is its largest
    rows[16] = rows[32] = 30.0
    at_once = O.quantize_reference(np.zeros((48, 3, 8)), np.zeros((3, 3)), rows, 0, 37)
    v, s = np.zeros((48, 3, 8)), np.zeros((3, 3))
    for t in range(37):
        v, s = O.quantize_reference(v, s, rows[t:t + 1], t, 1)
    np.testing.assert_array_equal(v, at_once[0])
    np.testing.assert_array_equal(s, at_once[1])
    back = O.cache8_rows(*at_once)[:37]
    assert np.all(np.abs(back - rows) <= np.maximum(np.abs(rows) / 16, s.max() * 2.0 ** -10))


def test_special_values():
    v, s = O.quantize_reference(np.zeros((16, 1, 4)), np.zeros((1, 1)), [[[np.inf, np.nan, 1.0, -np.inf]]], 0, 1)
    assert s[0, 0] == 2.0 ** -8
    np.testing.assert_array_equal(v[0, 0, [0, 2, 3]], [448, 256, -448])
    assert np.isnan(v[0, 0, 1])


def test_planted_quantize_mistakes_are_caught():
    rows = np.array([[[0.875, 0.1]], [[-0.5, 0.0]]])
    good = O.quantize_reference(np.zeros((16, 1, 2)), np.full((1, 1), 7.0), rows, 0, 2)
    kept = np.maximum(7.0, good[1])                         # a stale scale of an empty block taken over
    assert kept[0, 0] != good[1][0, 0]
    floor = np.floor(rows[:, 0] / good[1][0, 0] / 4) * 4    # truncation instead of rounding
    assert not np.array_equal(floor, good[0][:2, 0])


def test_fork_by_hand():
    table = np.array([[0, 1, -1], [0, 2, 3], [4, -1, -1]])
    refs = np.array([2, 1, 1, 1, 1, 0, 1])                  # page 6 is held outside the tables
    t, l, r = O.pages_fork_reference(table, [20, 40, 5], refs, 16, [1, 1, -1], [33, 16, 9])
    np.testing.assert_array_equal(t, [[0, 2, 3], [0, -1, -1], [-1, -1, -1]])
    np.testing.assert_array_equal(l, [33, 16, 0])
    np.testing.assert_array_equal(r, [2, 0, 1, 1, 0, 0, 1])


def test_fork_to_itself_changes_nothing_and_keeps_the_count():
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 65, 6)
    table = np.full((6, 4), -1)
    refs = np.zeros(20, dtype=int)
    for b in range(6):
        table[b, :-(-lens[b] // 16)] = rng.integers(0, 20, -(-lens[b] // 16))
        for p in table[b, :-(-lens[b] // 16)]:
            refs[p] += 1
    t, l, r = O.pages_fork_reference(table, lens, refs, 16, None, None)
    np.testing.assert_array_equal(t, table)
    np.testing.assert_array_equal(l, lens)
    np.testing.assert_array_equal(r, refs)
    t, l, r = O.pages_fork_reference(table, lens, refs, 16, rng.integers(0, 6, 6), None)
    assert r.sum() == (t >= 0).sum()


def test_extend_by_hand():
    # 0 and 1 share page 5's begun rows and both write: 0 copies, 1 keeps; 2 shares page 7 with a held prompt: copies
    table = np.array([[5, -1, -1], [5, -1, -1], [7, -1, -1]])
    refs = np.array([0, 1, 0, 0, 1, 2, 0, 2])
    t, l, r, copies, missing = O.pages_extend_reference(table, [10, 10, 4], refs, 16, [11, 40, 4])
    np.testing.assert_array_equal(t, [[0, -1, -1], [5, 2, 3], [7, -1, -1]])
    np.testing.assert_array_equal(r, [1, 1, 1, 1, 1, 1, 0, 2])
    assert copies == [(5, 0, 10)] and missing == 0
    t, l, r, copies, missing = O.pages_extend_reference(table, [10, 10, 4], refs, 16, [11, 40, 6])
    np.testing.assert_array_equal(t, [[0, -1, -1], [5, 2, 3], [6, -1, -1]])
    np.testing.assert_array_equal(r, [1, 1, 1, 1, 1, 1, 1, 1])
    assert copies == [(5, 0, 10), (7, 6, 4)] and missing == 0
    # a page too few: nothing happens
    refs[2] = 1
    t, l, r, copies, missing = O.pages_extend_reference(table, [10, 10, 4], refs, 16, [11, 40, 6])
    assert missing == 1 and copies == []
    np.testing.assert_array_equal(t, table)
    np.testing.assert_array_equal(r, refs)
    np.testing.assert_array_equal(l, [10, 10, 4])


def test_extend_writes_no_page_that_another_sequence_sees():
    rng = np.random.default_rng(3)
    for _ in range(50):
        B, pages = 6, 60
        table, lens, refs = np.full((B, 5), -1), np.zeros(B, dtype=int), np.zeros(pages, dtype=int)
        lens[0] = rng.integers(1, 60)
        table[0, :-(-lens[0] // 16)] = rng.permutation(pages)[:-(-lens[0] // 16)]
        refs[table[0][table[0] >= 0]] = 1
        table, lens, refs = O.pages_fork_reference(table, lens, refs, 16, rng.integers(-1, 1, B), None)
        new = np.minimum(lens + rng.integers(0, 20, B), 80)
        t, l, r, copies, missing = O.pages_extend_reference(table, lens, refs, 16, new)
        assert missing == 0
        for b in range(B):
            if l[b] > lens[b]:
                for j in range(lens[b] // 16, -(-l[b] // 16)):
                    assert r[t[b, j]] == 1 and (t == t[b, j]).sum() == 1


def test_compact_by_hand():
    table = np.array([[6, 1, -1], [6, 4, 9]])
    refs = np.array([0, 1, 0, 3, 1, 0, 2, 0, 0, 1])
    t, r, moved, live, copies = O.pages_compact_reference(table, [20, 48], refs, 16)
    assert live == 5 and copies == [(6, 0), (9, 2)]
    np.testing.assert_array_equal(moved, [-1, 1, -1, 3, 4, -1, 0, -1, -1, 2])
    np.testing.assert_array_equal(t, [[0, 1, -1], [0, 4, 2]])
    np.testing.assert_array_equal(r, [2, 1, 1, 3, 1, 0, 0, 0, 0, 0])


def test_a_planted_mistake_in_each_page_call_is_caught():
    # the first writer keeps the page instead of the last: another table
    table, refs = np.array([[5, -1], [5, -1]]), np.array([0, 0, 0, 0, 0, 2])
    t = O.pages_extend_reference(table, [3, 3], refs, 16, [4, 4])[0]
    with pytest.raises(AssertionError):
        np.testing.assert_array_equal(t, [[5, -1], [0, -1]])
    # pages moved from the top down instead of in order: another table
    refs = np.array([0, 0, 1, 1])
    t = O.pages_compact_reference(np.array([[2, 3]]), [32], refs, 16)[0]
    with pytest.raises(AssertionError):
        np.testing.assert_array_equal(t, [[1, 0]])
    # references of the entries before the call forgotten
    r = O.pages_fork_reference(np.array([[0, -1]]), [5], np.array([1, 0]), 16, None, [0])[2]
    with pytest.raises(AssertionError):
        np.testing.assert_array_equal(r, [1, 0])
