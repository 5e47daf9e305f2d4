"""The oracle of the target's cache against values worked out by hand."""
import math

import numpy as np
import pytest

from oracle import cache as C


def test_reserve_gives_the_lowest_free_pages_in_order():
    p = C.Pages(3, 6, 4, 3)
    assert p.reserve([2, 0], [5, 4]) == ([1, 1], 0)
    assert p.table.tolist() == [[2, -1, -1], [-1] * 3, [0, 1, -1]]
    assert p.counts.tolist() == [1, 0, 2] and p.refs.tolist() == [1, 1, 1, 0, 0, 0]
    assert p.free_words().tolist() == [0b111000]
    # what is held already is not given again; a padded sequence gets nothing
    assert p.reserve([2, -1], [8, 4]) == ([1, 0], 0) and p.counts[2] == 2


def test_reserve_until_nothing_is_left():
    p = C.Pages(3, 4, 4, 4)
    # 3 pages, then 2 that are not there; the sums count those, so one page is not given either
    assert p.reserve([0, 1, 2], [12, 8, 1]) == ([1, 0, 0], 4)
    assert p.counts.tolist() == [3, 0, 0]
    # more than a table holds, a slot twice, one outside
    assert p.reserve([0, 0], [1, 1]) == ([0, 0], 1)
    assert p.reserve([1], [17]) == ([0], 1)
    assert p.reserve([3, 1], [1, 1]) == ([0, 1], 1)


def test_commit_keeps_what_was_accepted():
    p = C.Pages(2, 8, 4, 4)
    p.reserve([1], [10])
    assert p.commit([1], [5]) == 0
    assert p.lengths.tolist() == [0, 5] and p.table[1].tolist() == [0, 1, -1, -1]
    assert p.refs.tolist() == [1, 1, 0, 0, 0, 0, 0, 0]
    assert p.commit([1], [4]) == 1 and p.lengths[1] == 5  # 9 tokens need a page that it does not have
    assert p.commit([1], [3]) == 0 and p.counts[1] == 2
    assert p.release([1]) == 0 and p.refs.sum() == 0 and p.lengths[1] == 0


def test_fork_shares_full_pages():
    p = C.Pages(3, 6, 4, 4)
    p.reserve([0], [6])
    p.commit([0], [6])
    assert p.fork([1, 2], [0, 0]) == ([1, 1], [[1, 2], [1, 3]], 0)
    assert p.table.tolist() == [[0, 1, -1, -1], [0, 2, -1, -1], [0, 3, -1, -1]]
    assert p.refs.tolist() == [3, 1, 1, 1, 0, 0] and p.lengths.tolist() == [6, 6, 6]
    assert p.fork([1], [0]) == ([0], [[-1, -1]], 1)  # not empty
    p.release([0])
    assert p.refs.tolist() == [2, 0, 1, 1, 0, 0]


def test_compact_moves_the_highest_to_the_lowest():
    p = C.Pages(2, 8, 1, 4)
    p.reserve([0, 1], [4, 4])
    p.commit([1], [4])
    p.release([0])  # pages 0..3
    assert p.compact(3) == [[7, 0], [6, 1], [5, 2]]
    assert p.table[1].tolist() == [4, 2, 1, 0]
    assert p.compact(3) == [[4, 3], [-1, -1], [-1, -1]]
    assert p.refs.tolist() == [1, 1, 1, 1, 0, 0, 0, 0]


@pytest.mark.parametrize("x,want", [(0.0, 0.0), (448.0, 448.0), (460.0, 448.0), (1e30, 448.0), (-1e30, -448.0), (1.0625, 1.0), (1.1875, 1.25),
                                    (1.07, 1.125), (2.0 ** -9, 2.0 ** -9), (2.0 ** -10, 0.0), (3 * 2.0 ** -10, 2.0 ** -8), (17.0, 16.0),
                                    (19.0, 20.0)])
def test_e4m3(x, want):
    assert C.e4m3(np.array([x]))[0] == want
    assert math.isnan(C.e4m3(np.array([float("nan")]))[0])


def test_attend():
    # two heads on one key-value head; scores of the second row: 0, ln 2, ln 3 and 0, 0, 0
    k = np.array([[[0.0]], [[math.log(2)]], [[math.log(3)]]])
    v = np.array([[[6.0]], [[12.0]], [[-6.0]]])
    q = np.array([[[1.0], [0.0]], [[1.0], [0.0]]])
    out, lse, size, _ = C.attend(q, k, v, 1, 1.0)
    assert np.allclose(out[..., 0], [[30 / 3, 18 / 2], [12 / 6, 12 / 3]])
    assert np.allclose(lse, np.log([[3, 2], [6, 3]]))
    assert np.allclose(size[1, :, 0], [48 / 6, 24 / 3])
    # a window of two, a token that is not seen, and nothing seen
    out, lse, _, _ = C.attend(q, k, v, 1, 1.0, window=2)
    assert np.allclose(out[1, :, 0], [6 / 5, 3])
    out, lse, _, _ = C.attend(q, k, v, 1, 1.0, gone=np.array([True, True, False]))
    assert out[0].tolist() == [[0.0], [0.0]] and np.isneginf(lse[0]).all() and np.allclose(out[1, :, 0], -6)
