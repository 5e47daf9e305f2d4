"""The target's cache where one thread, one row or one page stands beside another: what each
does is its own."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_gpu_r_pages import State  # noqa: E402


@pytest.mark.parametrize("n_pages", [64, 2000, 33_000, 70_001])
def test_compaction_changes_one_word_of_the_bitmap_both_ways(n_pages):
    """The word that the first page behind those in use lies in loses holes below that page and
    gets free pages above it, by two threads of which neither may undo the other's part."""
    rng = np.random.default_rng(n_pages)
    s = State(3, n_pages, 1, 1 << 17)
    words = n_pages // 32
    for _ in range(12):
        word, bit = int(rng.integers(words - 1)) * 32, int(rng.integers(0, 20))
        holes = int(rng.integers(1, 6))
        more = int(rng.integers(holes, 12))  # pages behind the holes: `holes` of them from page live on
        s.reserve([0, 1, 2], [word + bit, holes, more])
        s.commit([0, 1, 2], [word + bit, holes, more])
        s.release([1])
        live = word + bit + more
        assert (s.o.refs[:live] == 0).sum() == holes and (s.o.refs[live:] > 0).sum() == holes
        moves = s.compact(8)
        assert [m for m in moves if m[0] >= 0] == [[live + holes - 1 - i, word + bit + i] for i in range(holes)]
        s.release([0, 2])
