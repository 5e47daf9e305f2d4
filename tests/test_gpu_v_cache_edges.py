"""Attention over the paged cache where its work is cut: every kernel on sequences that are cut
into pieces, over several launches, at the largest numbers of rows and of key-value heads, one slot
named twice, and infinities that pass from a piece to its join."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.cache_util import up  # noqa: E402
from tests.test_gpu_t_attend import Call, _plant, bounds  # noqa: E402


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [48, 64, 128, 256])
@pytest.mark.parametrize("rows,group", [(1, 4), (4, 8), (6, 8), (9, 8), (17, 9)])
def test_every_kernel_on_cut_sequences(rows, group, D, e4m3):
    c = Call(200 + rows, [3000, 1, 700, 0, 2999], rows, kv=1, group=group, D=D, e4m3=e4m3, page=32)
    assert c.bytes > 0
    c.work[:c.bytes] = 0xff  # not a number, as floats
    c.run().check()


@pytest.mark.parametrize("rows,group", [(3, 4), (9, 8)])
def test_cut_sequences_with_a_window_and_fewer_rows(rows, group):
    Call(210, [3000, 900, 2500, 40], rows, kv=3, group=group, D=128, window=1000, last_row=[rows - 1, 0, -1, rows]).run().check()
    Call(211, [3000, 900, 2500, 40], rows, kv=3, group=group, D=64, window=777, packed=True).run().check()


def test_cut_sequences_in_several_launches():
    rng = np.random.default_rng(3)
    c = Call(212, list(rng.integers(0, 1500, 600)), 1, kv=1, group=2, page=64, last_row=list(rng.integers(-1, 1, 600)))
    c.run().check()


def test_the_most_rows():
    c = Call(213, [300, 0], 257, kv=1, group=64, D=16)
    c.run().check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_the_most_heads(e4m3):
    Call(214, [150, 3], 1, kv=1024, group=1, D=16, e4m3=e4m3).run().check()


@pytest.mark.parametrize("D,group", [(64, 4), (128, 12), (256, 8)])
def test_a_slot_named_twice(D, group):
    c = Call(215, [900, 900, 20], 4, group=group, D=D)
    p = c.paged
    p.d["slots"].copy_(up(p.slots[[0, 0, 2]]))
    c.q_dev.view(-1, 4, c.row)[1] = c.q_dev.view(-1, 4, c.row)[0]
    out, lse = c.run().result()
    want, wlse = Call(215, [900, 900, 20], 4, group=group, D=D).run().result()
    assert c.status.item() == 0
    assert np.array_equal(out[:4], want[:4]) and np.array_equal(lse[8:], wlse[8:])
    # the second stands elsewhere in the shares, and may differ from the first in its rounding
    o, l, size, extra = c.want(0)
    tol, ltol = bounds(D, 904, o, l, size, extra)
    assert (np.abs(out[4:8] - o) <= tol).all() and (np.abs(lse[4:8] - l) <= ltol).all()


@pytest.mark.parametrize("D,group,rows", [(64, 2, 6), (128, 4, 6), (128, 20, 6), (256, 16, 6)])
def test_an_infinity_in_a_piece_reaches_the_rows_that_see_it(D, group, rows):
    length = 3000
    kind = dict(D=D, group=group, page=32)
    clean = Call(216, [length, 70], rows, **kind).run().check()
    c = Call(216, [length, 70], rows, **kind)
    _plant(c, 1, [length + 2], float("inf"))
    out, lse = c.run().result()
    assert c.status.item() == 0
    assert np.array_equal(lse, clean[1])
    out, was = (x.reshape(2, rows, -1, D) for x in (out, clean[0]))
    assert np.array_equal(out[1], was[1]) and np.array_equal(out[0, :2], was[0, :2])
    assert np.isposinf(out[0, 2:, :group]).all() and np.array_equal(out[0, 2:, group:], was[0, 2:, group:])


def test_graphs_of_cut_sequences_replayed_between_eager_calls():
    c = Call(217, [3000, 100, 1700], 5, group=8, D=128, e4m3=True)
    want = c.run().result()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    other = Call(218, [50, 2000], 5, group=8, D=128, e4m3=True)
    for _ in range(3):
        c.out.fill_(7.0), c.lse.fill_(7.0), c.work[:c.bytes].fill_(0xff)
        g.replay()
        other.run().check()
        got = c.result()
        assert all(np.array_equal(a, b) for a, b in zip(got, want))


def test_shorter_lengths_than_when_captured():
    """A graph is of a bound, not of lengths: these are read when it runs."""
    c = Call(219, [3000, 100, 1700], 3, group=4, D=64)
    g = torch.cuda.CUDAGraph()
    c.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.run()
    p = c.paged
    for lengths in ([10, 0, 900], [2999, 100, 1]):
        p.lengths[p.slots] = lengths
        p.d["lengths"].copy_(up(p.lengths))
        c.out.fill_(7.0), c.lse.fill_(7.0)
        g.replay()
        c.check()
