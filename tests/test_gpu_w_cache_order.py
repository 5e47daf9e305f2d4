"""The target's cache where one thread, one row or one page stands beside another: what each
does is its own."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_gpu_r_pages import State  # noqa: E402
from tests.test_gpu_t_attend import Call, _plant, bounds  # noqa: E402


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


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,group", [(64, 2), (64, 12), (128, 2), (128, 20), (256, 1), (256, 16)])
@pytest.mark.parametrize("length,kv", [(150, 2), (3000, 2), (1400, 64), (1500, 64)])
def test_what_a_row_does_not_see_does_not_move_it(length, kv, D, group, e4m3):
    """Finite keys and values of later rows of the block, and those rows' queries, to the last
    bit: a large score of one row leaves the others' references where they are.  (With many
    key-value heads a piece of a sequence is several tiles for each wavefront.)"""
    rows, row = 6, 3
    c = Call(300, [length, 20], rows, D=D, group=group, e4m3=e4m3, kv=kv)
    p = c.paged
    want, want_lse = c.run().result()
    held = [x.clone() for x in p.pools]
    by = c.q[row:rows, :group].double().numpy().sum(-1) * c.scale * (p.kscale[0] if e4m3 else 1.0)  # the token's score for a key of ones
    key = 448.0 if e4m3 else 40.0
    for which, value in ((0, key), (0, -key), (1, 400.0)):
        out, lse = _plant(c, which, [length + row], value).run().result()
        assert c.status.item() == 0
        assert np.array_equal(out[:row], want[:row]) and np.array_equal(lse[:row], want_lse[:row])
        assert np.array_equal(out[:, group:], want[:, group:]) and np.array_equal(out[rows:], want[rows:])
        if which == 0:  # a score of 16 / log2(e) above a reference moves it
            high = value * by > want_lse[row:rows, :group] + 12.0
            assert (lse[row:rows, :group][high] > want_lse[row:rows, :group][high] + 11.0).all()
        for x, dev, was in zip(p.pools, p.dev, held):
            x.copy_(was), dev.copy_(was)
    c.q_dev.view(-1, c.row)[row:rows] *= 30.0
    out, lse = c.run().result()
    assert np.array_equal(out[:row], want[:row]) and np.array_equal(lse[:row], want_lse[:row])
    assert not np.array_equal(out[row:rows], want[row:rows]) and np.array_equal(out[rows:], want[rows:])


@pytest.mark.parametrize("D,group", [(64, 2), (128, 2), (128, 20), (256, 1), (256, 16)])
@pytest.mark.parametrize("page", [1, 4, 16, 32])
def test_pages_in_front_of_a_window_may_be_gone(page, D, group):
    """A layer with a window needs no page in front of it: that none is named there is no error,
    wherever the window begins within a tile."""
    rows, window = 3, 100
    for length in (110, 131, 147, 1000):
        kind = dict(D=D, group=group, page=page, window=window)
        want, want_lse = Call(310, [length, 40], rows, **kind).run().result()
        c = Call(310, [length, 40], rows, **kind)
        p = c.paged
        first = length + 1 - window  # what row 0 sees first
        p.table[p.slots[0], :first // page] = np.resize([-1, p.n_pages, 1 << 30], first // page)
        p.d["table"].copy_(torch.from_numpy(p.table))
        out, lse = c.run().result()
        assert np.array_equal(out, want) and np.array_equal(lse, want_lse)
        assert c.status.item() == 0
        # one page further is seen
        p.table[p.slots[0], first // page] = -1
        p.d["table"].copy_(torch.from_numpy(p.table))
        c.run().result()
        assert c.status.item() == 1


def _elements(c, which, token, d, what):
    """Puts `what` into channel d of key-value head 0 of one token of sequence 0."""
    p = c.paged
    page = int(p.table[p.slots[0]][token // p.page])
    p.view(p.pools[which])[page, 0, token % p.page, d] = what
    p.dev[which].copy_(p.pools[which])


@pytest.mark.parametrize("what", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("D,group", [(64, 2), (128, 2), (128, 20), (256, 1), (256, 16)])
@pytest.mark.parametrize("length", [90, 700, 3000])
def test_infinite_values_that_are_seen(length, D, group, what):
    """They stay in their element, and none of it is lost: wherever the sequence is cut, in weights
    that are large, small, and far below what fp32 holds."""
    rows, at = 3, 7
    for steep in (0.0, 4.0):  # with 4, scores rise by hundreds: most weights underflow
        c = Call(320, [length, 30], rows, D=D, group=group)
        p = c.paged
        rise = torch.zeros((length + rows, 2, D))
        rise[:, :, 0] = steep * torch.arange(length + rows)[:, None]
        rise[:, :, 1:] = torch.from_numpy(p.exact[0][0]).float()[:, :, 1:]
        p.fill(0, 0, rise.numpy())
        p.dev[0].copy_(p.pools[0])
        c.q[:, :, 0] = 4.0
        c.q_dev.copy_(c.q.reshape(-1).to(c.q_dev))
        want, want_lse = c.run().check()
        held = p.pools[1].clone()
        for token in (0, 40, length // 2, length - 1):
            _elements(c, 1, token, at, what)
            out, lse = c.run().result()
            got = out[:rows, :group, at].copy()
            out[:rows, :group, at] = want[:rows, :group, at]
            assert np.array_equal(out, want) and np.array_equal(lse, want_lse)
            if what != what:
                assert np.isnan(got).all()
            else:
                assert (np.isnan(got) | (got == what)).all()
                if not steep:
                    assert (got == what).all()
            p.pools[1].copy_(held)


@pytest.mark.parametrize("D,group", [(64, 2), (128, 20), (256, 1), (256, 16)])
@pytest.mark.parametrize("length", [90, 3000])
def test_infinite_scores(length, D, group):
    rows = 3
    kind = dict(D=D, group=group)

    def call():
        c = Call(330, [length, 30], rows, **kind)
        c.q[:, :, 0] = 1.0
        c.q_dev.copy_(c.q.reshape(-1).to(c.q_dev))
        return c
    want, want_lse = call().run().check()
    # -infinity: the token is as if it were not there
    c = call()
    gone = np.zeros(length + rows, bool)
    for token in (0, 33, 64, length - 1):
        _elements(c, 0, token, 0, -float("inf"))
        gone[token] = True
    out, lse = c.run().result()
    assert c.status.item() == 0
    o, l, size, extra = c.want(0, gone)
    tol, ltol = bounds(D, length + rows, o, l, size, extra)
    at = np.arange(group)  # heads of key-value head 0
    assert (np.abs(out[:rows] - o) <= tol)[:, at].all() and (np.abs(lse[:rows] - l) <= ltol)[:, at].all()
    assert np.array_equal(out[:, group:], want[:, group:]) and np.array_equal(lse[:, group:], want_lse[:, group:])
    # all of them: as if the row saw nothing
    c = call()
    raw = c.paged.view(c.paged.pools[0])
    raw[torch.from_numpy(c.paged.table[c.paged.slots[0]].astype(np.int64)).clamp(min=0).unique(), 0, :, 0] = -float("inf")
    c.paged.dev[0].copy_(c.paged.pools[0])
    out, lse = c.run().result()
    assert (out[:rows, :group] == 0).all() and (lse[:rows, :group] == -np.inf).all()
    assert np.array_equal(out[:, group:], want[:, group:])
    # +infinity, seen by the last row alone and by all
    for token, first in ((length + rows - 1, rows - 1), (5, 0)):
        c = call()
        _elements(c, 0, token, 0, float("inf"))
        out, lse = c.run().result()
        assert np.isnan(out[first:rows, :group]).all() and np.isnan(lse[first:rows, :group]).all()
        out[first:rows, :group], lse[first:rows, :group] = want[first:rows, :group], want_lse[first:rows, :group]
        assert np.array_equal(out, want) and np.array_equal(lse, want_lse)


@pytest.mark.parametrize("D,group", [(64, 16), (64, 64), (128, 64), (256, 8), (256, 64)])
def test_every_e4m3_code(D, group):
    """A row that sees one token gets that token's values, exactly; with queries of one channel
    each, lse is that channel of the key, within lse's rounding."""
    kv = 256 // group
    c = Call(340, [0], 1, D=D, group=group, kv=kv, e4m3=True, scaled=False, page=1, scale=1.0)
    p = c.paged
    codes = torch.arange(256, dtype=torch.uint8)
    page = int(p.table[p.slots[0]][0])
    # values: all codes, D to a key-value head, over and over
    of_value = codes.repeat(kv * D // 256 + 1)[:kv * D].view(kv, D)
    p.view(p.pools[1].view(torch.uint8))[page, :, 0] = of_value
    # keys: of each key-value head the channels that its queries ask for, all codes in all
    ask = min(group, D)
    of_key = torch.zeros((kv, D), dtype=torch.uint8)
    of_key[:, :ask] = codes.repeat(kv * ask // 256 + 1)[:kv * ask].view(kv, ask)
    of_key[(of_key & 0x7f) == 0x7f] = 0  # (not a number: felt by every query)
    p.view(p.pools[0].view(torch.uint8))[page, :, 0] = of_key
    for dev, pool in zip(p.dev, p.pools):
        dev.copy_(pool)
    c.q.zero_()
    c.q.view(kv, group, D)[:, torch.arange(group), torch.arange(group) % D] = 1.0
    c.q_dev.copy_(c.q.reshape(-1).to(c.q_dev))
    out, lse = c.run().result()
    assert c.status.item() == 0 and kv * ask >= 256 and kv * D >= 256
    value, key = (x.view(torch.float8_e4m3fn).double().numpy() for x in (of_value, of_key))
    assert np.array_equal(out.reshape(kv, group, D), np.broadcast_to(value[:, None], (kv, group, D)), equal_nan=True)
    s = key[:, np.arange(group) % D]
    tol = bounds(D, 1, 0.0, s, np.zeros((kv, group, 1)), (np.abs(s), np.abs(s)))[1]
    assert (np.abs(lse.reshape(kv, group) - s) <= tol).all()
