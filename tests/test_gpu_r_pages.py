"""The cache's pages against the oracle that does one sequence and one page after
the other, exactly, and copies of pages."""
import numpy as np
import pytest

from oracle import cache as C

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.cache_util import DEV, lib, up  # noqa: E402


class State:
    """A cache's tables on the GPU and in the oracle."""

    def __init__(self, n_slots, n_pages, page, max_pages, max_batch=None):
        L = self.L = lib()
        self.o = C.Pages(n_slots, n_pages, page, max_pages)
        self.sv = L.SpecVerify(max_batch or max(1, min(n_slots, 4096)), 16, 100, L.SV_BF16)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.guard = 16  # what lies behind the arrays stays

        def array(n):
            return torch.full((n + self.guard,), 0x5a5a5a5a, **i32)
        self.n = [n_slots * max_pages, n_slots, n_slots, n_pages, (n_pages + 31) // 32]
        self.arrays = [array(n) for n in self.n]
        self.cache = L.make_cache(n_slots=n_slots, n_pages=n_pages, page_size=page, max_pages=max_pages,
                                  page_table=self.arrays[0], lengths=self.arrays[1], page_counts=self.arrays[2],
                                  page_refs=self.arrays[3], free_pages=self.arrays[4])
        self.status = torch.full((1,), -5, **i32)
        self.call(0, L.SV_PAGES_CLEAR)
        self.same(0)

    def call(self, B, kind, **more):
        self.status.fill_(-5)
        self.sv.pages(self.L.make_pages_args(B, kind=kind, cache=self.cache, device_status=self.status, **more))

    def push(self):
        """The oracle's state on the GPU."""
        o = self.o
        for a, n, x in zip(self.arrays, self.n, (o.table, o.lengths, o.counts, o.refs, o.free_words().view(np.int32))):
            a[:n].copy_(torch.from_numpy(np.ascontiguousarray(x).reshape(-1).astype(np.int32)))

    def same(self, status):
        torch.cuda.synchronize()
        o = self.o
        names = ("table", "lengths", "counts", "refs", "free")
        want = (o.table, o.lengths, o.counts, o.refs, o.free_words().view(np.int32))
        for name, a, n, x in zip(names, self.arrays, self.n, want):
            got = a.cpu().numpy()
            assert np.array_equal(got[:n], np.ascontiguousarray(x).reshape(-1)), name
            assert (got[n:] == 0x5a5a5a5a).all(), name
        assert self.status.item() == status

    def reserve(self, slots, rows, most=None):
        rows = np.asarray(rows)
        granted = torch.full((len(slots),), 9, dtype=torch.int32, device=DEV)
        self.keep = [up(np.asarray(slots, np.int32)), up((rows - 1).astype(np.int32))]
        self.call(len(slots), self.L.SV_PAGES_RESERVE, slots=self.keep[0], rows=int(rows.max()) if most is None else most,
                  last_row=self.keep[1], granted=granted)
        want, status = self.o.reserve(slots, rows if most is None else np.minimum(rows, most))
        self.same(status)
        assert granted.tolist() == want
        return want

    def commit(self, slots, rows):
        rows = np.asarray(rows)
        self.keep = [up(np.asarray(slots, np.int32)), up((rows - 1).astype(np.int32))]
        self.call(len(slots), self.L.SV_PAGES_COMMIT, slots=self.keep[0], rows=int(rows.max()), last_row=self.keep[1])
        self.same(self.o.commit(slots, rows))

    def release(self, slots):
        self.keep = [up(np.asarray(slots, np.int32))]
        self.call(len(slots), self.L.SV_PAGES_RELEASE, slots=self.keep[0])
        self.same(self.o.release(slots))

    def fork(self, slots, sources):
        granted = torch.full((len(slots),), 9, dtype=torch.int32, device=DEV)
        copies = torch.full((len(slots) + 2, 2), 9, dtype=torch.int32, device=DEV)
        self.keep = [up(np.asarray(slots, np.int32)), up(np.asarray(sources, np.int32))]
        self.call(len(slots), self.L.SV_PAGES_FORK, slots=self.keep[0], from_slots=self.keep[1], granted=granted, copies=copies,
                  max_copies=len(slots) + 2)
        want, moves, status = self.o.fork(slots, sources)
        self.same(status)
        assert granted.tolist() == want and copies[:-2].tolist() == moves and (copies[-2:] == 9).all()
        return want, moves

    def compact(self, most):
        copies = torch.full((most + 1, 2), 9, dtype=torch.int32, device=DEV)
        self.call(0, self.L.SV_PAGES_COMPACT, copies=copies, max_copies=most)
        want = self.o.compact(most)
        self.same(0)
        assert copies[:-1].tolist() == want and (copies[-1] == 9).all()
        return want


@pytest.mark.parametrize("n_slots,n_pages,page,max_pages", [(1, 1, 1, 1), (3, 31, 16, 5), (5, 32, 8, 9), (7, 33, 1024, 4),
                                                            (70, 40000, 16, 700)])
def test_clear(n_slots, n_pages, page, max_pages):
    State(n_slots, n_pages, page, max_pages)


def test_a_step():
    s = State(6, 64, 8, 12)
    slots = [4, 0, 2]
    assert s.reserve(slots, [20, 1, 33]) == [1, 1, 1]
    s.commit(slots, [20, 1, 33])
    for accepted in ([1, 5, 3], [5, 5, 5], [1, 1, 1], [2, 3, 4]):
        s.reserve(slots, [5, 5, 5])
        s.commit(slots, accepted)
    s.release([0])
    s.reserve([1, 4], [9, 30])
    s.commit([1], [0])  # nothing was accepted: all reserved pages go back
    s.release([4, 2, 1])


def test_rows_beyond_the_bound_do_not_count():
    s = State(3, 20, 4, 6)
    s.reserve([1], [10], most=6)


def test_without_slots_and_last_rows():
    s = State(5, 40, 4, 8)
    granted = torch.zeros(5, dtype=torch.int32, device=DEV)
    s.call(5, s.L.SV_PAGES_RESERVE, rows=9, granted=granted)
    want, status = s.o.reserve(range(5), [9] * 5)
    s.same(status)
    assert granted.tolist() == want
    s.call(5, s.L.SV_PAGES_RESERVE, rows=10)
    s.same(s.o.reserve(range(5), [10] * 5)[1])
    s.call(4, s.L.SV_PAGES_COMMIT, rows=3)
    s.same(s.o.commit(range(4), [3] * 4))
    s.call(3, s.L.SV_PAGES_RELEASE)
    s.same(s.o.release(range(3)))


def test_pages_run_out():
    s = State(6, 10, 4, 10)
    # the third does not fit, nor the fifth behind it, the fourth needs nothing
    assert s.reserve([0, 1, 2, 3, 4], [16, 9, 17, 0, 1]) == [1, 1, 0, 1, 0]
    s.commit([0, 1], [16, 9])
    assert s.reserve([2], [12]) == [1]
    assert s.reserve([4], [1]) == [0]
    s.release([1])
    assert s.reserve([4, 5], [4, 9]) == [1, 0]


def test_a_request_for_more_than_the_pool():
    s = State(300, 64, 1, 1 << 20)
    assert s.reserve(list(range(5)), [60, 1 << 20, 1 << 20, 4, 0]) == [1, 0, 0, 0, 1]
    # sums beyond 32 bits
    assert s.reserve(list(range(100, 300)), [1 << 20] * 200) == [0] * 200


def test_bad_sequences():
    s = State(8, 64, 4, 6)
    s.reserve([0, 1, 2, 3], [10, 9, 8, 7])
    s.commit([0, 1, 2, 3], [10, 9, 8, 7])
    assert s.reserve([0, 1, 0, 8, -1, -2, 4], [9, 5, 9, 1, 1, 1, 1]) == [0, 1, 0, 0, 0, 0, 1]  # 0 is named twice
    assert s.reserve([5], [25]) == [0]          # more than a table holds
    assert s.reserve([5, 6], [-1, 4]) == [0, 1]  # a last row below -1
    s.commit([0, 1, 1, 2, -1, 9], [1, 1, 1, 20, 1, 1])
    s.release([3, 3, 0, -1, 100])
    s.o.lengths[2], s.o.counts[1] = -5, 7        # what no call leaves
    s.push()
    assert s.reserve([1, 2], [1, 1]) == [0, 0]
    s.commit([1, 2], [1, 1])


def test_fork():
    s = State(12, 64, 8, 6)
    s.reserve([0, 1, 2], [20, 16, 3])
    s.commit([0, 1, 2], [20, 16, 3])
    s.reserve([0], [17])  # pages behind the length are not shared
    granted, copies = s.fork([3, 4, 5, 6, 7], [0, 0, 1, 2, 8])  # 8 is empty
    assert granted == [1] * 5 and copies[2] == copies[4] == [-1, -1] and copies[0][0] == copies[1][0]
    s.reserve([3, 4, 5, 6, 7], [5] * 5)
    s.commit([3, 4, 5, 6, 7], [5, 1, 3, 2, 4])
    s.release([0, 3])  # what 4 shares stays
    s.fork([0, 3], [4, 4])
    s.release([4, 0, 3, 1, 5])


def test_bad_forks():
    s = State(12, 12, 8, 6)
    s.reserve([0, 1], [20, 16])
    s.commit([0, 1], [20, 16])
    assert s.fork([2, 2], [0, 0])[0] == [0, 0]                 # filled twice
    assert s.fork([2, 3], [0, 2])[0] == [0, 0]                 # a source that is filled by the same call
    assert s.fork([2], [2])[0] == [0]
    assert s.fork([1, 2, 3, -1, 12, 4], [0, 12, -1, 0, 0, 1])[0] == [0] * 6  # (1 is to be filled, if in vain)
    assert s.fork([5, 6, 7, 8, 9, 10, 11, 2], [0] * 8)[0] == [1, 1, 1, 1, 1, 1, 1, 0]  # pages run out
    s.o.table[0, 2] = 12                                        # a last page that is none
    s.push()
    got = torch.zeros(1, dtype=torch.int32, device=DEV)
    copies = torch.zeros((1, 2), dtype=torch.int32, device=DEV)
    a = [up(np.array([2], np.int32)), up(np.array([0], np.int32))]
    s.call(1, s.L.SV_PAGES_FORK, slots=a[0], from_slots=a[1], granted=got, copies=copies, max_copies=1)
    s.same(1)
    assert got.item() == 0 and copies.tolist() == [[-1, -1]]


def _busy(seed, n_slots, n_pages, page, max_pages, steps):
    """A server's hour in short."""
    rng = np.random.default_rng(seed)
    s = State(n_slots, n_pages, page, max_pages)
    for _ in range(steps):
        live = [i for i in range(n_slots) if s.o.counts[i]]
        empty = [i for i in range(n_slots) if not s.o.counts[i]]
        kind = rng.integers(6)
        if kind == 0 and empty:
            new = list(rng.permutation(empty)[:rng.integers(1, len(empty) + 1)])
            n = rng.integers(1, page * max_pages // 2 + 1, len(new))
            ok = np.array(s.reserve(new, n))
            s.commit(new, np.where(ok, n, 0))
        elif kind == 1 and live:
            s.release(list(rng.permutation(live)[:rng.integers(1, len(live) + 1)]))
        elif kind == 2 and live and empty:
            new = list(rng.permutation(empty)[:rng.integers(1, len(empty) + 1)])
            s.fork(new, list(rng.choice(live, len(new))))
        elif kind == 3:
            s.compact(int(rng.integers(0, n_pages)))
        elif live:
            some = list(rng.permutation(live))
            n = rng.integers(1, 6, len(some))
            ok = np.array(s.reserve(some, n))
            s.commit(some, np.where(ok, rng.integers(0, n + 1), 0))
    return s


@pytest.mark.parametrize("seed,sizes", [(0, (6, 40, 4, 20)), (1, (40, 300, 16, 30)), (2, (9, 33, 1, 40)), (3, (100, 4000, 8, 90))])
def test_busy(seed, sizes):
    _busy(seed, *sizes, steps=40)


def test_many_pages_and_sequences():
    # several tiles of the bitmap, sequences that begin in one and end in another
    s = State(600, 200_000, 16, 1100)
    rng = np.random.default_rng(5)
    slots = list(rng.permutation(600)[:300])
    s.reserve(slots, rng.integers(1, 16000, 300))
    s.commit(slots, [0] * 300)
    n = rng.integers(1, 10000, 300)
    s.reserve(slots, n)
    s.commit(slots, n)
    s.release(slots[::3])
    s.compact(5000)
    s.compact(200_000)
    s.reserve(slots[::3], rng.integers(1, 16000, 100))


@pytest.mark.parametrize("n_pages", [70_000, 98_304, 150_001])
def test_more_pages_than_one_workgroup_hands_out(n_pages):
    # whole tiles of the bitmap and a part of one, requests that fit, that just fit and that do not
    s = State(400, n_pages, 4, 400)
    rng = np.random.default_rng(n_pages)
    slots = list(rng.permutation(400)[:300])
    s.reserve(slots[:50], rng.integers(1, 1600, 50))
    s.release(slots[:50:2])  # holes
    granted = s.reserve(slots, rng.integers(900, 1601, 300))
    assert 0 in granted if n_pages < 90_000 else 1 in granted
    s.commit(slots, [1] * 300)
    s.release(slots[:250])
    s.reserve(slots[:250] + slots[:3], [1600] * 253)  # three are named twice


def test_the_largest_batch():
    s = State(4096, 9000, 4, 4)
    rng = np.random.default_rng(6)
    slots = list(rng.permutation(4096))
    granted = torch.zeros(4096, dtype=torch.int32, device=DEV)
    rows = rng.integers(1, 13, 4096)
    a = [up(np.asarray(slots, np.int32)), up((rows - 1).astype(np.int32))]
    s.call(4096, s.L.SV_PAGES_RESERVE, slots=a[0], rows=12, last_row=a[1], granted=granted)
    # (the oracle's way, with sums)
    need = -(-rows // 4)
    upto = need.cumsum()
    want = upto <= 9000
    torch.cuda.synchronize()
    assert s.status.item() == (0 if want.all() else 4)
    assert np.array_equal(granted.cpu().numpy(), want.astype(int))
    table = s.arrays[0][:s.n[0]].cpu().numpy().reshape(4096, 4)
    for b in np.flatnonzero(want)[:-1:97]:
        assert list(table[slots[b]][:need[b]]) == list(range(upto[b] - need[b], upto[b]))
    assert s.arrays[2][:4096].sum().item() == need[want].sum()


def test_compact_moves_as_many_as_it_may():
    s = State(4, 100, 1, 30)
    s.reserve([0, 1, 2], [30, 30, 30])
    s.commit([0, 1, 2], [30, 30, 30])
    s.release([0])
    assert s.compact(0) == []
    assert [m for m in s.compact(4) if m[0] >= 0] == [[89, 0], [88, 1], [87, 2], [86, 3]]
    assert len([m for m in s.compact(50) if m[0] >= 0]) == 26
    assert s.compact(3) == [[-1, -1]] * 3  # nothing is left to do
    assert s.o.free_words()[0] == 0


def test_empty_calls():
    s = State(4, 10, 4, 4)
    for kind in (s.L.SV_PAGES_RESERVE, s.L.SV_PAGES_COMMIT, s.L.SV_PAGES_RELEASE, s.L.SV_PAGES_FORK):
        s.call(0, kind)
        s.same(0)


@pytest.mark.parametrize("page_bytes,page_stride,n_pools", [(16, 16, 1), (32768, 32768, 3), (16400, 16416, 2), (80, 112, 70)])
def test_copies(page_bytes, page_stride, n_pools):
    L = lib()
    n_pages = 50
    rng = np.random.default_rng(3)
    pool_stride = n_pages * page_stride + 48
    data = torch.from_numpy(rng.integers(0, 256, n_pools * pool_stride).astype(np.uint8))
    order = rng.permutation(n_pages)
    pairs = np.stack([order[:20], order[20:40]], 1)
    pairs[1, 1] = pairs[0, 0]  # (not both: this pair is left out)
    pairs[1, 0] = -1
    pairs[4] = [-1, -1]
    pairs[5, 0] = pairs[6, 0]  # one page to two places
    dev, copies = data.to(DEV), up(pairs.astype(np.int32))
    status = torch.full((1,), -5, dtype=torch.int32, device=DEV)
    sv = L.SpecVerify(1, 1, 100, L.SV_BF16)
    args = L.make_pages_copy_args(20, copies=copies, pools=dev, n_pools=n_pools, pool_stride=pool_stride, page_stride=page_stride,
                                  page_bytes=page_bytes, n_pages=n_pages, device_status=status)
    sv.pages_copy(args)
    want = data.clone()
    for i in range(n_pools):
        for a, b in pairs:
            if a >= 0 and b >= 0:
                at = i * pool_stride
                want[at + b * page_stride:at + b * page_stride + page_bytes] = data[at + a * page_stride:at + a * page_stride + page_bytes]
    torch.cuda.synchronize()
    assert torch.equal(dev.cpu(), want) and status.item() == 0
    # pages that there are not are left out
    bad = pairs.copy()
    bad[7, 0], bad[8, 1], bad[9, 0] = n_pages, 1 << 30, -2
    copies.copy_(torch.from_numpy(bad.astype(np.int32)))
    dev.copy_(data)
    sv.pages_copy(args)
    for i in range(n_pools):
        for b in pairs[7:10, 1]:
            at = i * pool_stride + b * page_stride
            want[at:at + page_bytes] = data[at:at + page_bytes]
    torch.cuda.synchronize()
    assert torch.equal(dev.cpu(), want) and status.item() == 1
    args.n_copies = 0
    sv.pages_copy(args)
    assert status.item() == 0
