"""Attention of drafted blocks over the paged cache against fp64.

Tolerance.  With u = 2^-23 (twice the half step of fp32: the matrix core may
truncate), E = the scaled sum of |q k| and S = the largest |s| over the tokens that
a row sees, M = the weighted sum of |v|, T = those tokens:
- a score's products are exact and summed with fewer than D / 32 + 40 additions, so
  it is off by (D / 32 + 40) u E; its scale (three roundings: scale * log2 e, a key
  scale, the product with the score inside one fma) and the subtraction of the
  reference by (3 + 2) u S, since |s - ref| <= 2 S; exp2 by 2 u.  Together a weight
  is off by the relative w = (D / 32 + 40) u E + 5 u S + 2 u.
- rounding a weight to bf16: 2^-8 (half a step).
- sums over tokens: T / 32 + 60 additions at most on a term's way, through the
  splits' join: t = (T / 32 + 60) u each for the weights and for the values, with the
  factors of the joins among them.
- the division, a value's scale and the rounding of the result: 4 u and 2^-8 |out|.
So out is off by M (2^-8 + 2 w + 2 t + 4 u) (1 + 2^-7) + 2^-8 |out|, and
lse by w + t + 4 u |lse| + 4 u (its logarithm)."""
import numpy as np
import pytest

from oracle import cache as C

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.cache_util import DEV, Paged, bf16, lib, up  # noqa: E402

U = 2.0 ** -23


def bounds(D, T, out, lse, size, extra):
    terms, top = extra
    w = (D / 32 + 40) * U * terms + 5 * U * top + 2 * U
    t = (T / 32 + 60) * U
    with np.errstate(invalid="ignore"):
        low = w + t + 4 * U * np.abs(lse) + 4 * U
    return size * (2.0 ** -8 + 2 * w + 2 * t + 4 * U)[..., None] * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(out) + 1e-37, low


class Call:
    """A batch of blocks over a paged cache, its call and the result in fp64."""

    def __init__(self, seed, lengths, rows, *, group=4, kv=2, D=64, page=16, e4m3=False, by_token=False, row0=0, window=0,
                 packed=False, last_row=None, qpad=0, qshift=0, pad=0, scale=None, waste=float("nan"), max_len=None, scaled=True,
                 sharp=1.0, lse=True, counts=True):
        L = lib()
        rng = np.random.default_rng(seed)
        self.B, self.rows, self.group, self.D, self.row0, self.window = len(lengths), rows, group, D, row0, window
        self.heads = kv * group
        n = np.full(self.B, rows) if last_row is None else np.minimum(np.asarray(last_row) + 1, rows)
        if packed:
            n = rng.integers(0, rows + 1, self.B)
        self.n = n
        lengths = np.asarray(lengths)
        totals = np.where(n > 0, lengths + row0 + n, lengths)
        p = self.paged = Paged(rng, totals, lengths, kv=kv, D=D, page=page, e4m3=e4m3, by_token=by_token, pad=pad, waste=waste, scaled=scaled)
        for b in range(self.B):
            p.fill(b, 0, rng.standard_normal((totals[b], kv, D)) * sharp)
            p.fill(b, 1, rng.standard_normal((totals[b], kv, D)) + 0.5)
        self.scale = 1.0 / np.sqrt(D) if scale is None else scale
        lines = int(n.sum()) if packed else self.B * rows
        head = D + qpad
        row = self.heads * head + qpad
        self.q = bf16(rng.standard_normal((lines, self.heads, D)) * 1.5)
        raw = torch.full((qshift + lines * row,), float("nan"), dtype=torch.bfloat16)
        raw.as_strided((lines, self.heads, D), (row, head, 1), qshift).copy_(self.q)
        self.q_dev = raw.to(DEV)
        self.out = torch.full((qshift + max(lines, 1) * row,), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((max(lines, 1), self.heads), 7.0, device=DEV)
        self.status = torch.full((1,), -5, dtype=torch.int32, device=DEV)
        self.lines, self.row, self.head, self.shift, self.packed = lines, row, head, qshift, packed
        off = np.concatenate([[0], np.cumsum(n)])
        self.first = off[:-1] if packed else np.arange(self.B) * rows
        p.to_device()
        self.sv = L.SpecVerify(max(self.B, 1), max(1, row0 + rows - 1), 100, L.SV_BF16)
        self.keep = [up(off), None if last_row is None else up(np.asarray(last_row, np.int32))]
        if not counts:
            p.cache.page_counts = None
        self.args = L.make_attend_args(
            self.B, rows, row0=row0, cache=p.cache, kv=p.held, slots=p.d["slots"], row_offsets=self.keep[0] if packed else None,
            last_row=self.keep[1], heads=self.heads, queries=self.q_dev.data_ptr() + 2 * qshift, query_strides=(rows * row, row, head),
            outputs=self.out.data_ptr() + 2 * qshift, output_strides=(rows * row, row, head), lse=self.lse if lse else None,
            scale=self.scale, window=window, max_len=int(totals.max(initial=1)) if max_len is None else max_len,
            device_status=self.status)
        self.bytes = self.sv.attend_workspace_bytes(self.args)
        self.work = torch.full((self.bytes + 64,), 0x5a, dtype=torch.uint8, device=DEV)
        self.args.workspace, self.args.workspace_bytes = self.work.data_ptr(), self.bytes

    def run(self, stream=None):
        self.sv.attend(self.args, stream)
        return self

    def result(self):
        torch.cuda.synchronize()
        assert (self.work[self.bytes:] == 0x5a).all()
        out = self.out.cpu().as_strided((self.lines, self.heads, self.D), (self.row, self.head, 1), self.shift)
        # what lies between the rows stays
        rest = torch.ones(self.out.numel(), dtype=torch.bool)
        rest.as_strided((self.lines, self.heads, self.D), (self.row, self.head, 1), self.shift).zero_()
        assert (self.out.cpu()[rest] == 7.0).all()
        return out.double().numpy(), self.lse.cpu().double().numpy()

    def want(self, b, gone=None):
        p = self.paged
        q = self.q[self.first[b]:self.first[b] + self.n[b]].double().numpy()
        start = int(p.lengths[p.slots[b]]) + self.row0
        return C.attend(q, p.exact[0][b], p.exact[1][b], start, self.scale, self.window, gone)

    def check(self, skip=(), status=0):
        out, lse = self.result()
        assert self.status.item() == status
        touched = np.zeros(len(out), bool)
        for b in range(self.B):
            if b in skip:
                continue
            at = slice(self.first[b], self.first[b] + self.n[b])
            touched[at] = True
            o, l, size, extra = self.want(b)
            T = int(self.paged.totals[b])
            tol, ltol = bounds(self.D, min(T, self.window + self.rows) if self.window else T, o, l, size, extra)
            off = np.abs(out[at] - o)
            assert (off <= tol).all(), (b, (off / tol).max())
            off = np.abs(lse[at] - l)
            assert (off <= ltol).all(), (b, (off / ltol).max())
        assert (out[~touched] == 7.0).all() and (lse[~touched[:len(lse)]] == 7.0).all()
        return out, lse


@pytest.mark.parametrize("length", [0, 1, 2, 14, 15, 16, 31, 32, 33, 63, 126, 127, 128, 129, 255, 600])
@pytest.mark.parametrize("rows", [1, 5])
def test_lengths(length, rows):
    Call(length, [length], rows).run().check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 128, 144, 192, 256])
def test_head_sizes(D, e4m3):
    Call(D, [200, 3], 2, D=D, e4m3=e4m3, group=3).run().check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,group", [(1, 1), (1, 7), (1, 16), (1, 17), (2, 16), (5, 8), (9, 7), (9, 8), (17, 5), (17, 8), (17, 9), (3, 64)])
def test_rows_and_groups(rows, group, D, e4m3):
    Call(rows * group, [150, 40], rows, group=group, D=D, e4m3=e4m3, kv=1).run().check()


@pytest.mark.parametrize("by_token", [False, True])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 128, 1024])
def test_pages(page, by_token):
    Call(page, [0, 77, 300, 1025], 3, page=page, by_token=by_token, kv=3, D=64, group=2).run().check()


@pytest.mark.parametrize("page,D,e4m3", [(2, 256, True), (8, 128, False), (16, 128, True), (4, 80, True), (64, 256, False)])
def test_pages_of_other_types(page, D, e4m3):
    Call(page, [90, 301], 4, page=page, D=D, e4m3=e4m3, by_token=page < 16).run().check()


@pytest.mark.parametrize("window", [1, 2, 5, 31, 32, 33, 100, 1000])
@pytest.mark.parametrize("rows", [1, 9])
def test_windows(window, rows):
    Call(window, [0, 5, 31, 64, 257, 700], rows, window=window).run().check()


@pytest.mark.parametrize("row0", [1, 7])
def test_drafting_steps(row0):
    Call(row0, [0, 30, 200], 1, row0=row0).run().check()
    Call(row0, [0, 30, 200], 3, row0=row0).run().check()


@pytest.mark.parametrize("kv,group", [(1, 1), (2, 4), (8, 8)])
def test_long_sequences_are_split(kv, group):
    c = Call(5, [5000, 1, 700, 0, 4999], 3, kv=kv, group=group, D=128, page=32)
    assert c.bytes > 0
    c.run().check()


def test_a_long_length_bound_splits_the_same_result():
    a, b = Call(6, [900, 20], 2), Call(6, [900, 20], 2, max_len=0)
    b.args.max_len = 0
    c = Call(6, [900, 20], 2, max_len=900 + 2 + 31)
    for x in (a, b, c):
        x.run().check()


def test_packed_rows():
    for seed in range(3):
        Call(40 + seed, [100, 3, 0, 64, 310, 17], 5, packed=True, group=7).run().check()


def test_last_rows():
    c = Call(50, [100, 3, 0, 64], 5, last_row=[4, -1, 0, 9]).run()
    c.check()


def test_strides_and_alignment():
    Call(60, [100, 33], 3, qpad=5, qshift=3, pad=8).run().check()
    Call(61, [100, 33], 3, qpad=1, qshift=1, pad=16, by_token=True, D=128, e4m3=True).run().check()
    Call(62, [100, 33], 3, qpad=8, qshift=8, pad=24, D=80).run().check()


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30, 1e-42, 3.0])
@pytest.mark.parametrize("e4m3", [False, True])
def test_scales(scale, e4m3):
    Call(70, [100, 33], 3, scale=scale, e4m3=e4m3).run().check()


def test_e4m3_without_scales():
    Call(71, [100, 33], 3, e4m3=True, scaled=False).run().check()


def test_sharp_scores():
    # scores of hundreds: one token takes everything, and the references move often
    Call(72, [1000, 33], 4, D=128, sharp=30.0).run().check()


def test_rising_scores():
    # every tile's scores lie above those before it
    c = Call(73, [2000], 2, D=64, group=2, kv=1)
    p = c.paged
    rise = np.linspace(0.0, 60.0, 2002)
    k = np.zeros((2002, 1, 64))
    k[:, 0, 0] = rise
    c.q[:] = 0.0
    c.q[:, :, 0] = 8.0
    c.q[:, :, 1] = 0.1
    p.fill(0, 0, k)
    p.dev[0].copy_(p.pools[0])
    c.q_dev.as_strided(c.q.shape, (c.row, c.head, 1), c.shift).copy_(c.q.to(DEV))
    c.run().check()


def test_no_lse():
    c = Call(74, [100, 2000], 3, lse=False).run()
    out, lse = c.result()
    assert (lse == 7.0).all()
    o = c.want(1)[0]
    assert np.abs(out[3:] - o).max() < 0.1


def test_without_page_counts():
    Call(75, [100, 33], 3, counts=False).run().check()


def _plant(c, which, tokens, what):
    """Puts `what` into every channel of key-value head 0 of the tokens of sequence 0."""
    p, t = c.paged, torch.tensor(tokens)
    raw = p.view(p.pools[which].view(torch.uint8 if p.e4m3 else torch.int16))
    code = torch.tensor(what).to(p.dtype).view(raw.dtype).item()
    raw[torch.from_numpy(p.table[p.slots[0]].astype(np.int64))[t // p.page], 0, t % p.page] = code
    p.dev[which].copy_(p.pools[which])
    return c


@pytest.mark.parametrize("e4m3,what", [(False, float("nan")), (False, float("inf")), (False, -float("inf")), (True, float("nan"))])
@pytest.mark.parametrize("D,group", [(64, 2), (80, 5), (128, 20), (256, 16)])
@pytest.mark.parametrize("which", [0, 1])
def test_what_is_not_seen_is_not_felt(which, D, group, e4m3, what):
    rows, length, window = 6, 150, 90
    kind = dict(D=D, group=group, e4m3=e4m3)
    # a later row of the block
    want, want_lse = Call(80, [length], rows, **kind).run().check()
    out, lse = _plant(Call(80, [length], rows, **kind), which, [length + 3], what).run().result()
    assert np.array_equal(out[:3], want[:3]) and np.array_equal(lse[:3], want_lse[:3])
    assert np.array_equal(out[:, group:], want[:, group:])  # the other key-value head
    if which == 1:
        got = out[3:, :group]
        assert (np.isnan(got) if what != what else np.isinf(got) & (np.sign(got) == np.sign(what))).all()
        assert np.array_equal(lse, want_lse)
    # tokens before a window; the last of them is seen by rows 0 .. 2
    want, want_lse = Call(80, [length], rows, window=window, **kind).run().check()
    tokens = [0, 10, length - window, length + 3 - window]
    out, lse = _plant(Call(80, [length], rows, window=window, **kind), which, tokens, what).run().result()
    assert np.array_equal(out[3:], want[3:]) and np.array_equal(lse[3:], want_lse[3:])


def test_bad_pages_are_not_seen():
    for D in (64, 128):
        c = Call(90, [300, 60], 3, D=D, group=6)
        p = c.paged
        p.table[p.slots[0], 3] = p.n_pages
        p.table[p.slots[0], 7] = -1
        p.table[p.slots[0], 18] = 1 << 30  # tokens 288 .. 302: the rows' own among them
        c.paged.d["table"].copy_(torch.from_numpy(p.table))
        c.run()
        out, lse = c.result()
        assert c.status.item() == 1
        gone = np.zeros(303, bool)
        for i in (3, 7, 18):
            gone[i * 16:i * 16 + 16] = True
        for b, g in ((0, gone), (1, None)):
            o, l, size, extra = c.want(b, g)
            tol, ltol = bounds(D, 303, o, l, size, extra)
            at = slice(3 * b, 3 * b + 3)
            assert (np.abs(out[at] - o) <= tol).all() and (np.abs(lse[at] - l) <= ltol).all()


def test_a_row_that_sees_nothing():
    c = Call(91, [5, 20], 2)
    p = c.paged
    p.table[p.slots[0]] = -1
    p.d["table"].copy_(torch.from_numpy(p.table))
    out, lse = c.run().result()
    assert c.status.item() == 1
    assert (out[:2] == 0).all() and (lse[:2] == -np.inf).all()
    # split over the length as well
    c = Call(91, [2000, 20], 2)
    p = c.paged
    p.table[p.slots[0]] = -1
    p.d["table"].copy_(torch.from_numpy(p.table))
    out, lse = c.run().result()
    assert c.bytes and (out[:2] == 0).all() and (lse[:2] == -np.inf).all()


@pytest.mark.parametrize("what", ["slot", "length", "short", "bound", "padded", "last"])
def test_bad_sequences_are_left_alone(what):
    c = Call(92, [100, 60, 33], 3, last_row=[2, 2, 2])
    p = c.paged
    status = 1
    if what == "slot":
        p.d["slots"][1] = p.n_slots
    elif what == "length":
        p.d["lengths"][int(p.slots[1])] = -1
    elif what == "short":
        p.d["counts"][int(p.slots[1])] = 3
    elif what == "bound":
        p.d["lengths"][int(p.slots[1])] = 200
        p.d["counts"][int(p.slots[1])] = 1000
        c.args.max_len = 103
    elif what == "last":
        c.keep[1][1] = -2
    else:
        p.d["slots"][1] = -1
        status = 0
    c.run().check(skip=(1,), status=status)


def test_empty_batches():
    c = Call(93, [100], 3)
    c.args.B = 0
    c.run()
    assert c.status.item() == 0
    assert (c.out == 7.0).all()


def test_runs_are_the_same_and_a_large_workspace_will_do():
    c = Call(94, [3000, 100, 7], 9, group=8, D=128).run()
    a = c.result()
    c.out.fill_(7.0)
    big = torch.full((c.bytes + 4096,), 0xff, dtype=torch.uint8, device=DEV)  # NaN in it
    c.args.workspace, c.args.workspace_bytes = big.data_ptr(), big.numel()
    b = c.run().result()
    assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_a_sequence_does_not_feel_the_others():
    a = Call(95, [700, 100, 7], 4, group=8, D=128)
    out, lse = a.run().result()
    for t in a.paged.dev:
        t.view(a.paged.n_pages, -1)[torch.from_numpy(a.paged.table[a.paged.slots[1]][:7].astype(np.int64)).to(DEV)] = float("nan")
    a.out.fill_(7.0)
    o2, l2 = a.run().result()
    keep = np.r_[0:4, 8:12]
    assert np.array_equal(out[keep], o2[keep]) and np.array_equal(lse[keep], l2[keep]) and np.isnan(o2[4:8]).all()
