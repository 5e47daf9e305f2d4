"""Storing keys and values in pages: exactly the rows' values, at exactly their places."""
import numpy as np
import pytest

from oracle import cache as C

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.cache_util import DEV, Paged, bf16, lib, up  # noqa: E402


class Call:
    def __init__(self, seed, lengths, rows, *, row0=0, packed=False, last_row=None, xpad=0, xshift=0, **kind):
        L = lib()
        rng = np.random.default_rng(seed)
        self.B, self.rows, self.row0 = len(lengths), rows, row0
        n = np.full(self.B, rows) if last_row is None else np.minimum(np.asarray(last_row) + 1, rows)
        if packed:
            n = rng.integers(0, rows + 1, self.B)
        self.n, self.lengths = n, np.asarray(lengths)
        totals = np.where(n > 0, self.lengths + row0 + n, self.lengths)
        p = self.paged = Paged(rng, totals, lengths, **kind)
        lines = int(n.sum()) if packed else self.B * rows
        self.first = np.concatenate([[0], np.cumsum(n)])[:-1] if packed else np.arange(self.B) * rows
        head = p.D + xpad
        row = 2 * p.kv * head + xpad
        self.x = bf16(rng.standard_normal((lines, 2, p.kv, p.D)) * rng.choice([1e-4, 1.0, 30.0, 1e4], (lines, 2, p.kv, 1)))
        raw = torch.full((xshift + max(lines, 1) * row,), float("nan"), dtype=torch.bfloat16)
        raw.as_strided((lines, 2, p.kv, p.D), (row, p.kv * head, head, 1), xshift).copy_(self.x)
        self.dev = raw.to(DEV)
        p.to_device()
        self.status = torch.full((1,), -5, dtype=torch.int32, device=DEV)
        self.sv = L.SpecVerify(max(self.B, 1), 4, 100, L.SV_BF16)
        self.keep = [up(np.concatenate([[0], np.cumsum(n)])), None if last_row is None else up(np.asarray(last_row, np.int32))]
        at = self.dev.data_ptr() + 2 * xshift
        self.args = L.make_append_args(self.B, rows, row0=row0, cache=p.cache, kv=p.held, slots=p.d["slots"],
                                       row_offsets=self.keep[0] if packed else None, last_row=self.keep[1], keys=at,
                                       values=at + 2 * p.kv * head, strides=(rows * row, row, head), device_status=self.status)

    def codes(self, x, scale):
        """What is held for x [..., kv, D]: as e4m3's values, or the bf16 values."""
        if not self.paged.e4m3:
            return x.double().numpy()
        s = np.float32(1.0) if scale is None else scale[:, None]
        with np.errstate(all="ignore"):
            return C.e4m3((x.float().numpy() / s).astype(np.float32))  # divided in fp32

    def check(self, skip=(), gone=(), status=0):
        p = self.paged
        self.sv.append(self.args)
        torch.cuda.synchronize()
        assert self.status.item() == status
        for which, scale in ((0, p.kscale), (1, p.vscale)):
            raw = p.pools[which].clone()
            want = raw.double()
            view = p.view(want)
            stored = torch.zeros(want.shape, dtype=torch.bool)
            mark = p.view(stored)
            for b in range(self.B):
                if b in skip:
                    continue
                for r in range(self.n[b]):
                    t = self.lengths[b] + self.row0 + r
                    if (b, t // p.page) in gone:
                        continue
                    page = p.table[p.slots[b], t // p.page]
                    view[page, :, t % p.page] = torch.from_numpy(self.codes(self.x[self.first[b] + r, which], scale))
                    mark[page, :, t % p.page] = True
            got = p.dev[which].cpu()
            bits = torch.uint8 if p.e4m3 else torch.int16
            assert torch.equal(got.view(bits)[~stored], raw.view(bits)[~stored])  # nothing else is written
            assert torch.equal(torch.nan_to_num(got.double()[stored], nan=1e9), torch.nan_to_num(want[stored], nan=1e9))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("by_token", [False, True])
@pytest.mark.parametrize("page", [1, 4, 16, 128])
def test_pages(page, by_token, e4m3):
    Call(page, [0, 1, 17, 130], 5, page=page, by_token=by_token, e4m3=e4m3).check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kv,D", [(1, 16), (3, 80), (8, 128), (5, 256)])
def test_heads(kv, D, e4m3):
    Call(kv, [3, 40], 3, kv=kv, D=D, e4m3=e4m3).check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows(e4m3):
    Call(1, [5], 1, e4m3=e4m3, kv=1).check()
    Call(2, [0, 9], 700, e4m3=e4m3, kv=2, page=32).check()
    Call(3, [0, 9, 100, 31, 2], 40, e4m3=e4m3, packed=True).check()
    Call(4, [0, 9, 100, 31], 6, e4m3=e4m3, row0=3).check()
    Call(5, [0, 9, 100, 31], 6, e4m3=e4m3, last_row=[5, -1, 0, 77]).check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_strides(e4m3):
    Call(6, [0, 9, 100], 4, e4m3=e4m3, pad=16, xpad=3, xshift=1).check()
    Call(7, [0, 9, 100], 4, e4m3=e4m3, pad=32, xpad=8, xshift=8, by_token=True).check()
    Call(8, [0, 9, 100], 4, e4m3=e4m3, scaled=False).check()


def test_every_bf16_value_to_e4m3():
    c = Call(9, [0], 256, kv=1, D=256, e4m3=True, scaled=False, waste=0.0)
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(256, 1, 1, 256)
    c.x = every.expand(256, 2, 1, 256).contiguous()
    c.dev.as_strided((256, 2, 1, 256), (512, 256, 256, 1)).copy_(c.x.to(DEV))
    c.check()


def test_bad_sequences_and_pages():
    for what in ("slot", "length", "short", "last", "offsets", "padded", "page"):
        c = Call(10, [20, 40, 3], 5, last_row=None if what == "offsets" else [4, 4, 4], packed=what == "offsets")
        p = c.paged
        one = int(p.slots[1])
        skip, gone, status = (1,), (), 1
        if what == "slot":
            p.d["slots"][1] = p.n_slots
        elif what == "length":
            p.d["lengths"][one] = -3
        elif what == "short":
            p.d["counts"][one] = 2
        elif what == "last":
            c.keep[1][1] = -2
        elif what == "offsets":
            c.n = np.array([2, 3, 1])
            c.keep[0].copy_(torch.tensor([0, 2, -1, 0]))
            skip = (0, 1, 2)
            c.keep[0].copy_(torch.tensor([-2, 0, 9, 5]))  # before the first, too many, descending
        elif what == "padded":
            p.d["slots"][1] = -1
            status = 0
        else:
            skip, gone = (), ((1, 2),)
            p.d["table"][one, 2] = p.n_pages
        c.check(skip, gone, status)


def test_empty():
    c = Call(11, [20], 5)
    c.args.B = 0
    c.n = np.array([0])
    c.check()
