"""Paged caches on the GPU beside their contents in fp64, for the tests of append and attend."""
import numpy as np
import torch

DEV = "cuda:0"


def lib():
    from draft_verification_amd import binding
    return binding


def up(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


class Paged:
    """A pool of one layer.  totals: tokens of each sequence (its rows among them); every
    place that holds none of them, and whatever lies between the rows, is `waste`."""

    def __init__(self, rng, totals, lengths, *, kv=2, D=64, page=16, e4m3=False, by_token=False, pad=0, waste=float("nan"), extra=3,
                 scaled=True):
        L = lib()
        self.kv, self.D, self.page, self.e4m3, self.by_token = kv, D, page, e4m3, by_token
        totals = np.asarray(totals)
        held = -(-totals // page)
        B = len(totals)
        self.n_pages, self.n_slots, self.max_pages = int(held.sum()) + extra, B + 2, int(held.max(initial=0)) + 2
        order = rng.permutation(self.n_pages)
        self.slots = rng.permutation(self.n_slots)[:B].astype(np.int32)
        self.table = np.full((self.n_slots, self.max_pages), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[self.slots[b], :n] = order[at:at + n]
            at += n
        self.lengths = np.zeros(self.n_slots, np.int32)
        self.lengths[self.slots] = lengths
        self.counts = np.zeros(self.n_slots, np.int32)
        self.counts[self.slots] = held
        W = D + pad
        if by_token:
            self.strides, size = (page * kv * W + pad, W, kv * W), page * kv * W + pad
        else:
            self.strides, size = (kv * page * W + pad, page * W, W), kv * page * W + pad
        self.kscale = ((0.5 + rng.random(kv)) * 0.05).astype(np.float32) if e4m3 and scaled else None
        self.vscale = ((0.5 + rng.random(kv)) * 0.05).astype(np.float32) if e4m3 and scaled else None
        self.dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        self.pools, self.exact = [], []
        for scale in (self.kscale, self.vscale):
            pool = torch.full((self.n_pages, size), waste, dtype=torch.float32).to(self.dtype)
            self.pools.append(pool)
            self.exact.append([None] * B)
        self.totals = totals

    def view(self, pool):
        """[page][head][place][D] of a pool."""
        return pool.as_strided((self.n_pages, self.kv, self.page, self.D), self.strides + (1,))

    def fill(self, b, which, x):
        """Writes tokens 0 .. of sequence b: x [tokens][kv][D]; keeps what they stand for in fp64."""
        scale = (self.kscale, self.vscale)[which]
        s = 1.0 if scale is None else torch.from_numpy(scale)[:, None]
        held = bf16(x) if not self.e4m3 else (torch.from_numpy(np.asarray(x, np.float32)) / s).clamp(-448, 448).to(self.dtype)
        t = np.arange(len(x))
        pages = torch.from_numpy(self.table[self.slots[b]][t // self.page].astype(np.int64))
        raw = self.view(self.pools[which].view(torch.uint8 if self.e4m3 else torch.int16))
        raw[pages, :, torch.from_numpy(t % self.page)] = held.view(raw.dtype)
        self.exact[which][b] = held.double().numpy() * (1.0 if scale is None else scale.astype(np.float64)[:, None])

    def to_device(self):
        L = lib()
        self.dev = [p.to(DEV) for p in self.pools]
        self.d = dict(table=up(self.table), lengths=up(self.lengths), counts=up(self.counts), slots=up(self.slots),
                      kscale=None if self.kscale is None else up(self.kscale), vscale=None if self.vscale is None else up(self.vscale))
        self.cache = L.make_cache(n_slots=self.n_slots, n_pages=self.n_pages, page_size=self.page, max_pages=self.max_pages,
                                  page_table=self.d["table"], lengths=self.d["lengths"], page_counts=self.d["counts"])
        self.held = L.make_kv(kv_heads=self.kv, head_dim=self.D, type=L.SV_KV_E4M3 if self.e4m3 else L.SV_KV_BF16,
                              keys=self.dev[0], values=self.dev[1], strides=self.strides, key_scales=self.d["kscale"],
                              value_scales=self.d["vscale"])
        return self
