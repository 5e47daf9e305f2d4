"""The paged cache in fp64 (numpy), written from the formulas and rules of
include/spec_verify.h: its pages, the storing of rows, the attention over them.
Used by tests only."""
from __future__ import annotations

import numpy as np


class Pages:
    """Which slot holds which pages, one sequence and one page after the other."""

    def __init__(self, n_slots, n_pages, page_size, max_pages):
        self.page_size, self.max_pages = page_size, max_pages
        self.table = np.full((n_slots, max_pages), -1)
        self.lengths = np.zeros(n_slots, np.int64)
        self.counts = np.zeros(n_slots, np.int64)
        self.refs = np.zeros(n_pages, np.int64)

    def free_words(self):
        bits = np.packbits(self.refs == 0, bitorder="little")
        return np.concatenate([bits, np.zeros(-len(bits) % 4, np.uint8)]).view(np.uint32)

    def _for(self, tokens):
        return -(-int(tokens) // self.page_size)

    def _named(self, slots, sources=()):
        """Which sequences have a slot of their own."""
        n = len(self.lengths)
        names = [s for s in slots if 0 <= s < n]
        return [0 <= s < n and names.count(s) == 1 and s not in sources for s in slots]

    def _sound(self, s):
        """Whether a slot's numbers are ones that a call leaves."""
        return 0 <= self.counts[s] <= self.max_pages and self.lengths[s] >= 0

    def _drop(self, slot, keep):
        for i in range(keep, self.counts[slot]):
            self.refs[self.table[slot, i]] -= 1
            self.table[slot, i] = -1
        self.counts[slot] = keep

    def _give(self, needs):
        """needs: pages of each sequence, or None.  Returns the pages of each, or None."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        asked, out = 0, []
        for need in needs:
            asked += need or 0
            if need is None or (need and asked > len(free)):
                out.append(None)
                continue
            out.append(free[asked - need:asked])
        for pages in out:
            for p in pages or ():
                self.refs[p] = 1
        return out

    def reserve(self, slots, rows):
        """rows: of each sequence.  Returns (granted, status)."""
        fine, needs, status = self._named(slots), [], 0
        for s, n, ok in zip(slots, rows, fine):
            if s == -1:
                needs.append(None)
                continue
            total = self._for(self.lengths[s] + n) if ok and n >= 0 and self._sound(s) else self.max_pages + 1
            if total > self.max_pages:
                status |= 1
                needs.append(None)
            else:
                needs.append(max(0, total - self.counts[s]))
        got = self._give(needs)
        for s, need, pages in zip(slots, needs, got):
            if pages is None:
                status |= 4 if need is not None else 0
                continue
            self.table[s, self.counts[s]:self.counts[s] + len(pages)] = pages
            self.counts[s] += len(pages)
        return [int(p is not None) for p in got], status

    def commit(self, slots, rows):
        status = 0
        for s, n, ok in zip(slots, rows, self._named(slots)):
            if s == -1:
                continue
            if not ok or n < 0 or not self._sound(s) or self._for(self.lengths[s] + n) > self.counts[s]:
                status |= 1
                continue
            self.lengths[s] += n
            self._drop(s, self._for(self.lengths[s]))
        return status

    def release(self, slots):
        status = 0
        for s, ok in zip(slots, self._named(slots)):
            if s == -1:
                continue
            if not ok or not 0 <= self.counts[s] <= self.max_pages:
                status |= 1
                continue
            self.lengths[s] = 0
            self._drop(s, 0)
        return status

    def fork(self, slots, sources):
        """Returns (granted, copies, status)."""
        n = len(self.lengths)
        used = [f for s, f in zip(slots, sources) if s != -1]
        fine, needs, status = self._named(slots, used), [], 0
        for s, f, ok in zip(slots, sources, fine):
            if s == -1:
                needs.append(None)
                continue
            if not ok or not 0 <= f < n or f in slots or self.counts[s] or self.lengths[s] or not self._sound(f) \
                    or self._for(self.lengths[f]) > self.counts[f]:
                status |= 1
                needs.append(None)
                continue
            needs.append(int(self.lengths[f] % self.page_size != 0))
        got, copies = self._give(needs), []
        for s, f, need, pages in zip(slots, sources, needs, got):
            copies.append([-1, -1])
            if pages is None:
                status |= 4 if need is not None else 0
                continue
            full = int(self.lengths[f]) // self.page_size
            self.table[s, :full] = self.table[f, :full]
            for p in self.table[f, :full]:
                self.refs[p] += 1
            if pages:
                self.table[s, full] = pages[0]
                copies[-1] = [int(self.table[f, full]), pages[0]]
            self.counts[s], self.lengths[s] = full + len(pages), self.lengths[f]
        return [int(p is not None) for p in got], copies, status

    def compact(self, most):
        live = int((self.refs > 0).sum())
        holes = [p for p in range(live) if self.refs[p] == 0]
        far = [p for p in range(len(self.refs) - 1, live - 1, -1) if self.refs[p] > 0]
        moves = [list(m) for m in zip(far, holes)][:most]
        to = dict(moves)
        for s in range(len(self.lengths)):
            for i in range(self.counts[s]):
                self.table[s, i] = to.get(self.table[s, i], self.table[s, i])
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        return moves + [[-1, -1]] * (most - len(moves))


def e4m3(y: np.ndarray) -> np.ndarray:
    """The value with 3 bits of fraction and exponents -6 .. 8 nearest to y, ties to
    even; beyond the largest, the largest."""
    y = np.asarray(y, np.float64)
    with np.errstate(invalid="ignore"):
        c = np.where(np.isnan(y), 0, np.clip(y, -448, 448))
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(c), 2.0 ** -6))) - 3)
    return np.where(np.isnan(y), np.nan, np.round(c / step) * step)


def attend(q, k, v, start, scale, window=0, gone=None):
    """One sequence.  q [rows][heads][D]; k, v [tokens][kv][D]; row r at position start + r;
    gone: tokens that are not seen.  Returns (out, lse, size, exponent): size is the
    weighted sum of |v|, exponent bounds what rounds in a row's scores: the largest
    scaled sum of |q k| and the largest |s|, as a pair, over the tokens seen."""
    rows, heads, D = q.shape
    T, kv = k.shape[:2]
    group = heads // kv
    out, lse = np.zeros((rows, heads, D)), np.full((rows, heads), -np.inf)
    size, terms, top = np.zeros((rows, heads, D)), np.zeros((rows, heads)), np.zeros((rows, heads))
    for r in range(rows):
        p = start + r
        low = max(0, p - window + 1) if window else 0
        seen = np.arange(low, p + 1)
        if gone is not None:
            seen = seen[~gone[seen]]
        if not len(seen):
            continue
        for h in range(heads):
            kk, vv, x = k[seen, h // group], v[seen, h // group], q[r, h]
            with np.errstate(all="ignore"):
                s = kk @ x * scale
                m = s.max()
                e = np.exp(s - m)
                w = e / e.sum()
                out[r, h], size[r, h] = w @ vv, w @ np.abs(vv)
                lse[r, h] = m + np.log(e.sum())
                terms[r, h], top[r, h] = abs(scale) * (np.abs(kk) @ np.abs(x)).max(), np.abs(s).max()
    return out, lse, size, (terms, top)
