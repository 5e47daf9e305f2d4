"""The rules on logits, the token history and the 4-bit head in fp64 (numpy),
written from the formulas of include/spec_verify.h.  Used by tests only."""
from __future__ import annotations

import numpy as np

FP4 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def bits(words: np.ndarray, V: int) -> np.ndarray:
    """uint32 words -> the first V bits as bool."""
    w = np.ascontiguousarray(words).view(np.uint8)
    return np.unpackbits(w, bitorder="little")[:V].astype(bool)


def words(flags: np.ndarray) -> np.ndarray:
    """bool [..., V] -> uint32 [..., ceil(V / 32)]."""
    V = flags.shape[-1]
    pad = np.zeros(flags.shape[:-1] + (-V % 32,), bool)
    packed = np.packbits(np.concatenate([flags, pad], -1), axis=-1, bitorder="little")
    return np.ascontiguousarray(packed).view(np.uint32)


def process_row(l, prefix, counts, seen, rep, freq, pres, biases, allowed):
    """One row.  l: fp64 [V]; prefix: the drafted ids before it; counts, seen:
    its history, or None; biases: (id, value) pairs; allowed: bool [V] or None.
    Returns (row, live, size): size bounds what the fp32 arithmetic rounds, the
    sum of the absolute values that enter each token's result."""
    V = l.shape[0]
    c = np.zeros(V) if counts is None else np.where(seen, counts, 0).astype(np.float64)
    s = np.zeros(V, bool) if seen is None else seen.copy()
    for x in prefix:
        if 0 <= x < V:
            c[x] += 1
            s[x] = True
    with np.errstate(all="ignore"):
        l1 = np.where(s, np.where(l > 0, l / rep, l * rep), l)
        out = l1 - (freq * c + pres * (c > 0))
        size = np.abs(l1) + np.abs(freq) * c + np.abs(pres) * (c > 0)
        add = np.zeros(V)
        for v, x in biases:
            if 0 <= v < V:
                add[v] += x
                size[v] += abs(x)
        out = out + add
    if allowed is None:
        return out, -1, size
    out = np.where(allowed, out, -np.inf)
    return out, int((out > -np.inf).sum()), size


def history_update(counts, seen, sequences, output: bool):
    """counts int [slots][V] and seen bool [slots][V], changed in place.
    sequences: (slot, tokens, reset) each; resets come first."""
    for slot, _, reset in sequences:
        if reset and slot >= 0:
            counts[slot] = 0
            seen[slot] = False
    for slot, tokens, _ in sequences:
        if slot < 0:
            continue
        for v in tokens:
            if 0 <= v < counts.shape[1]:
                seen[slot, v] = True
                counts[slot, v] += output


def head_weights(packed_codes: np.ndarray, scales: np.ndarray, fp4: bool, group: int) -> np.ndarray:
    """uint8 [V][H/2] codes and fp64 [V][H/group] scale factors -> fp64 [V][H]."""
    V, half = packed_codes.shape
    code = np.empty((V, 2 * half), np.int64)
    code[:, 0::2] = packed_codes & 15
    code[:, 1::2] = packed_codes >> 4
    value = FP4[code] if fp4 else code - 8.0
    return value * np.repeat(scales, group, axis=1)
