"""The fp64 rules, history and 4-bit decoding against hand-made values, and the
argument checks of the calls (host only, no GPU)."""
import os

import numpy as np
import pytest

from oracle import rules as R

FAKE = 1 << 40  # an address that is never dereferenced: checks are host-only


@pytest.fixture(scope="module")
def B():
    from draft_verification_amd import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding


def test_bits_and_words_are_inverse():
    rng = np.random.default_rng(0)
    for V in (1, 31, 32, 33, 100):
        f = rng.random(V) < 0.5
        w = R.words(f)
        assert w.shape == ((V + 31) // 32,)
        assert np.array_equal(R.bits(w, V), f)
        assert all((int(w[v // 32]) >> (v % 32) & 1) == f[v] for v in range(V))


def test_process_row_by_hand():
    l = np.array([2.0, -2.0, 1.0, 0.0, 3.0])
    counts = np.array([2, 0, 7, 0, 0])
    seen = np.array([True, True, False, False, False])   # the 7 of an unseen token does not count
    allowed = np.array([True, True, True, True, False])
    out, live, _ = R.process_row(l, [0, 3], counts, seen, 2.0, 0.5, 0.25, [(1, 1.0), (1, 0.5), (9, 4.0)], allowed)
    assert np.array_equal(out, [2 / 2 - 0.5 * 3 - 0.25, -4 + 1.5, 1.0, 0 - 0.5 - 0.25, -np.inf])
    assert live == 4
    out, live, _ = R.process_row(l, [], None, None, 1.0, 0.5, 0.25, [], None)
    assert np.array_equal(out, l) and live == -1


def test_history_by_hand():
    counts, seen = np.zeros((2, 4), int), np.zeros((2, 4), bool)
    counts[0] = 9
    R.history_update(counts, seen, [(0, [1, 1, -1, 3], 1), (0, [1], 0), (-1, [2], 1)], True)
    assert counts.tolist() == [[0, 3, 0, 1], [0, 0, 0, 0]]
    assert seen.tolist() == [[False, True, False, True], [False] * 4]


def test_head_weights_by_hand():
    w = R.head_weights(np.array([[0x71, 0x9f]], np.uint8), np.array([[2.0]]), True, 4)
    assert w.tolist() == [[1.0, 12.0, -12.0, -1.0]]
    w = R.head_weights(np.array([[0x71, 0x9f]], np.uint8), np.array([[2.0, 0.5]]), False, 2)
    assert w.tolist() == [[-14.0, -2.0, 3.5, 0.5]]


# ---------------------------------------------------------------- argument checks

def _process(lib, **kw):
    a = dict(logits_in=FAKE, in_strides=(5000, 1000), logits_out=FAKE + 4096, out_strides=(5000, 1000))
    a.update(kw)
    return lib.make_process_args(a.pop("B", 3), a.pop("rows", 5), **a)


CFG = (8, 8, 1000, 1, 0)
PROCESS_OK = [
    dict(), dict(B=0, logits_in=None), dict(row0=4), dict(in_strides=(0, 1000)), dict(out_strides=(1000, 3000)),
    dict(logits_out=FAKE), dict(draft_tokens=FAKE, draft_stride=4), dict(masks=FAKE, mask_stride=32, n_masks=1, mask_index=FAKE),
    dict(history_counts=FAKE, history_seen=FAKE, n_slots=3), dict(history_counts=FAKE, history_seen=FAKE, n_slots=1, slots=FAKE),
    dict(bias_offsets=FAKE), dict(row_offsets=FAKE, in_strides=(-1, 1000), out_strides=(-1, 1000)),
    dict(rows=1, out_strides=(1000, 1000)),
]
PROCESS_BAD = [
    dict(B=-1), dict(B=9), dict(rows=0), dict(row0=-1), dict(row0=5), dict(logits_in=None), dict(logits_out=None),
    dict(in_strides=(5000, 999)), dict(out_strides=(5000, 999)), dict(in_strides=(-5000, 1000)),
    dict(out_strides=(-5000, 1000)), dict(out_strides=(0, 1000)), dict(out_strides=(4999, 1000)),
    dict(out_strides=(1000, 2999)), dict(logits_out=FAKE, out_strides=(6000, 1000)),
    dict(logits_out=FAKE, out_strides=(5500, 1100)), dict(row_offsets=FAKE, verify_len=FAKE),
    dict(draft_tokens=FAKE, draft_stride=3), dict(history_counts=FAKE, n_slots=3), dict(history_seen=FAKE, n_slots=3),
    dict(history_counts=FAKE, history_seen=FAKE, n_slots=2), dict(history_counts=FAKE, history_seen=FAKE, n_slots=0, slots=FAKE),
    dict(bias_offsets=FAKE, n_biases=2), dict(bias_offsets=FAKE, n_biases=2, bias_tokens=FAKE), dict(bias_offsets=FAKE, n_biases=-1),
    dict(masks=FAKE, mask_stride=31, n_masks=1, mask_index=FAKE), dict(masks=FAKE, mask_stride=32, n_masks=0, mask_index=FAKE),
    dict(masks=FAKE, mask_stride=32, n_masks=1),
]


@pytest.mark.parametrize("kw", PROCESS_OK)
def test_process_check_accepts(B, kw):
    assert B.process_check(B.Config(*CFG), _process(B, **kw)) == B.SV_OK


@pytest.mark.parametrize("kw", PROCESS_BAD)
def test_process_check_rejects(B, kw):
    assert B.process_check(B.Config(*CFG), _process(B, **kw)) == B.SV_EINVAL


def _history(lib, **kw):
    a = dict(tokens=FAKE, max_tokens=9, token_stride=9, kind=0, counts=FAKE, seen=FAKE, n_slots=3)
    a.update(kw)
    return lib.make_history_args(a.pop("B", 3), **a)


@pytest.mark.parametrize("kw", [dict(), dict(B=0, counts=None), dict(max_tokens=0, tokens=None), dict(n_slots=1, slots=FAKE),
                                dict(token_offsets=FAKE, n_tokens=0, token_stride=0), dict(kind=1, reset=FAKE, lengths=FAKE)])
def test_history_check_accepts(B, kw):
    assert B.history_check(B.Config(*CFG), _history(B, **kw)) == B.SV_OK


@pytest.mark.parametrize("kw", [dict(B=-1), dict(B=9), dict(max_tokens=-1), dict(kind=2), dict(counts=None), dict(seen=None),
                                dict(n_slots=0, slots=FAKE), dict(n_slots=2), dict(tokens=None), dict(token_stride=8),
                                dict(token_offsets=FAKE, lengths=FAKE), dict(token_offsets=FAKE, n_tokens=-1)])
def test_history_check_rejects(B, kw):
    assert B.history_check(B.Config(*CFG), _history(B, **kw)) == B.SV_EINVAL


def test_history_check_refuses_lists_past_the_limit(B):
    n = B.SV_MAX_HISTORY_TOKENS
    for most, rc in ((n, B.SV_OK), (n + 1, B.SV_EUNSUPPORTED), (2 ** 31 - 1, B.SV_EUNSUPPORTED)):
        assert B.history_check(B.Config(*CFG), _history(B, max_tokens=most, token_stride=2 ** 31)) == rc


def _head(B, **kw):
    a = dict(rows=72, hidden=256, format=1, group=64, packed=FAKE, hidden_states=FAKE, hidden_stride=256, logits=FAKE,
             logits_stride=1000)
    a.update(kw)
    return B.make_head_args(a.pop("rows"), **a)


def _pack(B, **kw):
    a = dict(hidden=256, format=1, group=64, weights=FAKE, weight_stride=128, scales=FAKE, scale_stride=4, packed=FAKE)
    a.update(kw)
    return B.make_head_pack_args(**a)


WEIGHTS_BAD = [
    (dict(hidden=0), "SV_EINVAL"), (dict(hidden=-64), "SV_EINVAL"), (dict(hidden=96), "SV_EINVAL"),
    (dict(hidden=65536 + 64), "SV_EINVAL"), (dict(format=2), "SV_EUNSUPPORTED"), (dict(group=16), "SV_EUNSUPPORTED"),
    (dict(format=0), "SV_EUNSUPPORTED"), (dict(packed=None), "SV_EINVAL"), (dict(packed=FAKE + 8), "SV_EINVAL"),
]


@pytest.mark.parametrize("kw,status", WEIGHTS_BAD + [
    (dict(rows=-1), "SV_EINVAL"), (dict(rows=73), "SV_EINVAL"), (dict(hidden_states=None), "SV_EINVAL"),
    (dict(logits=None), "SV_EINVAL"), (dict(hidden_stride=255), "SV_EINVAL"), (dict(logits_stride=999), "SV_EINVAL")])
def test_head_check_rejects(B, kw, status):
    assert B.head_check(B.Config(*CFG), _head(B, **kw)) == getattr(B, status)


@pytest.mark.parametrize("kw,status", WEIGHTS_BAD + [
    (dict(weights=None), "SV_EINVAL"), (dict(scales=None), "SV_EINVAL"), (dict(weight_stride=127), "SV_EINVAL"),
    (dict(scale_stride=3), "SV_EINVAL")])
def test_head_pack_check_rejects(B, kw, status):
    assert B.head_pack_check(B.Config(*CFG), _pack(B, **kw)) == getattr(B, status)


def test_head_checks_accept_and_size(B):
    cfg = B.Config(*CFG)
    assert B.head_check(cfg, _head(B)) == B.SV_OK
    assert B.head_check(cfg, _head(B, rows=0, logits=None)) == B.SV_OK
    assert B.head_pack_check(cfg, _pack(B)) == B.SV_OK
    # whole strips and steps: at least the values and their scales
    for fmt, group, es in ((0, 32, 1), (1, 32, 2), (1, 64, 2), (1, 128, 2)):
        for hidden in (group, 3 * group, 4096):
            n = B.head_packed_bytes(cfg, hidden, fmt, group)
            assert n >= 1000 * (hidden // 2 + hidden // group * es)
            assert n <= 1024 * (hidden + 128) * (0.5 + es / group)
    with pytest.raises(B.SpecVerifyError):
        B.head_packed_bytes(cfg, 100, 1, 64)


def test_bad_configuration_is_rejected_by_every_check(B):
    cfg = B.Config(4, 4, 0, 1, 0)
    for check, a in ((B.process_check, _process(B)), (B.history_check, _history(B)), (B.head_check, _head(B)),
                     (B.head_pack_check, _pack(B))):
        assert check(cfg, a) == B.SV_EINVAL
