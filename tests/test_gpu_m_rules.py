"""Penalties, biases and masks on logits, and the token history, against the
fp64 oracle (oracle/rules.py).

Tolerance.  The kernel's fp32 steps for one token are the penalised logit (at
most 2 half steps), frequency * count and the sum with the presence (2), their
subtraction (1) and one addition per bias: fewer than 6 + n roundings, each at
most 2^-24 of the sum of the absolute values involved (R.process_row's size).
The result is rounded once to the logits' type: half a step, 2^-8 of it for
bf16.  Untouched and masked tokens are exact."""
import numpy as np
import pytest

from oracle import rules as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"


def _lib():
    from draft_verification_amd import binding
    return binding


def _bf16(a):
    """fp32 values rounded to bf16 (nearest even), as fp32; and their bits."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.float().numpy(), t.view(torch.int16).numpy()


def _place(rows, shift, bs, rs, V, total):
    """Flat buffer of `total` elements with the rows [B][R][V] at their strides; the rest is 77."""
    flat = torch.full((total,), 77, dtype=torch.float32)
    for b in range(rows.shape[0]):
        for r in range(rows.shape[1]):
            at = shift + b * bs + r * rs
            flat[at:at + V] = torch.from_numpy(rows[b, r])
    return flat


class Case:
    def __init__(self, B=3, rows=2, row0=0, V=1000, dtype="bf16", packed=False, inplace=False, pad=0, shift=0, gap=0,
                 history=50, biases=5, masks=True, live=True, vlen=False, extremes=False, rows_outer=False, seed=1):
        self.__dict__.update(locals())


CASES = [
    Case(),
    Case(B=1, rows=1, V=1), Case(B=2, rows=3, V=7, dtype="f32", history=3), Case(B=1, rows=1, V=129280, row0=5),
    Case(V=2048), Case(V=2049, dtype="f32"), Case(V=4099, pad=3, shift=1, gap=5), Case(V=4099, pad=1, dtype="f32", shift=3),
    Case(V=1000, inplace=True), Case(V=50257, inplace=True, dtype="f32", rows=3), Case(V=333, inplace=True, live=False, pad=2),
    Case(packed=True, rows=4, B=9), Case(packed=True, rows=4, B=5, dtype="f32", inplace=True, V=777),
    Case(vlen=True, rows=5, row0=1, B=12), Case(row0=14, rows=3, B=2), Case(row0=100, rows=30, B=2, V=3001),
    Case(extremes=True), Case(extremes=True, dtype="f32", inplace=True), Case(masks=False, biases=0), Case(history=0, biases=0),
    Case(history=0, masks=False, biases=700, V=900), Case(biases=200, V=100, dtype="f32"), Case(rows_outer=True, rows=3, B=4),
    Case(B=40, rows=17, V=5000, history=3000), Case(rows=17, V=129280, B=2, dtype="f32", history=4000),
]


def build(c):
    """The call's inputs on the host, and the oracle's outputs."""
    rng = np.random.default_rng(c.seed)
    B, rows, V = c.B, c.rows, c.V
    p = {"c": c}
    l = (3 * rng.standard_normal((B, rows, V))).astype(np.float32)
    if c.extremes:
        for x in (np.inf, -np.inf, np.nan, 0.0, -3.3e38, 3.3e38):
            l[rng.random(l.shape) < 0.05] = x
    if c.dtype == "bf16":
        l = _bf16(l)[0]
    p["l"] = l
    n = np.full(B, rows)
    if c.packed:
        n = rng.integers(0, rows + 1, B)
    if c.vlen:
        L = rng.integers(0, rows + c.row0 + 3, B).astype(np.int32)
        p["vlen"] = L
        n = np.clip(L - c.row0 + 1, 0, rows)
    p["n"] = n
    n_slots = B + 2
    p["slots"] = rng.permutation(n_slots)[:B].astype(np.int32)
    if B > 1:
        p["slots"][B - 1] = -1
    p["counts"], seen = np.zeros((n_slots, V), np.int32), np.zeros((n_slots, V), bool)
    for s in range(n_slots):
        t = rng.integers(0, V, c.history)
        seen[s, t] = True
        np.add.at(p["counts"][s], t[::2], 1)
    p["seen_flags"], p["seen"] = seen, R.words(seen)
    K = c.row0 + rows - 1
    p["draft"] = rng.integers(0, V, (B, max(K, 1) + 1)).astype(np.int32)
    if K > 2:
        p["draft"][:, 2] = p["draft"][:, 0]  # the same id twice in a prefix
    p["rep"] = (0.6 + rng.random(B)).astype(np.float32)
    p["freq"] = (rng.random(B) - 0.3).astype(np.float32)
    p["pres"] = (rng.random(B) - 0.3).astype(np.float32)
    nb = rng.integers(0, c.biases + 1, B)
    p["boff"] = np.concatenate([[0], np.cumsum(nb)]).astype(np.int32)
    p["btok"] = rng.integers(0, V, p["boff"][-1]).astype(np.int32)
    p["bval"] = (2 * rng.standard_normal(p["boff"][-1])).astype(np.float32)
    if p["boff"][-1] > 2:
        p["btok"][1] = p["btok"][0]
        p["bval"][2] = -np.inf  # a banned token
    n_masks = 4
    flags = rng.random((n_masks, V)) < np.array([0.9, 0.02, 0.5, 0.0])[:, None]
    p["mask_flags"], p["masks"] = flags, R.words(flags)
    p["midx"] = rng.integers(-1, n_masks, (B, rows)).astype(np.int32)
    out, live, tol = l.astype(np.float64), np.full((B, rows), -1, np.int32), np.zeros((B, rows, V))
    for b in range(B):
        s = p["slots"][b]
        bias = list(zip(p["btok"][p["boff"][b]:p["boff"][b + 1]], p["bval"][p["boff"][b]:p["boff"][b + 1]].astype(float)))
        for r in range(n[b]):
            m = p["midx"][b, r] if c.masks else -1
            o, live[b, r], size = R.process_row(
                l[b, r].astype(np.float64), p["draft"][b, :c.row0 + r], p["counts"][s] if s >= 0 else None,
                seen[s] if s >= 0 else None, float(p["rep"][b]), float(p["freq"][b]), float(p["pres"][b]), bias,
                flags[m] if m >= 0 else None)
            out[b, r] = o
            same = (o == l[b, r]) | ~np.isfinite(o)
            with np.errstate(invalid="ignore", over="ignore"):
                tol[b, r] = np.where(same & (size == np.abs(l[b, r])), 0.0,
                                     (6 + nb[b]) * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(o) if c.dtype == "bf16" else 0.0))
    p.update(out=out, live=live, tol=tol)
    return p


def call(p, **change):
    """Uploads p and makes the call; returns (args, tensors)."""
    LB = _lib()
    c = p["c"]
    tdt = torch.bfloat16 if c.dtype == "bf16" else torch.float32
    B, rows, V = c.B, c.rows, c.V
    rs = V + c.pad
    bs = rows * rs + c.gap
    if c.rows_outer:
        rs, bs = c.B * V, V
    t = {}
    if c.packed:
        off = np.concatenate([[0], np.cumsum(p["n"])]).astype(np.int64)
        flat = torch.full((c.shift + max(int(off[-1]), 1) * rs,), 77.0)
        for b in range(B):
            for r in range(p["n"][b]):
                at = c.shift + int(off[b] + r) * rs
                flat[at:at + V] = torch.from_numpy(p["l"][b, r])
        t["row_offsets"] = torch.from_numpy(off).to(DEV)
    else:
        flat = _place(p["l"], c.shift, bs, rs, V, c.shift + (B * rows * V if c.rows_outer else B * bs))
    t["in"] = flat.to(tdt).to(DEV)
    t["out"] = t["in"] if c.inplace else torch.full_like(t["in"], 55)
    t["live"] = torch.full((B, rows), -9, dtype=torch.int32, device=DEV)
    t["status"] = torch.full((1,), -9, dtype=torch.int32, device=DEV)
    for k in ("slots", "counts", "draft", "rep", "freq", "pres", "boff", "btok", "bval", "midx"):
        t[k] = torch.from_numpy(p[k]).to(DEV)
    for k in ("seen", "masks"):
        t[k] = torch.from_numpy(p[k].view(np.int32)).to(DEV)
    if c.vlen:
        t["vlen"] = torch.from_numpy(p["vlen"]).to(DEV)
    kw = dict(row0=c.row0, logits_in=t["in"][c.shift:], in_strides=(bs, rs), logits_out=t["out"][c.shift:], out_strides=(bs, rs),
              row_offsets=t.get("row_offsets"), verify_len=t.get("vlen"), draft_tokens=t["draft"],
              draft_stride=p["draft"].shape[1], history_counts=t["counts"], history_seen=t["seen"],
              n_slots=p["counts"].shape[0], slots=t["slots"], repetition=t["rep"], frequency=t["freq"], presence=t["pres"],
              bias_offsets=t["boff"], bias_tokens=t["btok"], bias_values=t["bval"], n_biases=p["btok"].size,
              device_status=t["status"])
    if c.masks:
        kw.update(masks=t["masks"], mask_stride=p["masks"].shape[1], n_masks=p["masks"].shape[0], mask_index=t["midx"])
    if c.live:
        kw.update(live_tokens=t["live"])
    kw.update(change)
    sv = LB.SpecVerify(B, max(1, c.row0 + rows - 1), V, LB.SV_BF16 if c.dtype == "bf16" else LB.SV_F32)
    a = LB.make_process_args(B, rows, **kw)
    return sv, a, t, (bs, rs)


def rows_out(p, t, strides):
    """Output rows [B][rows][V] as fp64 (77 where the call has no row), and the mask of elements that belong to no processed row."""
    c = p["c"]
    bs, rs = strides
    flat = t["out"].float().cpu().numpy().astype(np.float64)
    free = np.ones(flat.shape, bool)
    got = np.full((c.B, c.rows, c.V), 77.0)
    off = np.concatenate([[0], np.cumsum(p["n"])])
    for b in range(c.B):
        for r in range(p["n"][b]):
            at = c.shift + (int(off[b] + r) * rs if c.packed else b * bs + r * rs)
            got[b, r] = flat[at:at + c.V]
            free[at:at + c.V] = False
    return got, flat, free


def compare(p, t, strides, untouched):
    got, flat, free = rows_out(p, t, strides)
    c = p["c"]
    assert np.array_equal(flat[free], untouched[free]), "elements outside the processed rows changed"
    for b in range(c.B):
        for r in range(p["n"][b]):
            want, tol, g = p["out"][b, r], p["tol"][b, r], got[b, r]
            top = 3.3895313892515355e38 if c.dtype == "bf16" else 3.4028234663852886e38
            over = np.abs(want) > top  # beyond the type: infinite, or the largest value by rounding
            assert np.array_equal(np.isnan(g), np.isnan(want)), (b, r)
            ok = np.isnan(want) | (g == want) | (over & (np.abs(g) >= top) & (np.sign(g) == np.sign(want)))
            with np.errstate(invalid="ignore"):
                ok |= np.abs(g - want) <= tol
            assert ok.all(), (b, r, np.flatnonzero(~ok)[:5], g[~ok][:5], want[~ok][:5], tol[~ok][:5])


@pytest.mark.parametrize("i", range(len(CASES)))
def test_process_matches_the_oracle(i):
    c = CASES[i]
    print(f"[case] process {i} {({k: v for k, v in c.__dict__.items() if k != 'self'})}", flush=True)
    p = build(c)
    sv, a, t, strides = call(p)
    untouched = t["out"].float().cpu().numpy().astype(np.float64)
    sv.process(a)
    torch.cuda.synchronize()
    assert int(t["status"]) == 0
    compare(p, t, strides, untouched)
    if c.live:
        want = p["live"].copy()
        if c.extremes:
            # the oracle's fp64 holds -3.3e38 * 1.1 = -3.6e38, which both types round to -infinity
            # (their lowest finite value is -3.4e38): count what is in the rows, which compare() has checked
            got = rows_out(p, t, strides)[0]
            want = np.where(want < 0, -1, (got > -np.inf).sum(-1))
        assert np.array_equal(t["live"].cpu().numpy(), want)
    if not c.inplace:  # the same call again, on its own outputs' leftovers: bit for bit the same
        first = t["out"].clone()
        sv.process(a)
        assert torch.equal(first.view(torch.int16), t["out"].view(torch.int16))


def test_masked_and_empty_rows_are_minus_infinity_whatever_the_logits():
    c = Case(B=1, rows=3, V=3001, extremes=True, biases=0, history=0)
    p = build(c)
    p["midx"][:] = [[3, 1, 3]]  # mask 3 allows nothing
    sv, a, t, strides = call(p)
    t["midx"].copy_(torch.from_numpy(p["midx"]))
    sv.process(a)
    got = rows_out(p, t, strides)[0]
    assert (got[0, 0] == -np.inf).all() and (got[0, 2] == -np.inf).all()
    assert (got[0, 1][~p["mask_flags"][1]] == -np.inf).all()
    assert t["live"].cpu().numpy()[0].tolist()[::2] == [0, 0]


def test_one_set_of_rows_shared_by_all_sequences():
    c = Case(B=4, rows=2, V=600)
    p = build(c)
    sv, a, t, strides = call(p)
    a.in_batch_stride = 0
    sv.process(a)
    got = rows_out(p, t, strides)[0]
    shared = build(c)
    shared["l"][:] = p["l"][:1]
    sv2, a2, t2, _ = call(shared)
    sv2.process(a2)
    assert np.array_equal(got, rows_out(shared, t2, strides)[0], equal_nan=True)


def _expect(p, change, b_bad, live=None):
    """Runs p with one device value changed: the status is set, the other sequences' rows are unchanged."""
    sv, a, t, strides = call(p)
    sv.process(a)
    ref = rows_out(p, t, strides)[0]
    sv, a, t, strides = call(p)
    before = t["out"].clone()
    change(t)
    sv.process(a)
    got = rows_out(p, t, strides)[0]
    assert int(t["status"]) == _lib().SV_STATUS_BAD_INPUT
    keep = [b for b in range(p["c"].B) if b != b_bad]
    assert np.array_equal(got[keep], ref[keep], equal_nan=True)
    return got[b_bad], ref[b_bad], t, before


def test_bad_slot_means_no_history():
    p = build(Case(history=300))
    for bad in (-2, 5, 2 ** 31 - 1):
        def change(t):
            t["slots"][1] = bad
        got, _, _, _ = _expect(p, change, 1)
        q = build(Case(history=300))
        sv, a, t, strides = call(q)
        t["slots"][1] = -1
        sv.process(a)
        assert int(t["status"]) == 0
        assert np.array_equal(got, rows_out(q, t, strides)[0][1], equal_nan=True)


def test_bad_ids_are_ignored():
    p = build(Case(row0=3, biases=40))
    for what, at, bad in (("draft", (1, 0), -1), ("draft", (1, 3), 1000), ("btok", (int(p["boff"][1]),), -5),
                          ("btok", (int(p["boff"][1]),), 1 << 30)):
        def change(t):
            t[what][at] = bad
        got, ref, _, _ = _expect(p, change, 1)
        assert (got != ref).sum() <= 4  # the tokens that the id named before, in two rows


def test_bad_bias_offsets_mean_no_biases():
    p = build(Case(B=2, biases=30))
    for bad in (-1, 10 ** 6):
        def change(t):
            t["boff"][2] = bad
        got, _, _, _ = _expect(p, change, 1)
        q = build(Case(B=2, biases=30))
        sv, a, t, strides = call(q)
        t["boff"][2] = t["boff"][1]
        sv.process(a)
        assert np.array_equal(got, rows_out(q, t, strides)[0][1], equal_nan=True)


def test_offsets_into_no_biases_are_reported():
    p = build(Case(biases=0, masks=False))
    for off, status in (([0, 0, 0, 0], 0), ([0, 0, 1, 1], 1), ([0, -1, 0, 0], 1), ([2 ** 31 - 1] * 4, 1)):
        sv, a, t, strides = call(p, bias_offsets=torch.tensor(off, dtype=torch.int32, device=DEV))
        untouched = t["out"].float().cpu().numpy().astype(np.float64)
        sv.process(a)
        assert int(t["status"]) == status
        compare(p, t, strides, untouched)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rep", [2.0 ** -126, 1.2e-38, 3e-20, 1.0, 7.7e19, 3.4e38])
def test_extreme_repetitions(dtype, rep):
    # values below the types' normal range (2^-126 for both) may be flushed
    p = build(Case(dtype=dtype, masks=False, biases=0))
    p["rep"][:] = rep
    c = p["c"]
    top = 3.3895313892515355e38 if dtype == "bf16" else 3.4028234663852886e38
    for b in range(c.B):
        s = p["slots"][b]
        for r in range(c.rows):
            o, _, size = R.process_row(p["l"][b, r].astype(np.float64), p["draft"][b, :r], p["counts"][s] if s >= 0 else None,
                                       p["seen_flags"][s] if s >= 0 else None, float(p["rep"][b]), float(p["freq"][b]),
                                       float(p["pres"][b]), [], None)
            p["out"][b, r] = np.where(np.abs(o) > 4 * top, np.sign(o) * np.inf, o)
            p["tol"][b, r] = 6 * 2.0 ** -24 * np.minimum(size, 4 * top) + 2.0 ** -126
            if dtype == "bf16":
                p["tol"][b, r] += 2.0 ** -8 * np.minimum(np.abs(o), top)
    sv, a, t, strides = call(p)
    untouched = t["out"].float().cpu().numpy().astype(np.float64)
    sv.process(a)
    assert int(t["status"]) == 0
    compare(p, t, strides, untouched)


@pytest.mark.parametrize("rep", [1e-39, 1e-45, 0.0])
def test_repetitions_below_the_normal_range_are_bad(rep):
    p = build(Case())

    def change(t):
        t["rep"][1] = rep
    got, _, _, _ = _expect(p, change, 1)
    q = build(Case())
    sv, a, t, strides = call(q)
    t["rep"][1] = 1.0
    sv.process(a)
    assert int(t["status"]) == 0
    assert np.array_equal(got, rows_out(q, t, strides)[0][1], equal_nan=True)


def test_bad_mask_index_leaves_no_token():
    p = build(Case())
    for bad in (-2, 4, 1 << 30):
        def change(t):
            t["midx"][1, 0] = bad
        got, ref, t, _ = _expect(p, change, 1)
        assert (got[0] == -np.inf).all() and np.array_equal(got[1], ref[1], equal_nan=True)
        assert int(t["live"][1, 0]) == 0


def test_bad_penalties_are_neutral():
    p = build(Case())
    for what, bad, neutral in (("rep", 0.0, 1.0), ("rep", -1.0, 1.0), ("rep", float("nan"), 1.0), ("rep", float("inf"), 1.0),
                               ("freq", float("nan"), 0.0), ("pres", float("inf"), 0.0)):
        def change(t):
            t[what][1] = bad
        got, _, _, _ = _expect(p, change, 1)
        q = build(Case())
        sv, a, t, strides = call(q)
        t[what][1] = neutral
        sv.process(a)
        assert np.array_equal(got, rows_out(q, t, strides)[0][1], equal_nan=True), (what, bad)


def test_bad_row_counts_leave_the_rows_alone():
    p = build(Case(vlen=True, rows=4, B=4))

    def change(t):
        t["vlen"][2] = -1
    got, _, t, before = _expect(p, change, 2)
    assert torch.equal(t["out"].view(4, -1)[2], before.view(4, -1)[2]) and (t["live"][2] == -1).all()
    c = Case(packed=True, rows=3, B=3)
    q = build(c)
    for off in ([0, 1, 5, 6], [0, 2, 1, 3]):  # four rows where three are the most; descending
        sv, a, t, _ = call(q)
        V = c.V
        flat = torch.zeros((8 * V,), dtype=torch.bfloat16, device=DEV)
        out = torch.full_like(flat, 55)
        off_t = torch.tensor(off, dtype=torch.int64, device=DEV)
        a.logits_in, a.logits_out, a.row_offsets = flat.data_ptr(), out.data_ptr(), off_t.data_ptr()
        sv.process(a)
        assert int(t["status"]) == 1
        assert (t["live"][1] == -1).all()
        bad_only = torch.ones(8, dtype=torch.bool)
        for b in (0, 2):
            bad_only[off[b]:off[b + 1]] = False
        assert (out.view(8, V)[bad_only] == 55).all()


# ---------------------------------------------------------------- history

def _history(B, V, n_slots, sequences, output, *, flat=False, most=None, seed=0, lengths=False, state=None, resets=True):
    """One call; sequences: (slot, tokens, reset).  Returns counts, seen (device), status."""
    LB = _lib()
    rng = np.random.default_rng(seed)
    most = max([len(t) for _, t, _ in sequences] + [0]) if most is None else most
    if state is None:
        counts = torch.from_numpy(rng.integers(0, 5, (n_slots, V)).astype(np.int32)).to(DEV)
        flags = rng.random((n_slots, V)) < 0.1
        seen = torch.from_numpy(R.words(flags).view(np.int32)).to(DEV)
    else:
        counts, seen = state
        flags = None
    slots = torch.tensor([s for s, _, _ in sequences], dtype=torch.int32, device=DEV)
    reset = torch.tensor([r for _, _, r in sequences], dtype=torch.int32, device=DEV)
    status = torch.full((1,), -9, dtype=torch.int32, device=DEV)
    kw = dict(slots=slots, reset=reset if resets else None, counts=counts, seen=seen, n_slots=n_slots, device_status=status,
              kind=LB.SV_HISTORY_OUTPUT if output else LB.SV_HISTORY_PROMPT, max_tokens=most)
    if flat:
        off = np.concatenate([[0], np.cumsum([len(t) for _, t, _ in sequences])])
        tokens = torch.tensor([x for _, t, _ in sequences for x in t] + [0], dtype=torch.int32, device=DEV)
        kw.update(tokens=tokens, token_offsets=torch.from_numpy(off.astype(np.int64)).to(DEV), n_tokens=int(off[-1]))
    else:
        pad = np.full((B, most + 3), 0 if lengths else -1, np.int32)
        for b, (_, t, _) in enumerate(sequences):
            pad[b, :len(t)] = t
        kw.update(tokens=torch.from_numpy(pad).to(DEV), token_stride=most + 3)
        if lengths:
            kw.update(lengths=torch.tensor([len(t) for _, t, _ in sequences], dtype=torch.int32, device=DEV))
    before = (counts.cpu().numpy().astype(np.int64), flags)
    sv = LB.SpecVerify(max(B, 1), 1, V, LB.SV_BF16)
    sv.history(LB.make_history_args(B, **kw))
    torch.cuda.synchronize()
    return before, counts.cpu().numpy(), seen.cpu().numpy().view(np.uint32), int(status)


@pytest.mark.parametrize("B,V,longest,flat,lengths,output", [
    (1, 600001, 40000, True, False, True), (2, 600001, 3000, False, False, False), (4100, 65, 3, False, False, True),
    (9, 5000, 33000, True, False, True), (5, 5000, 33000, True, False, False), (70, 3000, 600, False, True, True),
    (1, 1, 1, False, False, True), (1, 1000, 0, False, False, True), (3, 33, 5, False, True, True), (3, 129280, 700, True, False, True),
    (5, 4097, 3000, True, False, False), (64, 1000, 17, False, False, True), (2, 50257, 20000, False, True, False)])
def test_history_matches_the_oracle(B, V, longest, flat, lengths, output):
    print(f"[case] history {B} {V} {longest} {flat} {lengths} {output}", flush=True)
    rng = np.random.default_rng(B + V)
    slots = rng.permutation(B + 4)[:B]
    seqs = []
    for b in range(B):
        n = longest if b == 0 else int(rng.integers(0, longest + 1))
        t = (rng.random(n) ** 3 * V).astype(int).tolist()  # some ids come often
        if n > 2 and not lengths:
            t[1] = -1
        seqs.append((int(slots[b]) if b != 2 else -1, t, int(rng.integers(0, 2))))
    for resets in (True, False):
        mine = [(s, t, r if resets else 0) for s, t, r in seqs]
        before, counts, seen, status = _history(B, V, B + 4, mine, output, flat=flat, lengths=lengths, seed=B, resets=resets)
        want_c, want_s = before[0].copy(), before[1].copy()
        R.history_update(want_c, want_s, mine, output)
        assert status == 0
        assert np.array_equal(counts, want_c)
        assert np.array_equal(seen, R.words(want_s))


@pytest.mark.parametrize("seqs", [
    [(1, [3, 3, 5], 1), (1, [3, 7], 0), (1, [9], 1)], [(1, [3, 3, 5], 0), (0, [8], 0), (1, [3, 7], 1)],
    [(0, [2], 0), (1, [1] * 700, 0), (0, [2] * 40, 0), (1, [], 0)], [(0, [2] * 33000, 0), (0, [4], 1), (1, [5], 0)]])
def test_two_sequences_of_one_slot_both_count(seqs):
    before, counts, seen, status = _history(len(seqs), 100, 2, seqs, True)
    want_c, want_s = before[0].copy(), before[1].copy()
    R.history_update(want_c, want_s, seqs, True)
    assert status == 0 and np.array_equal(counts, want_c) and np.array_equal(seen, R.words(want_s))


@pytest.mark.parametrize("seqs,kw", [
    ([(0, [1, 2], 1), (7, [3], 1)], {}), ([(0, [1, 2], 1), (-2, [3], 1)], {}),
    ([(0, [1, 2], 1), (1, [100, 3, -7], 0)], {}), ([(0, [1], 1), (1, [3, 4, 5], 1)], dict(flat=True, most=2)),
    ([(0, [1], 1), (1, [3, 4, 5], 1)], dict(lengths=True, most=2)),
])
def test_bad_history_input_is_reported_and_skipped(seqs, kw):
    if kw.get("lengths"):  # the row is as wide as the tokens; the length says more than max_tokens
        kw = dict(kw, most=3)
        LB = _lib()
        counts = torch.zeros((2, 100), dtype=torch.int32, device=DEV)
        seen = torch.zeros((2, 4), dtype=torch.int32, device=DEV)
        status = torch.zeros((1,), dtype=torch.int32, device=DEV)
        tok = torch.tensor([[1, 0, 0], [3, 4, 5]], dtype=torch.int32, device=DEV)
        for bad in (3, -1):
            n = torch.tensor([1, bad], dtype=torch.int32, device=DEV)
            counts.zero_()
            LB.SpecVerify(2, 1, 100, LB.SV_F32).history(LB.make_history_args(
                2, tokens=tok, token_stride=3, max_tokens=2, lengths=n, kind=LB.SV_HISTORY_OUTPUT, counts=counts, seen=seen,
                n_slots=2, device_status=status))
            assert int(status) == 1 and counts.sum() == 1 and counts[0, 1] == 1
        return
    before, counts, seen, status = _history(2, 100, 2, seqs, True, **kw)
    assert status == 1
    fine = [(s, [v for v in t if v < 100], r) for s, t, r in seqs if 0 <= s < 2 and len(t) <= kw.get("most", 99)]
    want_c, want_s = before[0].copy(), before[1].copy()
    R.history_update(want_c, want_s, fine, True)
    assert np.array_equal(counts, want_c) and np.array_equal(seen, R.words(want_s))
