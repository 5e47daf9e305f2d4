"""The calls around verification at the far ends of their ranges: offsets past
2^31 elements, many rows and sequences, the widest vocabulary, two calls at once."""
import numpy as np
import pytest

from oracle import rules as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
FAR = 2 ** 31 + 40


def _lib():
    from draft_verification_amd import binding
    return binding


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _one_row(V, seed):
    """A row with its rules, and the oracle's result (fp32: at most 8 roundings of the sizes involved)."""
    rng = np.random.default_rng(seed)
    l = (3 * rng.standard_normal(V)).astype(np.float32)
    counts = np.zeros(V, np.int32)
    seen = np.zeros(V, bool)
    t = rng.integers(0, V, 500)
    seen[t] = True
    np.add.at(counts, t, 1)
    seen[-1], counts[-1] = True, 3
    allowed = rng.random(V) < 0.7
    draft = np.array([0, V - 1, int(t[0]), V // 2], np.int32)
    out, live, size = R.process_row(l.astype(np.float64), draft[:2], counts, seen, 1.25, 0.5, 0.25, [], allowed)
    return dict(l=l, counts=counts, seen=seen, allowed=allowed, draft=draft, out=out, live=live, tol=8 * 2.0 ** -24 * size)


def _same(got, q):
    want = q["out"]
    with np.errstate(invalid="ignore"):
        ok = (got == want) | (np.abs(got - want) <= q["tol"])
    assert ok.all(), np.flatnonzero(~ok)[:5]


@pytest.mark.parametrize("what", ["batch", "row", "packed"])
@pytest.mark.parametrize("inplace", [False, True])
def test_process_past_32_bits_of_elements(what, inplace):
    B = _lib()
    V = 2 ** 20
    q = _one_row(V, 1)
    flat = torch.zeros(FAR + V, dtype=torch.float32, device=DEV)
    flat[FAR:] = torch.from_numpy(q["l"]).to(DEV)
    out = flat if inplace else torch.zeros_like(flat)
    # the row in question is the last: of the second sequence, or of the second row
    Bn, rows = (1, 2) if what == "row" else (2, 1)
    n_slots = 2100  # its history lies past 2^31 counts, its mask past 2^31 bits
    counts = torch.zeros((n_slots, V), dtype=torch.int32, device=DEV)
    seen = torch.zeros((n_slots, V // 32), dtype=torch.int32, device=DEV)
    masks = torch.full((n_slots, V // 32), -1, dtype=torch.int32, device=DEV)
    counts[-1] = torch.from_numpy(q["counts"]).to(DEV)
    seen[-1] = torch.from_numpy(R.words(q["seen"]).view(np.int32)).to(DEV)
    masks[-1] = torch.from_numpy(R.words(q["allowed"]).view(np.int32)).to(DEV)
    draft = torch.from_numpy(np.tile(q["draft"], (Bn, 1))).to(DEV)
    f = lambda x: torch.full((Bn,), x, device=DEV)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    live, status = torch.zeros((Bn, rows), dtype=torch.int32, device=DEV), i([-9])
    strides = (FAR, V) if what == "batch" else (0, FAR)
    kw = dict(row0=1 if what == "row" else 2, logits_in=flat, in_strides=strides, logits_out=out, out_strides=strides,
              draft_tokens=draft, draft_stride=4, history_counts=counts, history_seen=seen, n_slots=n_slots,
              slots=i([n_slots - 1] * Bn), repetition=f(1.25), frequency=f(0.5), presence=f(0.25), masks=masks,
              mask_stride=V // 32, n_masks=n_slots, mask_index=i([0, n_slots - 1]).view(Bn, rows), live_tokens=live,
              device_status=status)
    if what == "packed":
        kw.update(row_offsets=torch.tensor([0, 0, 1], dtype=torch.int64, device=DEV), mask_index=i([[-1], [n_slots - 1]]),
                  logits_in=flat[FAR:], logits_out=out[FAR:])
        # row offsets themselves past 2^31 / V: rows 2048 of V elements start there
        first = FAR // V
        kw.update(row_offsets=torch.tensor([0, 0, 1], dtype=torch.int64, device=DEV) + first, in_strides=(0, V),
                  out_strides=(0, V), logits_in=flat[FAR - first * V:], logits_out=out[FAR - first * V:])
    sv = B.SpecVerify(2, 3, V, B.SV_F32)
    sv.process(B.make_process_args(Bn, rows, **kw))
    assert int(status) == 0
    _same(out[FAR:].cpu().numpy().astype(np.float64), q)
    assert int(live.flatten()[-1]) == q["live"]
    assert not out[V:FAR].any()


def test_history_past_32_bits_of_counts():
    B = _lib()
    V, n_slots = 2 ** 20, 2100
    counts = torch.ones((n_slots, V), dtype=torch.int32, device=DEV)
    seen = torch.full((n_slots, V // 32), -1, dtype=torch.int32, device=DEV)
    rng = np.random.default_rng(3)
    for n, reset in ((900, 1), (900, 0), (40000, 1), (40000, 0)):
        t = rng.integers(0, V, n).astype(np.int32)
        slots = torch.tensor([n_slots - 1, n_slots - 2], dtype=torch.int32, device=DEV)
        tok = torch.from_numpy(np.stack([t, t[::-1]]).copy()).to(DEV)
        before = counts[-3:].cpu().numpy()
        B.SpecVerify(2, 1, V, B.SV_BF16).history(B.make_history_args(
            2, tokens=tok, token_stride=n, max_tokens=n, kind=B.SV_HISTORY_OUTPUT, slots=slots,
            reset=torch.full((2,), reset, dtype=torch.int32, device=DEV), counts=counts, seen=seen, n_slots=n_slots))
        got, want = counts[-3:].cpu().numpy(), before.copy()
        if reset:
            want[1:] = 0
        np.add.at(want[1], t, 1)
        np.add.at(want[2], t, 1)
        assert np.array_equal(got, want), (n, reset)
        if reset:
            flags = np.zeros(V, bool)
            flags[t] = True
            for s in (-1, -2):
                assert np.array_equal(seen[s].cpu().numpy().view(np.uint32), R.words(flags)), (n, reset, s)
    assert (counts[:-2] == 1).all() and (seen[:-2] == -1).all()


@pytest.mark.parametrize("M,V,fmt", [(2, 1000, 0), (2, 1000, 1), (40, 66000, 0), (20, 82000, 1)])
def test_head_rows_past_32_bits_of_elements(M, V, fmt):
    B = _lib()
    H, group = 256, 32
    far = FAR // (M - 1) + 1
    g = torch.Generator(device=DEV).manual_seed(M)
    w = torch.randint(0, 256, (V, H // 2), dtype=torch.uint8, device=DEV, generator=g)
    if fmt == B.SV_W4_FP4:
        s = torch.randint(118, 124, (V, H // group), dtype=torch.uint8, device=DEV, generator=g)
    else:
        s = (0.5 + torch.rand((V, H // group), device=DEV, generator=g)).to(torch.bfloat16)
    sv = B.SpecVerify(M, 1, V, B.SV_BF16)
    packed = torch.empty(sv.head_packed_bytes(H, fmt, group), dtype=torch.uint8, device=DEV)
    sv.head_pack(B.make_head_pack_args(hidden=H, format=fmt, group=group, weights=w, weight_stride=H // 2, scales=s,
                                       scale_stride=H // group, packed=packed))
    near = torch.randn((M, H), device=DEV, generator=g).to(torch.bfloat16)
    x = torch.zeros((M - 1) * far + H, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros((M - 1) * far + V, dtype=torch.bfloat16, device=DEV)
    x.as_strided((M, H), (far, 1)).copy_(near)
    small = torch.empty((M, V), dtype=torch.bfloat16, device=DEV)
    kw = dict(hidden=H, format=fmt, group=group, packed=packed)
    sv.head(B.make_head_args(M, hidden_states=near, hidden_stride=H, logits=small, logits_stride=V, **kw))
    sv.head(B.make_head_args(M, hidden_states=x, hidden_stride=far, logits=out, logits_stride=far, **kw))
    assert torch.isfinite(small).all() and small.abs().max() > 0
    assert torch.equal(out.as_strided((M, V), (far, 1)), small)  # the same sums, elsewhere


@pytest.mark.parametrize("M", [3, 40])
@pytest.mark.parametrize("fmt,group", [(0, 32), (1, 128)])
def test_head_weights_past_4_gb(M, fmt, group):
    B = _lib()
    V, H = 2 ** 20, 9216
    g = torch.Generator(device=DEV).manual_seed(M)
    w = torch.randint(0, 256, (V, H // 2), dtype=torch.uint8, device=DEV, generator=g)
    if fmt == B.SV_W4_FP4:
        s = torch.randint(118, 124, (V, H // group), dtype=torch.uint8, device=DEV, generator=g)
    else:
        s = (0.5 + torch.rand((V, H // group), device=DEV, generator=g)).to(torch.bfloat16)
    sv = B.SpecVerify(M, 1, V, B.SV_F32)
    packed = torch.empty(sv.head_packed_bytes(H, fmt, group), dtype=torch.uint8, device=DEV)
    assert packed.numel() > 2 ** 32
    sv.head_pack(B.make_head_pack_args(hidden=H, format=fmt, group=group, weights=w, weight_stride=H // 2, scales=s,
                                       scale_stride=H // group, packed=packed))
    x = torch.randn((M, H), device=DEV, generator=g).to(torch.bfloat16)
    out = torch.empty((M, V), device=DEV)
    sv.head(B.make_head_args(M, hidden=H, format=fmt, group=group, packed=packed, hidden_states=x, hidden_stride=H,
                             logits=out, logits_stride=V))
    at = torch.tensor([0, 1, 77, V // 2 - 1, V // 2, V - 65, V - 64, V - 2, V - 1], device=DEV)
    sc = s[at].double().cpu().numpy()
    W = R.head_weights(w[at].cpu().numpy(), np.exp2(sc - 127) if fmt == B.SV_W4_FP4 else sc, fmt == B.SV_W4_FP4, group)
    xd = x.double().cpu().numpy()
    scale = np.repeat(np.exp2(sc - 127) if fmt == B.SV_W4_FP4 else sc, group, 1)
    # INT4 adds (code + 16) x and takes 24 x off, all times the scale
    size = np.abs(xd) @ (np.abs(W) if fmt == B.SV_W4_FP4 else np.abs(W + 24 * scale) + 24 * scale).T
    off = np.abs(out[:, at].double().cpu().numpy() - xd @ W.T)
    assert (off <= (H / 32 + 40) * 2.0 ** -23 * size).all(), (off / size).max()


def test_many_rows_of_many_sequences():
    # 2060 sequences of 130 rows are 3 chunks of rows to a workgroup's 64
    B = _lib()
    Bn, rows, V = 2060, 130, 72
    rng = np.random.default_rng(9)
    l = torch.from_numpy((3 * rng.standard_normal((Bn, rows, V))).astype(np.float32)).to(DEV)
    seen = rng.random((Bn, V)) < 0.2
    counts = (seen * rng.integers(0, 4, (Bn, V))).astype(np.int32)
    draft = rng.integers(0, V, (Bn, rows - 1)).astype(np.int32)
    allowed = rng.random((3, V)) < 0.5
    midx = rng.integers(-1, 3, (Bn, rows)).astype(np.int32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    out = torch.zeros_like(l)
    live, status = torch.zeros((Bn, rows), dtype=torch.int32, device=DEV), torch.full((1,), -9, dtype=torch.int32, device=DEV)
    f = lambda x: torch.full((Bn,), x, device=DEV)
    sv = B.SpecVerify(Bn, rows - 1, V, B.SV_F32)
    sv.process(B.make_process_args(
        Bn, rows, logits_in=l, in_strides=(rows * V, V), logits_out=out, out_strides=(rows * V, V), draft_tokens=dev(draft),
        draft_stride=rows - 1, history_counts=dev(counts), history_seen=dev(R.words(seen).view(np.int32)), n_slots=Bn,
        repetition=f(1.25), frequency=f(0.5), presence=f(0.25), masks=dev(R.words(allowed).view(np.int32)), mask_stride=3,
        n_masks=3, mask_index=dev(midx), live_tokens=live, device_status=status))
    assert int(status) == 0
    host, got, lv = l.cpu().numpy().astype(np.float64), out.cpu().numpy().astype(np.float64), live.cpu().numpy()
    for b in (0, 1, 2, 1030, 2058, 2059):
        for r in range(rows):
            m = midx[b, r]
            o, n, size = R.process_row(host[b, r], draft[b, :r], counts[b], seen[b], 1.25, 0.5, 0.25, [], allowed[m] if m >= 0 else None)
            with np.errstate(invalid="ignore"):
                ok = (got[b, r] == o) | (np.abs(got[b, r] - o) <= 8 * 2.0 ** -24 * size)
            assert ok.all() and lv[b, r] == n, (b, r)
    # every sequence again, alone
    alone = torch.zeros_like(out)
    for b0 in range(0, Bn, 515):
        n = min(515, Bn - b0)
        sv.process(B.make_process_args(
            n, rows, logits_in=l[b0:], in_strides=(rows * V, V), logits_out=alone[b0:], out_strides=(rows * V, V),
            draft_tokens=dev(draft[b0:b0 + n]), draft_stride=rows - 1, history_counts=dev(counts[b0:b0 + n]),
            history_seen=dev(R.words(seen[b0:b0 + n]).view(np.int32)), n_slots=n, repetition=f(1.25), frequency=f(0.5),
            presence=f(0.25), masks=dev(R.words(allowed).view(np.int32)), mask_stride=3, n_masks=3,
            mask_index=dev(midx[b0:b0 + n])))
        torch.cuda.synchronize()
    assert torch.equal(alone, out)


@pytest.mark.parametrize("inplace", [False, True])
def test_more_sequences_than_one_launch_takes(inplace):
    B = _lib()
    Bn, V = 70001, 40
    rng = np.random.default_rng(11)
    l = torch.from_numpy((3 * rng.standard_normal((Bn, V))).astype(np.float32)).to(DEV)
    seen = rng.random((Bn, V)) < 0.3
    counts = (seen * rng.integers(0, 4, (Bn, V))).astype(np.int32)
    allowed = rng.random((Bn, V)) < 0.6
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    out = l.clone() if inplace else torch.zeros_like(l)
    src = out if inplace else l
    i32 = dict(dtype=torch.int32, device=DEV)
    live, status = torch.zeros((Bn, 1), **i32), torch.full((1,), -9, **i32)
    f = lambda x: torch.full((Bn,), x, device=DEV)
    keep = [dev(counts), dev(R.words(seen).view(np.int32)), dev(R.words(allowed).view(np.int32)), torch.arange(Bn, **i32)]
    sv = B.SpecVerify(Bn, 1, V, B.SV_F32)
    sv.process(B.make_process_args(
        Bn, 1, logits_in=src, in_strides=(V, V), logits_out=out, out_strides=(V, V), history_counts=keep[0],
        history_seen=keep[1], n_slots=Bn, repetition=f(1.25), frequency=f(0.5), presence=f(0.25), masks=keep[2],
        mask_stride=2, n_masks=Bn, mask_index=keep[3], live_tokens=live, device_status=status))
    assert int(status) == 0
    host, got, lv = l.cpu().numpy().astype(np.float64), out.cpu().numpy().astype(np.float64), live.cpu().numpy()
    for b in [0, 1, 65534, 65535, 65536, 65537, 70000] + rng.integers(0, Bn, 300).tolist():
        o, n, size = R.process_row(host[b], [], counts[b], seen[b], 1.25, 0.5, 0.25, [], allowed[b])
        with np.errstate(invalid="ignore"):
            ok = (got[b] == o) | (np.abs(got[b] - o) <= 8 * 2.0 ** -24 * size)
        assert ok.all() and lv[b, 0] == n, b


def test_two_calls_at_once_on_one_handle():
    B = _lib()
    V, H = 50257, 512
    sv = B.SpecVerify(8, 4, V, B.SV_BF16)
    g = torch.Generator(device=DEV).manual_seed(2)
    w = torch.randint(0, 256, (V, H // 2), dtype=torch.uint8, device=DEV, generator=g)
    s = torch.randint(118, 124, (V, H // 32), dtype=torch.uint8, device=DEV, generator=g)
    packed = torch.empty(sv.head_packed_bytes(H, B.SV_W4_FP4, 32), dtype=torch.uint8, device=DEV)
    sv.head_pack(B.make_head_pack_args(hidden=H, format=B.SV_W4_FP4, group=32, weights=w, weight_stride=H // 2, scales=s,
                                       scale_stride=H // 32, packed=packed))

    def side(seed, M):
        """A chain of the three calls with buffers of its own."""
        g = torch.Generator(device=DEV).manual_seed(seed)
        x = torch.randn((M, H), device=DEV, generator=g).to(torch.bfloat16)
        logits = torch.zeros((M, V), dtype=torch.bfloat16, device=DEV)
        counts = torch.zeros((M, V), dtype=torch.int32, device=DEV)
        seen = torch.zeros((M, (V + 31) // 32), dtype=torch.int32, device=DEV)
        tok = torch.randint(0, V, (M, 3000), dtype=torch.int32, device=DEV, generator=g)
        status = torch.zeros(2, dtype=torch.int32, device=DEV)
        pen = torch.full((M,), 1.5, device=DEV)
        hist = B.make_history_args(M, tokens=tok, token_stride=3000, max_tokens=3000, kind=B.SV_HISTORY_OUTPUT, counts=counts,
                                   seen=seen, n_slots=M, device_status=status)
        head = B.make_head_args(M, hidden=H, format=B.SV_W4_FP4, group=32, packed=packed, hidden_states=x, hidden_stride=H,
                                logits=logits, logits_stride=V)
        proc = B.make_process_args(M, 1, logits_in=logits, in_strides=(V, V), logits_out=logits, out_strides=(V, V),
                                   history_counts=counts, history_seen=seen, n_slots=M, repetition=pen, frequency=pen,
                                   presence=pen, device_status=status[1:])
        keep = (x, tok, pen)

        def run(stream=0):
            for _ in range(5):
                sv.history(hist, stream=stream)
                sv.head(head, stream=stream)
                sv.process(proc, stream=stream)

        def clear():
            counts.zero_()
            seen.zero_()
            logits.zero_()
        return run, clear, (logits, counts, seen, status), keep

    sides = [side(1, 8), side(2, 5)]
    want = []
    for run, clear, out, _ in sides:
        run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
        clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st, (run, _, _, _) in zip(streams, sides):
        run(st.cuda_stream)
    torch.cuda.synchronize()
    for (_, _, out, _), ref in zip(sides, want):
        for t, r in zip(out, ref):
            assert torch.equal(t, r)
