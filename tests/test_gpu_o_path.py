"""The calls of one decoding step together, as an engine makes them: for every
drafted position the 4-bit head, the rules on its logits and a draw; then the
target's head over the whole block, the rules, verification, and the history.
Checked call by call against the oracles, and captured in a HIP graph."""
import numpy as np
import pytest

from oracle import oracle as O
from oracle import rules as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
B, K, V, H = 5, 3, 3001, 192
T = 0.8


class Step:
    """Inputs, state and buffers of one step; logits in fp32."""

    def __init__(self, seed):
        from draft_verification_amd import binding as L
        self.L = L
        rng = np.random.default_rng(seed)
        self.sv = L.SpecVerify(B, K, V, L.SV_F32)
        self.codes = [rng.integers(0, 256, (V, H // 2)).astype(np.uint8) for _ in range(2)]
        s8 = rng.integers(120, 124, (V, H // 32)).astype(np.uint8)
        sb = torch.from_numpy((0.02 * (0.5 + rng.random((V, H // 64)))).astype(np.float32)).to(torch.bfloat16)
        self.scale = [np.ldexp(1.0, s8.astype(int) - 127), sb.double().numpy()]
        self.head = []
        for fmt, group, codes, scale in ((L.SV_W4_FP4, 32, self.codes[0], torch.from_numpy(s8)),
                                         (L.SV_W4_INT4, 64, self.codes[1], sb)):
            packed = torch.empty(self.sv.head_packed_bytes(H, fmt, group), dtype=torch.uint8, device=DEV)
            self.sv.head_pack(L.make_head_pack_args(hidden=H, format=fmt, group=group, weights=torch.from_numpy(codes).to(DEV),
                                                    weight_stride=H // 2, scales=scale.to(DEV), scale_stride=H // group,
                                                    packed=packed))
            self.head.append(dict(hidden=H, format=fmt, group=group, packed=packed))
        torch.cuda.synchronize()  # the sources may go

        def hidden(*shape):
            return torch.from_numpy(rng.standard_normal(shape + (H,)).astype(np.float32)).to(torch.bfloat16).to(DEV)
        self.xd, self.xt = hidden(K, B), hidden(B, K + 1)
        self.draft = torch.zeros((B, K, V), device=DEV)
        self.target = torch.zeros((B, K + 1, V), device=DEV)
        self.tokens = torch.zeros((B, K), dtype=torch.int32, device=DEV)
        self.zeros = torch.zeros((B, 1), dtype=torch.int32, device=DEV)
        self.none = torch.zeros((B,), dtype=torch.int32, device=DEV)
        self.u_draw = torch.from_numpy(rng.random((K, B, 2)).astype(np.float32)).to(DEV)
        self.u = torch.from_numpy(rng.random((B, K + 1)).astype(np.float32)).to(DEV)

        def i32(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=DEV)
        self.draw_len, self.draw_out, self.draw_vl = i32(K, B), i32(K, B, 2), i32(K, B)
        self.acc, self.out, self.vl, self.status = i32(B), i32(B, K + 1), i32(B), i32(4)
        self.live = i32(B, K + 1)
        # requests: history, penalties, biases, and a grammar for two of them
        self.n_slots = B + 1
        self.slots = torch.tensor([3, 0, -1, 5, 1], dtype=torch.int32, device=DEV)
        h = [rng.integers(0, V, 400) for _ in range(self.n_slots)]
        self.counts0, self.seen0 = np.zeros((self.n_slots, V), np.int64), np.zeros((self.n_slots, V), bool)
        R.history_update(self.counts0, self.seen0, [(s, t, 0) for s, t in enumerate(h)], True)
        self.counts = torch.from_numpy(self.counts0.astype(np.int32)).to(DEV)
        self.seen = torch.from_numpy(R.words(self.seen0).view(np.int32)).to(DEV)
        self.rep, self.freq, self.pres = (1.0 + 0.4 * rng.random(B)).astype(np.float32), (0.3 * rng.random(B)).astype(np.float32), \
            (0.3 * rng.random(B)).astype(np.float32)
        self.boff = np.array([0, 4, 4, 9, 9, 10], np.int32)
        self.btok, self.bval = rng.integers(0, V, 10).astype(np.int32), (3 * rng.standard_normal(10)).astype(np.float32)
        self.mask = rng.random((3, V)) < np.array([0.5, 0.05, 0.9])[:, None]
        self.midx = np.full((B, K + 1), -1, np.int32)
        self.midx[1], self.midx[3] = [0, 1, 2, 0], [2, 2, 1, 1]
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
        self.dev = dict(slots=self.slots, repetition=up(self.rep), frequency=up(self.freq), presence=up(self.pres),
                        bias_offsets=up(self.boff), bias_tokens=up(self.btok), bias_values=up(self.bval), n_biases=10,
                        history_counts=self.counts, history_seen=self.seen, n_slots=self.n_slots)
        self.masks, self.midx_dev = up(R.words(self.mask).view(np.int32)), up(self.midx)
        self.midx_col = [self.midx_dev[:, j:j + 1].contiguous() for j in range(K)]

    def state(self):
        return [self.counts, self.seen, self.tokens]

    def outputs(self):
        return [self.draft, self.target, self.tokens, self.draw_out, self.acc, self.out, self.vl, self.live, self.counts,
                self.seen, self.status]

    def run(self, stream=None):
        L, sv = self.L, self.sv
        masks = dict(masks=self.masks, mask_stride=self.masks.shape[1], n_masks=3)
        for j in range(K):
            row = self.draft[:, j]  # one row of every sequence's block
            sv.head(L.make_head_args(B, hidden_states=self.xd[j], hidden_stride=H, logits=row, logits_stride=K * V,
                                     **self.head[0]), stream)
            sv.process(L.make_process_args(B, 1, row0=j, logits_in=row, in_strides=(K * V, V), logits_out=row,
                                           out_strides=(K * V, V), draft_tokens=self.tokens, draft_stride=K,
                                           mask_index=self.midx_col[j], device_status=self.status[:1], **masks, **self.dev),
                       stream)
            # a draw from the row: verification of no position, whose bonus token it is
            sv.run(L.make_args(B, 1, target=row, target_strides=(K * V, V), tokens=self.zeros, uniforms=self.u_draw[j],
                               temperature=T, verify_len=self.none, draft_mode=L.SV_DRAFT_ONEHOT,
                               accepted_len=self.draw_len[j], out_tokens=self.draw_out[j], verify_len_out=self.draw_vl[j]),
                   stream)
            with torch.cuda.stream(torch.cuda.current_stream() if stream is None else torch.cuda.ExternalStream(stream)):
                self.tokens[:, j].copy_(self.draw_out[j][:, 0])
        rows = B * (K + 1)
        sv.head(L.make_head_args(rows, hidden_states=self.xt, hidden_stride=H, logits=self.target, logits_stride=V,
                                 **self.head[1]), stream)
        sv.process(L.make_process_args(B, K + 1, logits_in=self.target, in_strides=((K + 1) * V, V), logits_out=self.target,
                                       out_strides=((K + 1) * V, V), draft_tokens=self.tokens, draft_stride=K,
                                       mask_index=self.midx_dev, live_tokens=self.live, device_status=self.status[1:2],
                                       **masks, **self.dev), stream)
        sv.run(L.make_args(B, K, target=self.target, target_strides=((K + 1) * V, V), draft=self.draft,
                           draft_strides=(K * V, V), tokens=self.tokens, uniforms=self.u, temperature=T,
                           accepted_len=self.acc, out_tokens=self.out, verify_len_out=self.vl,
                           device_status=self.status[2:3]), stream)
        sv.history(L.make_history_args(B, tokens=self.out, token_stride=K + 1, max_tokens=K + 1, kind=L.SV_HISTORY_OUTPUT,
                                       slots=self.slots, counts=self.counts, seen=self.seen, n_slots=self.n_slots,
                                       device_status=self.status[3:]), stream)

    def rules(self, l, b, j, tokens, counts, seen):
        s = int(self.slots[b])
        e = slice(self.boff[b], self.boff[b + 1])
        m = self.midx[b, j]
        return R.process_row(l, tokens[b, :j], counts[s] if s >= 0 else None, seen[s] if s >= 0 else None, float(self.rep[b]),
                             float(self.freq[b]), float(self.pres[b]), list(zip(self.btok[e], self.bval[e].astype(float))),
                             self.mask[m] if m >= 0 else None)


def _close(got, want, tol):
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine])
    off = np.abs(got[fine] - want[fine])
    assert (off <= tol[fine]).all(), off.max()


def test_a_step_call_by_call():
    s = Step(11)
    s.run()
    torch.cuda.synchronize()
    assert s.status.tolist() == [0, 0, 0, 0]
    host = lambda t: t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()  # noqa: E731
    tokens, draft, target = host(s.tokens), host(s.draft), host(s.target)
    for which, x, logits in ((0, s.xd.transpose(0, 1), draft), (1, s.xt, target)):
        W = R.head_weights(s.codes[which], s.scale[which], which == 0, 32 if which == 0 else 64)
        mag = np.abs(W) if which == 0 else np.abs(W) + 48 * np.repeat(s.scale[1], 64, 1)
        x = x.double().cpu().numpy()
        for b in range(B):
            for j in range(logits.shape[1]):
                want, live, size = s.rules(W @ x[b, j], b, j, tokens, s.counts0, s.seen0)
                # the head's bound (its own test states it), through a penalty of at most 1.4, and the rules'
                tol = 1.4 * (H / 32 + 40) * 2.0 ** -23 * (mag @ np.abs(x[b, j])) + 12 * 2.0 ** -24 * size
                _close(logits[b, j].astype(np.float64), want, tol)
                if which:
                    assert host(s.live)[b, j] == live
    for j in range(K):  # the draws, from the very logits
        row = np.repeat(draft[:, j:j + 1], 2, 1)
        o = O.verify(row, None, np.zeros((B, 1), np.int32), host(s.u_draw[j]), T, dtype=O.F32, verify_len=np.zeros(B, np.int32),
                     draft_mode=O.DRAFT_ONEHOT)
        ok = o.margin == 0
        assert np.array_equal(host(s.draw_out[j])[ok, 0], o.out_tokens[ok, 0])
    o = O.verify(target, draft, tokens, host(s.u), T, dtype=O.F32)
    ok = o.margin == 0
    assert ok.sum() >= B - 1
    assert np.array_equal(host(s.acc)[ok], o.accepted_len[ok]) and np.array_equal(host(s.out)[ok], o.out_tokens[ok])
    counts, seen = s.counts0.copy(), s.seen0.copy()
    R.history_update(counts, seen, [(int(sl), o, 0) for sl, o in zip(s.slots.cpu(), host(s.out))], True)
    assert np.array_equal(host(s.counts), counts) and np.array_equal(host(s.seen).view(np.uint32), R.words(seen))
    # a token that the grammar excludes is neither drawn nor emitted
    for b in (1, 3):
        for j, t in enumerate(host(s.out)[b]):
            assert t < 0 or s.mask[s.midx[b, j], t]


def test_a_step_on_another_stream_and_replayed():
    s = Step(12)
    start = [t.clone() for t in s.state()]

    def restore():
        for t, was in zip(s.state(), start):
            t.copy_(was)
    s.run()
    torch.cuda.synchronize()
    want = [t.clone() for t in s.outputs()]
    side = torch.cuda.Stream()
    restore()
    for t in s.outputs()[:2]:
        t.fill_(7.0)
    side.wait_stream(torch.cuda.current_stream())
    s.run(side.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(s.outputs(), want))
    restore()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for k in range(4):
        restore()
        if k == 2:  # eager work of the same handle and buffers between two replays
            s.run()
            restore()
        for t in s.outputs()[:2]:
            t.fill_(float(k))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(s.outputs(), want)), k
        _ = torch.ones(1000, device=DEV).sum().item()
