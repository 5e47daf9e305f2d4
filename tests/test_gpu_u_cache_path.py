"""The target's cache through verification steps, as an engine makes them: pages for the
block, for each layer append and attend, the head, verification, the history, and the pages
cut back to what was accepted.  On streams, captured, two calls at once, and at offsets past
32 bits."""
import numpy as np
import pytest

from oracle import cache as C
from oracle import oracle as O
from oracle import rules as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.cache_util import DEV, bf16, lib, up  # noqa: E402
from tests.test_gpu_t_attend import Call, bounds  # noqa: E402

B, K, V, HEADS, KV, D, PAGE, LAYERS = 4, 3, 1501, 6, 2, 64, 4, 2
H = HEADS * D
N_PAGES, MAX_PAGES, N_SLOTS = 40, 12, 6


class Engine:
    """One target with a paged cache.  Keys, values and queries of a step come from outside."""

    def __init__(self, seed, e4m3=False):
        L = self.L = lib()
        rng = self.rng = np.random.default_rng(seed)
        self.sv = L.SpecVerify(B, K, V, L.SV_F32)
        self.codes = rng.integers(0, 256, (V, H // 2)).astype(np.uint8)
        s8 = rng.integers(119, 122, (V, H // 32)).astype(np.uint8)
        self.packed = torch.empty(self.sv.head_packed_bytes(H, L.SV_W4_FP4, 32), dtype=torch.uint8, device=DEV)
        self.sv.head_pack(L.make_head_pack_args(hidden=H, format=L.SV_W4_FP4, group=32, weights=up(self.codes), weight_stride=H // 2,
                                                scales=up(s8), scale_stride=H // 32, packed=self.packed))
        torch.cuda.synchronize()
        i32 = dict(dtype=torch.int32, device=DEV)
        self.o = C.Pages(N_SLOTS, N_PAGES, PAGE, MAX_PAGES)
        self.table, self.lengths = torch.empty((N_SLOTS, MAX_PAGES), **i32), torch.empty(N_SLOTS, **i32)
        self.counts, self.refs, self.free = torch.empty(N_SLOTS, **i32), torch.empty(N_PAGES, **i32), torch.empty(2, **i32)
        self.cache = L.make_cache(n_slots=N_SLOTS, n_pages=N_PAGES, page_size=PAGE, max_pages=MAX_PAGES, page_table=self.table,
                                  lengths=self.lengths, page_counts=self.counts, page_refs=self.refs, free_pages=self.free)
        kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        self.pools = torch.full((2 * LAYERS, N_PAGES, KV, PAGE, D), float("nan"), dtype=torch.float32).to(kind).to(DEV)
        self.kv = [L.make_kv(kv_heads=KV, head_dim=D, type=L.SV_KV_E4M3 if e4m3 else L.SV_KV_BF16, keys=self.pools[2 * i],
                             values=self.pools[2 * i + 1], strides=(KV * PAGE * D, PAGE * D, D)) for i in range(LAYERS)]
        self.slots = torch.tensor([2, 5, 0, 3], **i32)
        self.qkv = torch.zeros((LAYERS, B, K + 1, HEADS + 2 * KV, D), dtype=torch.bfloat16, device=DEV)
        self.att = torch.zeros((LAYERS, B, K + 1, HEADS, D), dtype=torch.bfloat16, device=DEV)
        self.logits = torch.zeros((B, K + 1, V), device=DEV)
        self.draft = torch.zeros((B, K), **i32)
        self.u = torch.zeros((B, K + 1), device=DEV)
        self.acc, self.out, self.vl = torch.zeros(B, **i32), torch.zeros((B, K + 1), **i32), torch.zeros(B, **i32)
        self.hist_counts, self.hist_seen = torch.zeros((N_SLOTS, V), **i32), torch.zeros((N_SLOTS, (V + 31) // 32), **i32)
        self.granted, self.status = torch.zeros(B, **i32), torch.zeros(8, **i32)
        self.copies = torch.zeros((B, 2), **i32)
        self.attend_args = []
        for i in range(LAYERS):
            a = L.make_attend_args(B, K + 1, cache=self.cache, kv=self.kv[i], slots=self.slots, heads=HEADS, queries=self.qkv[i],
                                   query_strides=self._strides(), outputs=self.att[i], output_strides=((K + 1) * H, H, D),
                                   scale=D ** -0.5, device_status=self.status[3 + i:])
            self.attend_args.append(a)
        self.work = torch.empty(self.sv.attend_workspace_bytes(self.attend_args[0]), dtype=torch.uint8, device=DEV)
        for a in self.attend_args:
            a.workspace, a.workspace_bytes = self.work.data_ptr(), self.work.numel()
        self.sv.pages(L.make_pages_args(0, kind=L.SV_PAGES_CLEAR, cache=self.cache))
        self.held = [[[], []] for _ in range(B * LAYERS)]  # what each sequence's layers hold, fp64

    def _strides(self):
        row = (HEADS + 2 * KV) * D
        return (K + 1) * row, row, D

    def inputs(self):
        """A step's projections, drafted tokens and random numbers."""
        self.qkv.copy_(bf16(self.rng.standard_normal(self.qkv.shape)))
        self.draft.copy_(torch.from_numpy(self.rng.integers(0, V, (B, K)).astype(np.int32)))
        self.u.copy_(torch.from_numpy(self.rng.random((B, K + 1)).astype(np.float32)))

    def prompts(self, n):
        """Fills the sequences with prompts of n tokens, n - 1 rows at a time or fewer."""
        L = self.L
        last = up(np.asarray(n, np.int32) - 1)
        rows = max(n)
        self.sv.pages(L.make_pages_args(B, kind=L.SV_PAGES_RESERVE, cache=self.cache, slots=self.slots, rows=rows, last_row=last))
        x = bf16(self.rng.standard_normal((LAYERS, B, rows, 2, KV, D)))
        dev = x.to(DEV)
        for i in range(LAYERS):
            self.sv.append(L.make_append_args(B, rows, cache=self.cache, kv=self.kv[i], slots=self.slots, last_row=last,
                                              keys=dev[i], values=dev[i].data_ptr() + 2 * KV * D,
                                              strides=(rows * 2 * KV * D, 2 * KV * D, D)))
            for b in range(B):
                for w in (0, 1):
                    self.held[b * LAYERS + i][w] = list(x[i, b, :n[b], w].double().numpy())
        self.sv.pages(L.make_pages_args(B, kind=L.SV_PAGES_COMMIT, cache=self.cache, slots=self.slots, rows=rows, last_row=last))
        slots = self.slots.tolist()
        assert self.o.reserve(slots, n)[0] == [1] * B and self.o.commit(slots, n) == 0
        torch.cuda.synchronize()

    def step(self, stream=None):
        L, sv = self.L, self.sv
        where = dict(cache=self.cache, slots=self.slots)
        sv.pages(L.make_pages_args(B, kind=L.SV_PAGES_RESERVE, rows=K + 1, granted=self.granted, device_status=self.status[:1], **where), stream)
        for i in range(LAYERS):
            k = self.qkv[i].data_ptr() + 2 * H
            sv.append(L.make_append_args(B, K + 1, kv=self.kv[i], keys=k, values=k + 2 * KV * D, strides=self._strides(),
                                         device_status=self.status[1 + i:], **where), stream)
            sv.attend(self.attend_args[i], stream)
        sv.head(L.make_head_args(B * (K + 1), hidden=H, format=L.SV_W4_FP4, group=32, packed=self.packed, hidden_states=self.att[-1],
                                 hidden_stride=H, logits=self.logits, logits_stride=V), stream)
        sv.run(L.make_args(B, K, target=self.logits, target_strides=((K + 1) * V, V), tokens=self.draft, uniforms=self.u, temperature=1.0,
                           draft_mode=L.SV_DRAFT_ONEHOT, accepted_len=self.acc, out_tokens=self.out, verify_len_out=self.vl,
                           device_status=self.status[5:]), stream)
        sv.history(L.make_history_args(B, tokens=self.out, token_stride=K + 1, max_tokens=K + 1, kind=L.SV_HISTORY_OUTPUT, slots=self.slots,
                                       counts=self.hist_counts, seen=self.hist_seen, n_slots=N_SLOTS, device_status=self.status[6:]), stream)
        sv.pages(L.make_pages_args(B, kind=L.SV_PAGES_COMMIT, rows=K + 1, last_row=self.acc, device_status=self.status[7:], **where), stream)

    def state(self):
        return [self.table, self.lengths, self.counts, self.refs, self.free, self.hist_counts, self.hist_seen, self.pools]

    def outputs(self):
        return self.state()[:-1] + [self.att, self.logits, self.acc, self.out, self.granted, self.status]

    def check_pages(self):
        torch.cuda.synchronize()
        for t, x in zip((self.table, self.lengths, self.counts, self.refs, self.free),
                        (self.o.table, self.o.lengths, self.o.counts, self.o.refs, self.o.free_words().view(np.int32))):
            assert np.array_equal(t.cpu().numpy(), x)

    def check_step(self):
        torch.cuda.synchronize()
        assert self.status.tolist() == [0] * 8 and self.granted.tolist() == [1] * B
        slots, acc = self.slots.tolist(), self.acc.tolist()
        for b in range(B):
            for i in range(LAYERS):
                new = self.qkv[i, b].double().cpu().numpy()
                k, v = (np.array(self.held[b * LAYERS + i][w] + list(new[:, HEADS + w * KV:HEADS + (w + 1) * KV])) for w in (0, 1))
                start = len(k) - K - 1
                assert start == int(self.o.lengths[slots[b]])
                o, l, size, extra = C.attend(new[:, :HEADS], k, v, start, D ** -0.5)
                tol, _ = bounds(D, len(k), o, l, size, extra)
                assert (np.abs(self.att[i, b].double().cpu().numpy() - o) <= tol).all()
                for w in (0, 1):  # accepted rows stay
                    self.held[b * LAYERS + i][w] += list(new[:acc[b] + 1, HEADS + w * KV:HEADS + (w + 1) * KV])
        o = O.verify(self.logits.cpu().numpy(), None, self.draft.cpu().numpy(), self.u.cpu().numpy(), 1.0, dtype=O.F32, draft_mode=O.DRAFT_ONEHOT)
        ok = o.margin == 0
        assert np.array_equal(np.array(acc)[ok], o.accepted_len[ok])
        assert self.o.reserve(slots, [K + 1] * B)[1] == 0 and self.o.commit(slots, [a + 1 for a in acc]) == 0
        self.check_pages()


def test_steps_call_by_call():
    e = Engine(21)
    e.prompts([9, 1, 16, 4])
    for _ in range(3):
        e.inputs()
        # drafted tokens that verification takes often: the head's own choice
        e.step()
        e.check_step()


def test_accepted_rows_are_kept_and_rejected_ones_overwritten():
    e = Engine(22)
    e.prompts([5, 3, 8, 2])
    lengths = []
    for _ in range(4):
        e.inputs()
        save = [t.clone() for t in e.state()]
        e.step()
        torch.cuda.synchronize()
        # what the first pass would emit is drafted: all of it is accepted
        first = e.out[:, 0].clone()
        for t, was in zip(e.state(), save):
            t.copy_(was)
        e.draft[:, 0] = first
        e.u.fill_(1e-6)
        e.step()
        e.check_step()
        lengths.append(e.acc.tolist())
    assert max(max(x) for x in lengths) >= 1


def test_a_step_on_another_stream_and_replayed():
    e = Engine(23, e4m3=True)
    e.prompts([9, 2, 7, 4])
    e.inputs()
    start = [t.clone() for t in e.state()]

    def restore():
        for t, was in zip(e.state(), start):
            t.view(torch.uint8).copy_(was.view(torch.uint8))
        e.att.fill_(7.0)
        e.status.fill_(-3)
    restore()
    e.step()
    torch.cuda.synchronize()
    want = [t.clone() for t in e.outputs()]
    restore()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    e.step(side.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(e.outputs(), want))
    restore()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        e.step()
    for k in range(4):
        restore()
        if k == 2:  # eager work of the same handle and buffers between two replays
            e.step()
            restore()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(e.outputs(), want)), k
        _ = torch.ones(1000, device=DEV).sum().item()


def test_fork_shares_pages_and_copies_the_last():
    e = Engine(24)
    L = e.L
    e.prompts([9, 1, 16, 4])
    slots = e.slots.tolist()
    new, src = [1, 4, -1, -1], [2, 0, 0, 0]  # of 9 and of 16 tokens
    dev = [up(np.asarray(x, np.int32)) for x in (new, src)]
    e.sv.pages(L.make_pages_args(B, kind=L.SV_PAGES_FORK, cache=e.cache, slots=dev[0], from_slots=dev[1], granted=e.granted, copies=e.copies,
                                 max_copies=B))
    size = KV * PAGE * D * 2
    e.sv.pages_copy(L.make_pages_copy_args(B, copies=e.copies, pools=e.pools, n_pools=2 * LAYERS, pool_stride=N_PAGES * size, page_stride=size,
                                           page_bytes=size, n_pages=N_PAGES))
    assert e.o.fork(new, src)[0] == e.granted.tolist() == [1, 1, 0, 0]
    e.check_pages()
    # the forks attend as their sources do, and what they append does not reach these
    e.inputs()
    e.qkv[:, 1] = e.qkv[:, 0]
    e.qkv[:, 3] = e.qkv[:, 2]
    e.slots.copy_(torch.tensor([2, 1, 0, 4], dtype=torch.int32))
    e.step()
    torch.cuda.synchronize()
    assert e.status.tolist() == [0] * 8
    assert torch.equal(e.att[:, 0], e.att[:, 1]) and torch.equal(e.att[:, 2], e.att[:, 3])
    shared = [int(p) for p in e.table[1].tolist() if p in e.table[2].tolist() and p >= 0]
    assert len(shared) == 2 and slots[0] == 2


def test_compacted_pages_hold_the_same():
    e = Engine(25)
    L = e.L
    e.prompts([9, 14, 16, 4])
    one = up(np.array([5], np.int32))
    e.sv.pages(L.make_pages_args(1, kind=L.SV_PAGES_RELEASE, cache=e.cache, slots=one))
    e.inputs()
    e.slots[1] = -1
    moves = torch.zeros((20, 2), dtype=torch.int32, device=DEV)
    size = KV * PAGE * D * 2
    a = e.attend_args[0]

    def attend():  # over what is committed: the last row of it
        a.rows, a.row0 = 1, 0
        e.lengths.sub_(1)
        e.sv.attend(a)
        e.lengths.add_(1)
        torch.cuda.synchronize()
        return e.att[0][:, 0][[0, 2, 3]].clone()
    before = attend()
    e.sv.pages(L.make_pages_args(0, kind=L.SV_PAGES_COMPACT, cache=e.cache, copies=moves, max_copies=20))
    e.sv.pages_copy(L.make_pages_copy_args(20, copies=moves, pools=e.pools, n_pools=2 * LAYERS, pool_stride=N_PAGES * size, page_stride=size,
                                           page_bytes=size, n_pages=N_PAGES))
    assert (moves[:, 0] >= 0).sum() >= 3
    for src in moves[:, 0].tolist():  # what was left may be anything
        if src >= 0:
            e.pools[:, src] = float("nan")
    assert torch.equal(attend(), before) and torch.isfinite(before).all()
    assert int(e.table.max()) == int((e.refs > 0).sum()) - 1


def test_two_calls_at_once_and_two_graphs_with_workspaces_of_their_own():
    a, b = Call(101, [3000, 700, 64], 4, group=8, D=128), Call(102, [2500, 31, 1500], 4, group=8, D=128)
    wa, wb = a.run().result(), b.run().result()
    assert a.bytes and b.bytes
    b.sv = a.sv  # one handle
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        a.out.fill_(7.0), b.out.fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(4):
            a.run(s1.cuda_stream)
            b.run(s2.cuda_stream)
        torch.cuda.synchronize()
        assert all(np.array_equal(x, y) for x, y in zip(a.result() + b.result(), wa + wb))
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for _ in range(3):
        a.out.fill_(7.0), b.out.fill_(7.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(x, y) for x, y in zip(a.result() + b.result(), wa + wb))


def test_pools_past_4_gb():
    """The same tokens in pages at the far end of a large pool: the same results, and appended at the same places."""
    L = lib()
    small = Call(103, [700, 90], 3, group=4, kv=8, D=128, page=128).run()
    want = small.check()
    p = small.paged
    far = 20_000  # pages of 256 KB
    shift = far - p.n_pages
    pools = [torch.empty((far, p.pools[0].shape[1]), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for pool, t in zip(pools, p.dev):
        pool[shift:] = t
    table = up(np.where(p.table >= 0, p.table + shift, -1).astype(np.int32))
    cache = L.make_cache(n_slots=p.n_slots, n_pages=far, page_size=p.page, max_pages=p.max_pages, page_table=table, lengths=p.d["lengths"],
                         page_counts=p.d["counts"])
    kv = L.make_kv(kv_heads=p.kv, head_dim=p.D, type=L.SV_KV_BF16, keys=pools[0], values=pools[1], strides=p.strides)
    small.args.cache, small.args.kv = cache, kv
    small.out.fill_(7.0)
    got = small.run().result()
    assert all(np.array_equal(x, y) for x, y in zip(got, want))
    x = bf16(np.random.default_rng(0).standard_normal((2, 3, 2, 8, 128)))
    dev = x.to(DEV)
    small.sv.append(L.make_append_args(2, 3, cache=cache, kv=kv, slots=p.d["slots"], keys=dev, values=dev.data_ptr() + 2 * 1024,
                                       strides=(3 * 2048, 2048, 128)))
    for b in range(2):
        for r in range(3):
            t = int(p.lengths[p.slots[b]]) + r
            page = int(table[int(p.slots[b]), t // 128])
            for w in (0, 1):
                assert torch.equal(pools[w][page].view(8, 128, 128)[:, t % 128].cpu(), x[b, r, w])


def test_tables_past_2_gb_of_entries():
    """Slots whose entries lie past 2^31 in the table, pages of one token."""
    L = lib()
    small = Call(104, [50, 9], 2, page=1, waste=0.0).run()
    want = small.check()
    p = small.paged
    wide = 1 << 30
    table = torch.empty(4 * wide, dtype=torch.int32, device=DEV)
    slots = [3, 2]
    for b, s in enumerate(slots):
        table[s * wide:s * wide + p.max_pages] = up(p.table[p.slots[b]])
    lengths, counts = (up(np.zeros(4, np.int32)) for _ in range(2))
    for b, s in enumerate(slots):
        lengths[s], counts[s] = int(p.lengths[p.slots[b]]), int(p.counts[p.slots[b]])
    refs = torch.zeros(p.n_pages, dtype=torch.int32, device=DEV)
    for b in range(2):
        refs[up(p.table[p.slots[b]][:p.counts[p.slots[b]]]).long()] = 1
    free = torch.zeros((p.n_pages + 31) // 32, dtype=torch.int32, device=DEV)
    bits = np.packbits(np.pad(refs.cpu().numpy() == 0, (0, -p.n_pages % 32)), bitorder="little").view(np.int32)
    free.copy_(torch.from_numpy(bits))
    cache = L.make_cache(n_slots=4, n_pages=p.n_pages, page_size=1, max_pages=wide, page_table=table, lengths=lengths, page_counts=counts,
                         page_refs=refs, free_pages=free)
    dev = up(np.asarray(slots, np.int32))
    small.args.cache, small.args.slots = cache, dev.data_ptr()
    small.out.fill_(7.0)
    got = small.run().result()
    assert all(np.array_equal(x, y) for x, y in zip(got, want))
    # the rows are given up and their pages come back, the lowest first
    sv, status = small.sv, torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.pages(L.make_pages_args(2, kind=L.SV_PAGES_COMMIT, cache=cache, slots=dev, rows=0, device_status=status))
    assert counts.tolist() == [0, 0, 9, 50] and status.item() == 0
    lowest = (refs == 0).nonzero()[0].item()
    sv.pages(L.make_pages_args(2, kind=L.SV_PAGES_RESERVE, cache=cache, slots=dev, rows=1))
    assert table[3 * wide + 50].item() == lowest and counts.tolist() == [0, 0, 10, 51]


def test_copies_in_pools_past_4_gb():
    L = lib()
    n_pages, size = 70_000, 65_536
    pools = torch.empty((2, n_pages, size // 4), dtype=torch.int32, device=DEV)
    pools[:, 3] = 11
    pools[1, 69_999] = 12
    pairs = up(np.array([[3, 69_998], [69_999, 2]], np.int32))
    sv = L.SpecVerify(1, 1, 100, L.SV_BF16)
    sv.pages_copy(L.make_pages_copy_args(2, copies=pairs, pools=pools, n_pools=2, pool_stride=n_pages * size, page_stride=size, page_bytes=size,
                                         n_pages=n_pages))
    assert (pools[:, 69_998] == 11).all() and (pools[1, 2] == 12).all()


def test_a_very_long_sequence():
    """200000 tokens of one sequence, against fp64."""
    L = lib()
    T, rows, page, d = 200_000, 2, 64, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    n_pages = T // page + 1
    order = torch.randperm(n_pages, generator=g, device=DEV)
    k, v = (torch.randn((n_pages * page, d), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = (3 * torch.randn((rows, 2, d), generator=g, device=DEV)).to(torch.bfloat16)
    pools = [torch.empty((n_pages, 1, page, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for pool, x in zip(pools, (k, v)):
        pool[order] = x.view(n_pages, 1, page, d)
    table, lengths = order.to(torch.int32), up(np.array([T - rows], np.int32))
    cache = L.make_cache(n_slots=1, n_pages=n_pages, page_size=page, max_pages=n_pages, page_table=table, lengths=lengths)
    kv = L.make_kv(kv_heads=1, head_dim=d, type=L.SV_KV_BF16, keys=pools[0], values=pools[1], strides=(page * d, page * d, d))
    out, lse = torch.zeros_like(q), torch.zeros((rows, 2), device=DEV)
    sv = L.SpecVerify(1, 4, 100, L.SV_BF16)
    a = L.make_attend_args(1, rows, cache=cache, kv=kv, heads=2, queries=q, query_strides=(0, 2 * d, d), outputs=out,
                           output_strides=(0, 2 * d, d), lse=lse, scale=0.125)
    work = torch.empty(sv.attend_workspace_bytes(a), dtype=torch.uint8, device=DEV)
    a.workspace, a.workspace_bytes = work.data_ptr(), work.numel()
    sv.attend(a)
    for r in range(rows):
        seen = T - rows + r + 1
        kk, vv = k[:seen].double(), v[:seen].double()
        for h in range(2):
            s = kk @ q[r, h].double() * 0.125
            l = torch.logsumexp(s, 0)
            w = torch.exp(s - l)
            o, size = w @ vv, w @ vv.abs()
            terms = 0.125 * (kk.abs() @ q[r, h].double().abs()).max().item()
            tol, ltol = bounds(d, seen, o.cpu().numpy()[None], np.array([l.item()]), size.cpu().numpy()[None],
                               (np.array([terms]), np.array([s.abs().max().item()])))
            assert (np.abs(out[r, h].double().cpu().numpy() - o.cpu().numpy()) <= tol[0]).all()
            assert abs(lse[r, h].item() - l.item()) <= ltol[0]


def test_many_sequences():
    """More sequences than a launch takes, of every age, padded ones among them."""
    rng = np.random.default_rng(7)
    lengths = np.where(rng.random(700) < 0.02, 600, rng.integers(0, 40, 700))
    c = Call(105, list(lengths), 2, kv=1, group=3, page=8, last_row=list(rng.integers(-1, 3, 700)))
    c.run().check()
