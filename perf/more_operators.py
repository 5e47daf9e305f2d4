"""The target's cache around draft verification, as its operators are measured:
the attention of a drafted block over a paged key-value cache, the storing of
the block's keys and values in its pages, and the pages' own bookkeeping
(reserving, committing, forking, releasing, compacting, copying).

``run`` computes each in its plain form (elementary torch operations in 32
bits, rounded once) or, with ``own`` set, through the library's entry points.
``exact`` computes the same from the definition in 64 bits.

The operators, with ``len`` the tokens that a sequence's slot holds and token t
of it at place t % page_size of page table[slot][t // page_size]:

- attend: row r of a sequence stands at position p = len + row0 + r and sees the
  positions t <= p (with a window: t > p - window). For head h and its
  key-value head h // (heads / kv_heads),
    s_t = scale * <q, k_t>,  out = sum_t exp(s_t - lse) v_t,
    lse = log sum_t exp(s_t)
- append: row r's keys and values go to position len + row0 + r; in 8 bits they
  are held as e4m3(x / scale) with one scale per key-value head.
- pages: reserve gives every sequence the pages its next rows need, the lowest
  free ones first, in the order of the sequences; commit moves a slot's length
  past its first rows and gives the pages behind it back; release empties slots;
  fork gives a slot the pages of another: full ones are shared, the last one
  is copied to a page of its own; compact moves the highest pages to the lowest
  free ones. A page is free where no table names it.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one request, one token, a short conversation: nothing but latency
        dict(name="attend one token", op="attend", B=1, rows=1, row0=0, packed=False, least=1000, most=1000, heads=32,
             kv=8, D=128, e4m3=False, page=16, by_token=False, window=0),
        # one request, one token, a whole code base in its prompt: split over the length
        dict(name="attend one long request", op="attend", B=1, rows=1, row0=0, packed=False, least=131000, most=131000,
             heads=32, kv=8, D=128, e4m3=False, page=16, by_token=False, window=0),
        # a drafting step: the third drafted token of a batch of all ages, no keys shared
        dict(name="attend a drafting step", op="attend", B=64, rows=1, row0=2, packed=False, least=100, most=4000,
             heads=16, kv=16, D=64, e4m3=False, page=32, by_token=True, window=0),
        # an ordinary verify batch over a cache in 8 bits
        dict(name="attend a verify batch", op="attend", B=64, rows=9, row0=0, packed=False, least=200, most=8000,
             heads=32, kv=8, D=128, e4m3=True, page=32, by_token=False, window=0),
        # the largest verify batch: every row of a block of 16
        dict(name="attend a large batch", op="attend", B=256, rows=17, row0=0, packed=False, least=500, most=4000,
             heads=64, kv=8, D=128, e4m3=False, page=16, by_token=False, window=0),
        # rows packed by admission, a layer with a window, seven heads to a key head
        dict(name="attend packed rows", op="attend", B=100, rows=5, row0=0, packed=True, least=1, most=6000, heads=28,
             kv=4, D=256, e4m3=False, page=64, by_token=True, window=1024),
        # the keys and values of a verify batch's rows, of one layer
        dict(name="append a step", op="append", B=256, rows=17, row0=0, packed=False, least=500, most=4000, kv=8, D=128,
             e4m3=False, page=16, by_token=False),
        # the keys and values of whole prompts, of one layer, to 8 bits
        dict(name="append prompts", op="append", B=8, rows=8192, row0=0, packed=True, least=0, most=0, kv=8, D=128,
             e4m3=True, page=32, by_token=True),
        # a small batch is admitted anew: its old pages go, its prompts' pages come
        dict(name="admit a batch", op="admit", B=16, slots=64, rows=2000, pages=6000, page=16, others=0.5),
        # a large batch with long prompts in a large pool
        dict(name="admit a large batch", op="admit", B=256, slots=512, rows=16000, pages=600_000, page=16, others=0.5),
        # several answers to every prompt: its pages shared, the last one copied in every layer
        dict(name="fork a batch", op="fork", B=256, parents=64, rows=17, prompt=2000, pages=12000, page=16, layers=8,
             kv=8, D=64),
        # after a busy hour the pool is packed again
        dict(name="compact a pool", op="compact", slots=256, prompt=1200, pages=16384, page=16, layers=4, kv=8, D=64,
             held=0.55, moves=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend"] * 6 + ["append"] * 3 + ["admit", "fork", "compact"])
    page = rng.choice([8, 16, 32, 64, 128])
    if op == "admit":
        B = _log(rng, 1, 256)
        rows = _log(rng, 1, 16000)
        pages = 2 * B * (rows // page + 2) + rng.randint(0, 5000)
        return dict(op=op, B=B, slots=B + rng.randint(0, 256), rows=rows, pages=pages, page=page,
                    others=round(rng.uniform(0.1, 0.7), 2))
    if op == "fork":
        B = _log(rng, 1, 256)
        parents = _log(rng, 1, 64)
        prompt = _log(rng, 1, 4000)
        rows = rng.randint(1, 17)
        pages = parents * (prompt // page + 1) + B * (17 // page + 4) + rng.randint(0, 1000)
        return dict(op=op, B=B, parents=parents, rows=rows, prompt=prompt, pages=pages, page=page,
                    layers=rng.randint(1, max(1, min(8, 1_200_000_000 // (pages * page * 1024 * 2)))), kv=8, D=64)
    if op == "compact":
        slots = _log(rng, 1, 256)
        prompt = _log(rng, 1, 1500)
        held = round(rng.uniform(0.2, 0.8), 2)
        pages = int(slots * (prompt // page + 1) / held) + 1
        return dict(op=op, slots=slots, prompt=prompt, pages=pages, page=page,
                    layers=rng.randint(1, max(1, min(8, 1_200_000_000 // (pages * page * 1024 * 2)))), kv=8, D=64, held=held,
                    moves=_log(rng, 1, 4096))
    D = rng.choice([64, 128, 256])
    kv = rng.choice([1, 2, 4, 8, 16])
    e4m3 = rng.random() < 0.4
    by_token, packed, row0 = rng.random() < 0.4, rng.random() < 0.3, rng.choice([0, 0, rng.randint(1, 16)])
    shape = dict(page=page, by_token=by_token, kv=kv, D=D, e4m3=e4m3)
    if op == "append":
        rows = _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(256, 130_000_000 // (rows * kv * D))))
        most = _log(rng, 1, max(1, min(4000, 1_000_000_000 // (B * kv * D))))
        return dict(op=op, B=B, rows=rows, row0=row0, packed=packed, least=rng.randint(0, most), most=most, **shape)
    rows = rng.choice([1, 1, _log(rng, 1, 17), _log(rng, 1, 17)])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    group = max(1, min(group, 64 // kv))
    most = _log(rng, 1, 131000)
    # no more than the largest listed one has to read, and to multiply
    B = max(1, min(256, 800_000_000 // (most * kv * D), 60_000_000_000 // (most * kv * D * group * rows)))
    B = _log(rng, 1, B)
    least = most if B == 1 else _log(rng, 1, most)
    return dict(op=op, B=B, rows=rows, row0=row0, packed=packed, least=least, most=most, heads=kv * group,
                window=rng.choice([0, 0, _log(rng, 1, 4096)]), **shape)


# ------------------------------------------------------------------ inputs

def _words(bits):
    """bool [n] -> int32 [ceil(n / 32)], bit i % 32 of word i / 32."""
    n = bits.shape[0]
    full = torch.zeros((n + 31) // 32 * 32, dtype=torch.int32, device=bits.device)
    full[:n] = bits
    w = (full.view(-1, 32) << torch.arange(32, dtype=torch.int32, device=bits.device)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _rows(case, r, s):
    """How many rows each sequence has, and where they lie."""
    B, rows = case["B"], case["rows"]
    n = np.full(B, rows)
    if case["packed"]:
        n = r.permutation(np.resize(np.linspace((rows + 1) // 2 if rows > 64 else 1, rows, 5).astype(int), B))  # as many in all, whatever the seed
        s["row_off"] = _dev(np.concatenate([[0], np.cumsum(n)]))
    s["n"], s["n_dev"], s["most_rows"] = n, _dev(n), int(n.max())
    s["seq"] = _dev(np.repeat(np.arange(B), n))
    s["place"] = _dev(np.concatenate([np.arange(k) for k in n]))
    return n


def _cache(case, r, s, need):
    """A pool whose pages were given and taken for a long time: a slot's lie anywhere."""
    B, page = case["B"], case["page"]
    held = (need + page - 1) // page
    used = int(held.sum())
    n_pages, n_slots, max_pages = used + used // 8 + 5, B + 3, int(held.max()) + 2
    slots = r.permutation(n_slots)[:B]
    pages = r.permutation(n_pages)[:used]
    table = np.full((n_slots, max_pages), -1)
    there = np.arange(max_pages)[None, :] < held[:, None]
    mine = np.full((B, max_pages), -1)
    mine[there] = pages
    table[slots] = mine
    lengths, counts = np.zeros(n_slots, np.int64), np.zeros(n_slots, np.int64)
    lengths[slots], counts[slots] = s["len"], held
    s.update(table=_dev(table.astype(np.int32)), lengths=_dev(lengths.astype(np.int32)), counts=_dev(counts.astype(np.int32)),
             slots=_dev(slots.astype(np.int32)), n_pages=n_pages, n_slots=n_slots, max_pages=max_pages)


def _to_e4m3(x, scale):
    return (x / scale).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)


def _pools(case, g, s, fill):
    """One layer's pages: element (page, head, token, d); by token or by head within a page."""
    kv, D, page = case["kv"], case["D"], case["page"]
    shape = (s["n_pages"], page, kv, D) if case["by_token"] else (s["n_pages"], kv, page, D)
    for name in ("keys", "values"):
        if case["e4m3"]:
            scale = (0.5 + torch.rand(kv, generator=g, device=DEV)) * 0.03
            s[name + "_scale"] = scale
        x = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
        if fill:
            x.normal_(0.0, 1.0, generator=g)
        if case["e4m3"]:
            x = torch.cat([_to_e4m3(part.float(), scale.view((1, 1, kv, 1) if case["by_token"] else (1, kv, 1, 1)))
                           for part in x.split(max(1, 200_000_000 // (kv * page * D)))])
        s[name] = x


def _lengths(case, r):
    lo, hi = case["least"], case["most"]
    if hi == 0:
        return np.zeros(case["B"], np.int64)
    n = np.exp(np.linspace(math.log(max(lo, 1)), math.log(hi), case["B"])).round().astype(np.int64)  # as many in all, whatever the seed
    return r.permutation(n)


def _inputs_rows(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng(seed)
    s = {}
    n = _rows(case, r, s)
    s["len"] = _lengths(case, r)
    s["len_dev"] = _dev(s["len"])
    total = s["len"] + case["row0"] + n
    s["most"] = int(total.max())
    _cache(case, r, s, total)
    _pools(case, g, s, case["op"] == "attend")
    lead = (int(n.sum()),) if case["packed"] else (case["B"], case["rows"])
    kv, D = case["kv"], case["D"]
    if case["op"] == "append":
        # keys and values as a fused projection leaves them, side by side
        s["kv"] = torch.empty(lead + (2 * kv, D), dtype=torch.bfloat16, device=DEV).normal_(0.0, 1.0, generator=g)
        return s
    heads = case["heads"]
    q = torch.empty(lead + (heads, D), device=DEV).normal_(0.0, 2.0, generator=g)
    if D >= 64:  # a position that draws attention: some directions of a query are shared by many keys
        q[..., 3] += 4.0
    s["q"] = q.to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(D)
    return s


def _holdings(r, n_pages, held, max_pages):
    """Tables of slots that hold so many pages each, picked from all over the pool."""
    table = np.full((len(held), max_pages), -1)
    there = np.arange(max_pages)[None, :] < held[:, None]
    table[there] = r.permutation(n_pages)[:int(held.sum())]
    return table


def _inputs_pages(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng(seed)
    op, page, P = case["op"], case["page"], case["pages"]
    s = {}
    if op == "admit":
        B, slots = case["B"], case["slots"]
        lens = np.linspace((case["rows"] + 1) // 2, case["rows"], B).astype(np.int64)
        s["n"] = _dev(r.permutation(lens).astype(np.int32) - 1)  # the last row of each prompt
        order = r.permutation(slots)
        s["slots"] = _dev(order[:B].astype(np.int32))
        max_pages = (case["rows"] + page - 1) // page + 1
        # others hold their share of the pool, the admitted ones what their last requests held
        budget = int(P * case["others"])
        held = np.zeros(slots, np.int64)
        if slots > B:
            held[order[B:]] = np.minimum(max_pages, budget // (slots - B))
        left = max(0, (P - int(held.sum())) // B)
        held[order[:B]] = np.minimum(r.integers(0, max_pages + 1, B), left)
        lengths = held * page
    elif op == "fork":
        B, parents = case["B"], case["parents"]
        max_pages = (case["prompt"] + case["rows"] + page - 1) // page + 2
        slots = parents + B + 1
        order = r.permutation(slots)
        s["slots"] = _dev(order[parents:parents + B].astype(np.int32))
        s["from"] = _dev(order[:parents][np.arange(B) % parents].astype(np.int32))
        s["accepted"] = _dev(r.integers(0, case["rows"], B).astype(np.int32))
        lengths = np.zeros(slots, np.int64)
        lengths[order[:parents]] = r.permutation(np.linspace((case["prompt"] + 1) // 2, case["prompt"], parents).astype(np.int64))
        held = (lengths + page - 1) // page
    else:
        slots = case["slots"]
        max_pages = (case["prompt"] + page - 1) // page + 1
        lengths = r.permutation(np.linspace((case["prompt"] + 1) // 2, case["prompt"], slots).astype(np.int64))
        held = (lengths + page - 1) // page
        lengths[held.cumsum() > P] = 0
        held = (lengths + page - 1) // page
    table = _holdings(r, P, held, max_pages)
    refs = np.zeros(P, np.int64)
    refs[table[table >= 0]] = 1
    s.update(table=_dev(table.astype(np.int32)), lengths=_dev(lengths.astype(np.int32)), counts=_dev(held.astype(np.int32)),
             refs=_dev(refs.astype(np.int32)), n_slots=slots, max_pages=max_pages)
    s["free"] = _words(s["refs"] == 0)
    if op != "admit":  # all layers' keys and values, one pool after the other
        s["pools"] = torch.empty((2 * case["layers"], P, page * case["kv"] * case["D"]), dtype=torch.bfloat16, device=DEV)
        s["pools"].normal_(0.0, 1.0, generator=g)
    if op == "compact":
        s["start"] = [s[k].clone() for k in ("table", "refs", "free")]
    return s


def _inputs(case, seed):
    return _inputs_rows(case, seed) if case["op"] in ("attend", "append") else _inputs_pages(case, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        _prepare_own(case, s)
    return s


# ------------------------------------------------------------------ the library's calls

def _prepare_own(case, s):
    """What a user's program keeps: the handle, the output buffers, the
    workspace, and the argument structs that name them."""
    from draft_verification_amd import binding as B
    op = case["op"]
    if op in ("admit", "fork", "compact"):
        Bn = case.get("B", 1)
        s["sv"] = B.SpecVerify(Bn, 16, 1000, B.SV_BF16)
        cache = B.make_cache(n_slots=s["n_slots"], n_pages=case["pages"], page_size=case["page"], max_pages=s["max_pages"],
                             page_table=s["table"], lengths=s["lengths"], page_counts=s["counts"], page_refs=s["refs"],
                             free_pages=s["free"])
        s["granted"] = torch.zeros(Bn, dtype=torch.int32, device=DEV)

        def pages(kind, **more):
            return B.make_pages_args(Bn if kind != B.SV_PAGES_COMPACT else 0, kind=kind, cache=cache, **more)
        if op == "admit":
            s["args"] = [pages(B.SV_PAGES_RELEASE, slots=s["slots"]),
                         pages(B.SV_PAGES_RESERVE, slots=s["slots"], rows=case["rows"], last_row=s["n"], granted=s["granted"]),
                         pages(B.SV_PAGES_COMMIT, slots=s["slots"], rows=case["rows"], last_row=s["n"])]
            return
        moves = Bn if op == "fork" else case["moves"]
        s["copies"] = torch.zeros((moves, 2), dtype=torch.int32, device=DEV)
        if op == "fork":
            s["args"] = [pages(B.SV_PAGES_RELEASE, slots=s["slots"]),
                         pages(B.SV_PAGES_FORK, slots=s["slots"], from_slots=s["from"], granted=s["granted"],
                               copies=s["copies"], max_copies=moves),
                         pages(B.SV_PAGES_RESERVE, slots=s["slots"], rows=case["rows"]),
                         pages(B.SV_PAGES_COMMIT, slots=s["slots"], rows=case["rows"], last_row=s["accepted"])]
        else:
            s["args"] = [pages(B.SV_PAGES_COMPACT, copies=s["copies"], max_copies=moves)]
        size = 2 * s["pools"].shape[2]
        s["copy"] = B.make_pages_copy_args(moves, copies=s["copies"], pools=s["pools"], n_pools=s["pools"].shape[0],
                                           pool_stride=case["pages"] * size, page_stride=size, page_bytes=size,
                                           n_pages=case["pages"])
        return
    kv, D, page = case["kv"], case["D"], case["page"]
    s["sv"] = B.SpecVerify(case["B"], max(1, case["row0"] + min(case["rows"], 240) - 1), 1000, B.SV_BF16)
    cache = B.make_cache(n_slots=s["n_slots"], n_pages=s["n_pages"], page_size=page, max_pages=s["max_pages"],
                         page_table=s["table"], lengths=s["lengths"], page_counts=s["counts"])
    strides = (page * kv * D, D, kv * D) if case["by_token"] else (page * kv * D, page * D, D)
    held = B.make_kv(kv_heads=kv, head_dim=D, type=B.SV_KV_E4M3 if case["e4m3"] else B.SV_KV_BF16, keys=s["keys"],
                     values=s["values"], strides=strides, key_scales=s.get("keys_scale"), value_scales=s.get("values_scale"))
    where = dict(cache=cache, kv=held, slots=s["slots"], row0=case["row0"], row_offsets=s.get("row_off"))
    rows = s["most_rows"]
    if case["op"] == "append":
        row = 2 * kv * D
        s["args"] = B.make_append_args(case["B"], rows, keys=s["kv"], values=s["kv"].data_ptr() + 2 * kv * D,
                                       strides=(rows * row, row, D), **where)
        return
    row = case["heads"] * D
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(s["q"].shape[:-1], device=DEV)
    args = B.make_attend_args(case["B"], rows, heads=case["heads"], queries=s["q"], query_strides=(rows * row, row, D),
                              outputs=s["out"], output_strides=(rows * row, row, D), lse=s["lse"], scale=s["scale"],
                              window=case["window"], max_len=s["most"], **where)
    s["work"] = torch.empty(max(16, s["sv"].attend_workspace_bytes(args)), dtype=torch.uint8, device=DEV)
    args.workspace, args.workspace_bytes = s["work"].data_ptr(), s["work"].numel()
    s["args"] = args


def _run_own(s):
    op = s["case"]["op"]
    if op == "attend":
        s["sv"].attend(s["args"])
        return [s["out"], s["lse"]]
    if op == "append":
        s["sv"].append(s["args"])
        return [s["keys"], s["values"]]
    if op == "compact":  # every pass finds the same holes
        _again(s)
    for args in s["args"]:
        s["sv"].pages(args)
    if op == "admit":
        return [s[k] for k in ("table", "lengths", "counts", "refs", "free", "granted")]
    s["sv"].pages_copy(s["copy"])
    out = [s[k] for k in ("table", "lengths", "counts", "refs", "free", "copies", "pools")]
    return out + [s["granted"]] if op == "fork" else out


# ------------------------------------------------------------------ the plain forms

def _again(s):
    for k, was in zip(("table", "refs", "free"), s["start"]):
        s[k].copy_(was)


def _held(s, name, pages):
    """The tokens of the sequences' pages as float32 [B][kv][tokens][D]."""
    case = s["case"]
    x = s[name]
    B, P = pages.shape
    if case["e4m3"]:
        x = x.view(torch.uint8)
    x = x.index_select(0, pages.reshape(-1)).view((B, P) + tuple(x.shape[1:]))
    x = x.permute(0, 3, 1, 2, 4) if case["by_token"] else x.permute(0, 2, 1, 3, 4)
    if case["e4m3"]:
        x = x.contiguous().view(torch.float8_e4m3fn).float() * s[name + "_scale"].view(1, -1, 1, 1, 1)
    return x.float().reshape(B, case["kv"], P * case["page"], case["D"])


def _plain_attend(s):
    case = s["case"]
    B, kv, D, heads, page = case["B"], case["kv"], case["D"], case["heads"], case["page"]
    rows = s["most_rows"]
    q = s["q"].float()
    if case["packed"]:
        q = torch.zeros((B, rows, heads, D), device=DEV).index_put_((s["seq"], s["place"]), q)
    group = heads // kv
    q = q.view(B, rows, kv, group, D).permute(0, 2, 1, 3, 4).reshape(B, kv, rows * group, D)
    pages = s["table"].index_select(0, s["slots"].long())[:, :(s["most"] + page - 1) // page].long().clamp(min=0)
    at = torch.arange(pages.shape[1] * page, device=DEV)
    p = (s["len_dev"] + case["row0"])[:, None] + torch.arange(rows, device=DEV)
    sees = at <= p[..., None]
    if case["window"]:
        sees &= at > p[..., None] - case["window"]
    k = _held(s, "keys", pages)
    score = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(B, kv, rows, group, -1)
    del k
    score.masked_fill_(~sees[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    e = score.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    v = _held(s, "values", pages)
    there = at < (s["len_dev"] + case["row0"] + s["n_dev"])[:, None]
    v.masked_fill_(~there[:, None, :, None], 0.0)
    out = (e.view(B, kv, rows * group, -1) @ v).view(B, kv, rows, group, D) / total
    lse = (top + total.log()).squeeze(-1)
    out = out.permute(0, 2, 1, 3, 4).reshape(B, rows, heads, D)
    lse = lse.permute(0, 2, 1, 3).reshape(B, rows, heads)
    if case["packed"]:
        out, lse = out[s["seq"], s["place"]], lse[s["seq"], s["place"]]
    return [out.to(torch.bfloat16), lse.contiguous()]


def _plain_append(s):
    case = s["case"]
    kv, D, page = case["kv"], case["D"], case["page"]
    at = s["len_dev"].index_select(0, s["seq"]) + case["row0"] + s["place"]
    where = s["table"][s["slots"].long().index_select(0, s["seq"]), at // page].long()
    x = s["kv"].view(-1, 2, kv, D)
    for i, name in enumerate(("keys", "values")):
        new, pool = x[:, i], s[name]
        if case["e4m3"]:
            new = _to_e4m3(new.float(), s[name + "_scale"][:, None]).view(torch.uint8)
            pool = pool.view(torch.uint8)
        if case["by_token"]:
            pool[where, at % page] = new
        else:
            pool[where, :, at % page] = new
    return [s["keys"], s["values"]]


def _give_back(s, slots, keep):
    """The pages of the slots past the first `keep` go back."""
    table = s["table"].index_select(0, slots)
    at = torch.arange(table.shape[1], device=DEV)
    gone = (at >= keep[:, None]) & (at < s["counts"].index_select(0, slots)[:, None])
    s["refs"].index_add_(0, table.clamp(min=0).view(-1), gone.view(-1).to(torch.int32), alpha=-1)
    s["table"].index_copy_(0, slots, torch.where(gone, -1, table))
    s["counts"].index_copy_(0, slots, torch.minimum(keep, s["counts"].index_select(0, slots)))


def _lowest_free(s, need):
    """(the k-th lowest free page for every k, whether each sequence gets what it needs, what came before it)."""
    free = s["refs"] == 0
    rank = torch.where(free, free.cumsum(0) - 1, free.shape[0])
    kth = torch.zeros(free.shape[0] + 1, dtype=torch.int64, device=DEV)
    kth.index_put_((rank,), torch.arange(free.shape[0], device=DEV))
    upto = need.cumsum(0)
    return kth, (need == 0) | (upto <= free.sum()), upto - need


def _plain_reserve(s, slots, n):
    page = s["case"]["page"]
    held = s["counts"].index_select(0, slots).long()
    need = ((s["lengths"].index_select(0, slots) + n + page - 1) // page - held).clamp(min=0)
    kth, ok, before = _lowest_free(s, need)
    need = torch.where(ok, need, 0)
    at = torch.arange(s["max_pages"], device=DEV)
    new = (at >= held[:, None]) & (at < (held + need)[:, None])
    given = kth[torch.where(new, before[:, None] + at - held[:, None], 0)]
    s["table"].index_copy_(0, slots, torch.where(new, given.to(torch.int32), s["table"].index_select(0, slots)))
    s["refs"].index_add_(0, given.view(-1), new.view(-1).to(torch.int32))
    s["counts"].index_copy_(0, slots, (held + need).to(torch.int32))
    return ok.to(torch.int32)


def _plain_commit(s, slots, n):
    length = s["lengths"].index_select(0, slots) + n
    s["lengths"].index_copy_(0, slots, length)
    _give_back(s, slots, (length + s["case"]["page"] - 1) // s["case"]["page"])


def _plain_release(s, slots):
    _give_back(s, slots, torch.zeros_like(slots, dtype=torch.int32))
    s["lengths"].index_fill_(0, slots, 0)


def _plain_fork(s, slots, source):
    page = s["case"]["page"]
    length = s["lengths"].index_select(0, source)
    part = (length % page != 0).long()
    kth, ok, before = _lowest_free(s, part)
    full = length // page
    at = torch.arange(s["max_pages"], device=DEV)
    table = s["table"].index_select(0, source)
    shared = (at < full[:, None]) & ok[:, None]
    s["refs"].index_add_(0, table.clamp(min=0).view(-1), shared.view(-1).to(torch.int32))
    cut = (part > 0) & ok
    new = torch.where(cut, kth[torch.where(cut, before, 0)], 0)
    s["refs"].index_add_(0, new, cut.to(torch.int32))
    own_page = (at == full[:, None]) & cut[:, None]
    was = table.gather(1, full.long()[:, None])[:, 0]
    s["table"].index_copy_(0, slots, torch.where(own_page, new[:, None].to(torch.int32), torch.where(shared, table, -1)))
    s["counts"].index_copy_(0, slots, torch.where(ok, full + part, 0).to(torch.int32))
    s["lengths"].index_copy_(0, slots, torch.where(ok, length, 0))
    return ok.to(torch.int32), torch.stack([torch.where(cut, was, -1), torch.where(cut, new, -1).to(torch.int32)], 1)


def _plain_compact(s):
    case = s["case"]
    P, most = case["pages"], case["moves"]
    live = s["refs"] > 0
    n = live.sum()
    at = torch.arange(P, device=DEV)
    hole, far = ~live & (at < n), live & (at >= n)
    spare = most + 1
    # the i-th lowest hole and the i-th highest page
    low = torch.where(hole, hole.cumsum(0) - 1, spare).clamp(max=spare)
    high = torch.where(far, far.flip(0).cumsum(0).flip(0) - 1, spare).clamp(max=spare)
    to = torch.full((spare + 1,), -1, dtype=torch.int64, device=DEV).index_put_((low,), at)[:most]
    src = torch.full((spare + 1,), -1, dtype=torch.int64, device=DEV).index_put_((high,), at)[:most]
    moved = (torch.arange(most, device=DEV) < far.sum())
    to, src = torch.where(moved, to, -1), torch.where(moved, src, -1)
    moving = far & (high < most)
    new_place = torch.where(moving, to[high.clamp(max=most - 1)], at)
    table = s["table"]
    s["table"].copy_(torch.where(table >= 0, new_place[table.clamp(min=0).long()], -1))
    refs = s["refs"]
    s["refs"].copy_(torch.where(moving, 0, refs).index_add_(0, new_place, torch.where(moving, refs, 0)))
    return torch.stack([src, to], 1).to(torch.int32)


def _plain_copy(s, copies):
    """In every pool, page copies[i][0] goes to copies[i][1]."""
    src, to = copies[:, 0].long(), copies[:, 1].long()
    some = src >= 0
    src, to = torch.where(some, src, 0), torch.where(some, to, 0)
    # pairs of nothing copy page 0 to itself, as any pair that brings page 0's new contents does
    first = torch.where(to[None, :] == 0, some[None, :], False)
    src = torch.where(some, src, torch.where(first.any(), src[first[0].to(torch.int32).argmax()], 0))
    s["pools"].index_copy_(1, to, s["pools"].index_select(1, src))


def _plain_pages(s):
    case = s["case"]
    op = case["op"]
    if op == "compact":
        _again(s)
        copies = _plain_compact(s)
    else:
        slots = s["slots"].long()
        _plain_release(s, slots)
        if op == "admit":
            granted = _plain_reserve(s, slots, s["n"] + 1)
            _plain_commit(s, slots, torch.where(granted > 0, s["n"] + 1, 0))
        else:
            granted, copies = _plain_fork(s, slots, s["from"].long())
            _plain_reserve(s, slots, case["rows"])
            _plain_commit(s, slots, s["accepted"] + 1)
    s["free"].copy_(_words(s["refs"] == 0))
    state = [s[k] for k in ("table", "lengths", "counts", "refs", "free")]
    if op == "admit":
        return state + [granted]
    _plain_copy(s, copies)
    state += [copies, s["pools"]]
    return state + [granted] if op == "fork" else state


def _run_plain(s):
    op = s["case"]["op"]
    if op == "attend":
        return _plain_attend(s)
    return _plain_append(s) if op == "append" else _plain_pages(s)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def _mean_rows(case):
    rows = case["rows"]
    if not case["packed"]:
        return float(rows)
    return float(np.linspace((rows + 1) // 2 if rows > 64 else 1, rows, 5).astype(int).mean())


def work(case):
    op = case["op"]
    if op in ("attend", "append"):
        B, kv, D, rows = case["B"], case["kv"], case["D"], _mean_rows(case)
        held = 2.0 * kv * D * (1 if case["e4m3"] else 2)
        if op == "append":
            return {"bytes": B * rows * (held + 4.0 * kv * D), "flops": 2.0 * B * rows * kv * D}
        lens = _lengths(case, np.random.default_rng(0)) + case["row0"]
        sees = np.minimum(lens + rows / 2, case["window"]) if case["window"] else lens + rows / 2
        read = np.minimum(lens, case["window"]) + rows if case["window"] else lens + rows
        return {"bytes": float(read.sum()) * held + B * rows * case["heads"] * (4.0 * D + 4),
                "flops": 4.0 * rows * case["heads"] * D * float(sees.sum())}
    if op == "compact":
        live = case["slots"] * 0.75 * case["prompt"] / case["page"]
        moves = min(case["moves"], live * max(0.0, 1 - live / case["pages"]))
        table = case["slots"] * live / max(1, case["slots"]) * 8
        return {"bytes": table + case["pages"] * 4.125 + moves * case["layers"] * case["page"] * case["kv"] * case["D"] * 8.0,
                "flops": float(case["pages"])}
    given = case["B"] * 0.75 * (case["rows"] if op == "admit" else case["prompt"]) / case["page"]
    # a page given or taken: its table entry and its count, read and written
    small = case["pages"] / 4.0 + 2 * given * 12.0
    if op == "admit":
        return {"bytes": small, "flops": 2 * given}
    return {"bytes": small + case["B"] * case["layers"] * case["page"] * case["kv"] * case["D"] * 8.0, "flops": 2 * given}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_attend(s, case):
    B, kv, D, page = case["B"], case["kv"], case["D"], case["page"]
    group = case["heads"] // kv
    outs, lses = [], []
    table = s["table"].cpu().numpy()
    slots = s["slots"].tolist()
    first = np.concatenate([[0], np.cumsum(s["n"])])
    for b in range(B):
        n, start = int(s["n"][b]), int(s["len"][b]) + case["row0"]
        T = start + n
        low = max(0, start - case["window"] + 1) // page * page if case["window"] else 0
        pages = torch.from_numpy(table[slots[b]][low // page:(T + page - 1) // page].astype(np.int64)).to(DEV)
        q = (s["q"][first[b]:first[b + 1]] if case["packed"] else s["q"][b]).double()
        seen = []
        for name in ("keys", "values"):
            x = s[name][pages].double() if not case["e4m3"] else s[name].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
            x = x.flatten(0, 1) if case["by_token"] else x.permute(0, 2, 1, 3).flatten(0, 1)  # [tokens][kv][D]
            if case["e4m3"]:
                x = x * s[name + "_scale"].double()[:, None]
            seen.append(x[:T - low])
        p = start + torch.arange(n, device=DEV)[:, None]
        t = low + torch.arange(T - low, device=DEV)[None, :]
        out_of_sight = t > p
        if case["window"]:
            out_of_sight |= t <= p - case["window"]
        o, l = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=DEV)
        for h in range(kv):
            k, v = seen[0][:, h], seen[1][:, h]
            for i in range(h * group, (h + 1) * group):
                z = torch.mv(k, q[0, i])[None] if n == 1 else q[:, i] @ k.t()
                z = (z / math.sqrt(D)).masked_fill(out_of_sight, -math.inf)
                l[:, i] = torch.logsumexp(z, 1)
                o[:, i] = torch.exp(z - l[:, i:i + 1]) @ v
        outs.append(o)
        lses.append(l)
    if case["packed"]:
        return [torch.cat(outs), torch.cat(lses)]
    return [torch.stack(outs), torch.stack(lses)]


def _exact_e4m3(y):
    """The nearest value with 3 bits of fraction, exponents -6 to 8, ties to even."""
    y = y.clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _exact_append(s, case):
    page = case["page"]
    first = np.concatenate([[0], np.cumsum(s["n"])])
    slots = s["slots"].tolist()
    flat = s["kv"].view(-1, 2, case["kv"], case["D"])
    out = []
    for i, name in enumerate(("keys", "values")):
        pool = s[name].double() if not case["e4m3"] else s[name].float().double()
        for b in range(case["B"]):
            new = flat[first[b]:first[b + 1], i].double()
            if case["e4m3"]:
                new = _exact_e4m3(new / s[name + "_scale"].double()[:, None])
            t = int(s["len"][b]) + case["row0"] + torch.arange(int(s["n"][b]), device=DEV)
            pages = s["table"][slots[b]][t // page].long()
            if case["by_token"]:
                pool[pages, t % page] = new
            else:
                pool[pages, :, t % page] = new
        out.append(pool)
    return out


def _exact_pages(s, case):
    """One sequence and one page after the other."""
    page, op = case["page"], case["op"]
    table, lengths, counts, refs = ([list(x) for x in s["table"].tolist()], s["lengths"].tolist(), s["counts"].tolist(),
                                    s["refs"].tolist())
    copies, granted = [], []
    if op == "compact":
        live = sum(1 for c in refs if c)
        holes = [p for p in range(live) if not refs[p]]
        far = [p for p in range(len(refs) - 1, live - 1, -1) if refs[p]]
        copies = [list(x) for x in zip(far, holes)][:case["moves"]]
        to = dict(copies)
        table = [[to.get(p, p) for p in row] for row in table]
        for src, dst in copies:
            refs[dst], refs[src] = refs[src], 0
        copies += [[-1, -1]] * (case["moves"] - len(copies))
    else:
        slots = s["slots"].tolist()
        for slot in slots:
            for i in range(counts[slot]):
                refs[table[slot][i]] -= 1
                table[slot][i] = -1
            counts[slot] = lengths[slot] = 0
        free = iter([p for p in range(len(refs)) if not refs[p]])
        left = sum(1 for c in refs if not c)
        if op == "fork":
            for slot, source in zip(slots, s["from"].tolist()):
                L = lengths[source]
                copies.append([-1, -1])
                granted.append(int(L % page == 0 or left > 0))
                if not granted[-1]:
                    continue
                for i in range(L // page):
                    table[slot][i] = table[source][i]
                    refs[table[slot][i]] += 1
                if L % page:
                    new, left = next(free), left - 1
                    refs[new] = 1
                    table[slot][L // page] = new
                    copies[-1] = [table[source][L // page], new]
                counts[slot], lengths[slot] = -(-L // page), L
        rows = (s["n"] + 1).tolist() if op == "admit" else [case["rows"]] * case["B"]
        keep = rows if op == "admit" else (s["accepted"] + 1).tolist()
        asked, have, done = 0, left, []
        for slot, n in zip(slots, rows):
            need = max(0, -(-(lengths[slot] + n) // page) - counts[slot])
            asked += need
            done.append(int(need == 0 or asked <= have))
            if done[-1]:
                for _ in range(need):
                    new = next(free)
                    refs[new] = 1
                    table[slot][counts[slot]] = new
                    counts[slot] += 1
        if op == "admit":
            granted = done
        for slot, n, ok in zip(slots, keep, done):
            lengths[slot] += n if ok else 0
            for i in range(-(-lengths[slot] // page), counts[slot]):
                refs[table[slot][i]] -= 1
                table[slot][i] = -1
            counts[slot] = min(counts[slot], -(-lengths[slot] // page))

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)
    words = np.packbits(np.array(refs) == 0, bitorder="little")
    words = np.concatenate([words, np.zeros(-len(words) % 4, np.uint8)]).view(np.int32)
    out = [i32(table), i32(lengths), i32(counts), i32(refs), _dev(words)]
    if op == "admit":
        return out + [i32(granted)]
    pools = s["pools"]
    for src, to in copies:
        if src >= 0:
            pools[:, to] = pools[:, src]
    out += [i32(copies), pools.double()]
    return out + [i32(granted)] if op == "fork" else out


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s, case)
    return _exact_append(s, case) if case["op"] == "append" else _exact_pages(s, case)
