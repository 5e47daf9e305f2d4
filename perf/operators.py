"""The operators around draft verification, as they are measured: the 4-bit
output head that makes the logits, the penalties, biases and grammar masks on
them, and the token history that the penalties read.

``run`` computes each in its plain form (elementary torch operations in 32
bits, rounded once) or, with ``own`` set, through the library's entry points.
``exact`` computes the same from the definition in 64 bits.

The operators:

- process: row r of sequence b stands at place j = row0 + r of the drafted
  block.  With c_v = the history's count of v plus the drafted prefix's
  (x_1..x_j), seen_v = the history's mark of v or v in that prefix:
    l1 = seen_v ? (l > 0 ? l / repetition : l * repetition) : l
    l2 = l1 - (frequency * c_v + presence * [c_v > 0])
    l3 = l2 + the sum of v's biases
    out = v allowed by the row's mask ? l3 : -inf
  live = how many tokens a masked row has left above -inf (-1: no mask).
- history: a reset clears a slot; prompt tokens are marked as seen; output
  tokens are marked and counted; ids of -1 are padding.
- head: y = x W^T with W held in 4 bits: fp4 (e2m1 values, one power-of-two
  scale per 32) or int4 (q - 8, one bf16 scale per group).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one sequence drafting one token: nothing but latency
        dict(name="process one row", op="process", B=1, rows=1, row0=2, V=129280, bf16=True, packed=False,
             history=2000, biases=16, masked=1.0),
        # an ordinary verify batch, every row of the block, some requests with a grammar
        dict(name="process a batch", op="process", B=64, rows=9, row0=0, V=129280, bf16=True, packed=False,
             history=4096, biases=300, masked=0.25),
        # the headline verify batch: 4352 rows
        dict(name="process a large batch", op="process", B=256, rows=17, row0=0, V=129280, bf16=True, packed=False,
             history=8192, biases=32, masked=0.1),
        # rows packed by admission (1 to 5 of them a sequence), fp32 logits
        dict(name="process packed fp32 rows", op="process", B=512, rows=5, row0=0, V=129280, bf16=False, packed=True,
             history=1000, biases=0, masked=0.3),
        # constrained decoding only, in place, rows of an odd length without padding
        dict(name="mask in place", op="mask", B=100, rows=5, V=50257, bf16=True, masked=0.8),
        # one request is admitted: its prompt, and the tokens it had generated before it was preempted
        dict(name="history of one request", op="history", B=1, slots=8, V=129280, prompt=900, output=100),
        # a full batch is (re)admitted with long prompts
        dict(name="history of a batch", op="history", B=256, slots=256, V=129280, prompt=8192, output=1024),
        # the drafter's head for one token
        dict(name="head of one token fp4", op="head", rows=1, V=129280, H=7168, fmt="fp4", group=32, bf16=True),
        # a drafting step of 64 sequences
        dict(name="head of 64 rows fp4", op="head", rows=64, V=129280, H=4096, fmt="fp4", group=32, bf16=True),
        # a small model's head: an odd vocabulary, 90 groups of 32, fp32 logits
        dict(name="head of 5 rows int4", op="head", rows=5, V=50257, H=2880, fmt="int4", group=32, bf16=False),
        # the target's head over the rows that admission let through
        dict(name="head of 559 rows int4", op="head", rows=559, V=129280, H=4096, fmt="int4", group=128, bf16=True),
        # one drafting step of a batch: head, then penalties and masks in place
        dict(name="head and process", op="step", B=16, row0=3, V=129280, H=7168, fmt="fp4", group=32, bf16=True,
             history=2000, biases=64, masked=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["process", "process", "mask", "history", "head", "head", "head", "step"])
    V = _log(rng, 1000, 160000)
    bf16 = rng.random() < 0.7
    if op in ("process", "mask"):
        rows = _log(rng, 1, 17)
        B = _log(rng, 1, max(1, min(512, 560_000_000 // (V * rows * (1 if bf16 else 2)))))
        if op == "mask":
            return dict(op=op, B=B, rows=rows, V=V, bf16=bf16, masked=round(rng.uniform(0.1, 1.0), 2))
        return dict(op=op, B=B, rows=rows, row0=rng.choice([0, 0, rng.randint(1, 16)]), V=V, bf16=bf16,
                    packed=rng.random() < 0.3, history=_log(rng, 1, 16000), biases=rng.choice([0, _log(rng, 1, 400)]),
                    masked=round(rng.uniform(0.0, 1.0), 2))
    if op == "history":
        B = _log(rng, 1, 256)
        return dict(op=op, B=B, slots=B + rng.randint(0, 64), V=V, prompt=_log(rng, 1, 8192), output=_log(rng, 1, 1024))
    fmt = rng.choice(["fp4", "int4"])
    group = 32 if fmt == "fp4" else rng.choice([32, 64, 128])
    H = max(1, _log(rng, 256, 8192) // group) * group
    if op == "step":
        return dict(op=op, B=_log(rng, 1, 128), row0=rng.randint(0, 16), V=V, H=H, fmt=fmt, group=group, bf16=bf16,
                    history=_log(rng, 1, 8000), biases=rng.choice([0, _log(rng, 1, 300)]), masked=round(rng.uniform(0, 1), 2))
    rows = _log(rng, 1, max(1, min(1024, 290_000_000_000 // (V * H))))
    return dict(op=op, rows=rows, V=V, H=H, fmt=fmt, group=group, bf16=bf16)


# ------------------------------------------------------------------ inputs

def _words(bits):
    """bool [n][V] -> int32 [n][ceil(V / 32)], bit v % 32 of word v / 32."""
    n, V = bits.shape
    W = (V + 31) // 32
    full = torch.zeros((n, W * 32), dtype=torch.int32, device=bits.device)
    full[:, :V] = bits
    w = (full.view(n, W, 32) << torch.arange(32, dtype=torch.int32, device=bits.device)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _bits(words, V):
    """int32 [n][W] -> bool [n][V]."""
    b = (words.unsqueeze(-1) >> torch.arange(32, dtype=torch.int32, device=words.device)) & 1
    return b.view(words.shape[0], -1)[:, :V].bool()


def _tokens(g, shape, V):
    """Token ids as text has them: a few come often, most hardly ever."""
    u = torch.rand(shape, generator=g, device=DEV)
    return (u.pow(4) * V).to(torch.int32).clamp_(max=V - 1)


def _rules(case, g, r, B, rows, row0, V):
    """What a batch of requests brings: history, draft, penalties, biases, masks."""
    s = {}
    n_slots = B + 3
    slots = torch.randperm(n_slots, generator=g, device=DEV)[:B].to(torch.int32)
    if B > 2:
        slots[B // 2] = -1  # a request without a history
    H = case["history"]
    tok = _tokens(g, (n_slots, H), V).long()
    is_out = torch.rand((n_slots, H), generator=g, device=DEV) < 0.3
    counts = torch.zeros((n_slots, V), dtype=torch.int32, device=DEV).scatter_add_(1, tok, is_out.to(torch.int32))
    seen = torch.zeros((n_slots, V), dtype=torch.bool, device=DEV).scatter_(1, tok, True)
    s.update(counts=counts, seen=_words(seen), slots=slots)
    K = max(1, row0 + rows - 1)
    s["draft"] = _tokens(g, (B, K), V)
    s["rep"] = 1.0 + 0.5 * torch.rand(B, generator=g, device=DEV)
    s["freq"] = 0.8 * torch.rand(B, generator=g, device=DEV) - 0.1
    s["pres"] = 1.0 * torch.rand(B, generator=g, device=DEV)
    n = r.integers(0, case["biases"] + 1, B) if case["biases"] else np.zeros(B, np.int64)
    n = np.minimum(n, V)
    s["bias_off"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(DEV)
    total = int(n.sum())
    first = torch.from_numpy(r.integers(0, V, B)).to(DEV)
    b = torch.repeat_interleave(torch.arange(B, device=DEV), torch.from_numpy(n).to(DEV))
    place = torch.arange(total, device=DEV) - s["bias_off"].long()[b]
    step = 7919 if V % 7919 else 1
    s["bias_tok"] = ((first[b] + place * step) % V).to(torch.int32)  # in no order, each once
    s["bias_val"] = 4.0 * torch.randn(total, generator=g, device=DEV)
    s["bias_seq"] = b
    _masks(case, s, g, r, B, rows, V)
    return s


def _masks(case, s, g, r, B, rows, V):
    """Masks of a grammar's states: some allow nearly every token, some a few."""
    n = min(96, B * rows)
    share = torch.from_numpy(np.where(r.random(n) < 0.5, 0.97, 20.0 / V)).to(DEV)
    bits = torch.rand((n, V), generator=g, device=DEV) < share[:, None]
    if n > 3:
        bits[n // 2] = False  # a dead end: no token is allowed
    s["masks"] = _words(bits)
    idx = r.integers(0, n, (B, rows))
    idx[r.random(B) >= case["masked"]] = -1  # requests without a grammar
    s["mask_idx"] = torch.from_numpy(idx.astype(np.int32)).to(DEV)


def _weights(case, g):
    V, H, G = case["V"], case["H"], case["group"]
    w = torch.randn((V, H), generator=g, device=DEV, dtype=torch.bfloat16)
    if case["fmt"] == "fp4":
        w = w * 2.0
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV, dtype=torch.bfloat16)
        code = torch.bucketize(w.abs(), edges, out_int32=True).to(torch.uint8)
        code |= (w < 0).to(torch.uint8) << 3
        scale = torch.randint(127 - 9, 127 - 5, (V, H // G), generator=g, device=DEV, dtype=torch.uint8)
    else:
        code = (w * 2.5).round().clamp_(-8, 7).add_(8).to(torch.uint8)
        scale = ((0.5 + torch.rand((V, H // G), generator=g, device=DEV)) * 0.01).to(torch.bfloat16)
    del w
    return code[:, 0::2] | (code[:, 1::2] << 4), scale


def _hidden(g, rows, H):
    """Normalised hidden states: unit variance, a few channels far larger."""
    x = torch.randn((rows, H), generator=g, device=DEV)
    big = torch.rand(H, generator=g, device=DEV) < 0.004
    return torch.where(big, x * 12.0, x).to(torch.bfloat16)


def _inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng(seed)
    op, V = case["op"], case["V"]
    if op == "history":
        B, S = case["B"], case["slots"]
        n = r.integers((case["prompt"] + 1) // 2, case["prompt"] + 1, B)
        off = np.concatenate([[0], np.cumsum(n)])
        s = dict(prompt=_tokens(g, (int(off[-1]),), V), prompt_off=torch.from_numpy(off).to(DEV), most=int(n.max()),
                 slots=torch.from_numpy(r.permutation(S)[:B].astype(np.int32)).to(DEV),
                 reset=torch.ones(B, dtype=torch.int32, device=DEV))
        out = _tokens(g, (B, case["output"]), V)
        keep = torch.from_numpy(r.integers(1, case["output"] + 1, B)).to(DEV)
        s["output"] = torch.where(torch.arange(case["output"], device=DEV) < keep[:, None], out, -1)
        s["counts"] = torch.zeros((S, V), dtype=torch.int32, device=DEV)
        s["seen"] = torch.zeros((S, (V + 31) // 32), dtype=torch.int32, device=DEV)
        return s
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    s = {"dt": dt}
    if op == "head":
        s["w"], s["scale"] = _weights(case, g)
        s["x"] = _hidden(g, case["rows"], case["H"])
        return s
    B = case["B"]
    if op == "step":
        s.update(_rules(case, g, r, B, 1, case["row0"], V))
        s["w"], s["scale"] = _weights(case, g)
        s["x"] = _hidden(g, B, case["H"])
        s["seq"] = torch.arange(B, device=DEV)
        s["place"] = torch.zeros(B, dtype=torch.int64, device=DEV)
        return s
    rows = case["rows"]
    n = np.full(B, rows)
    if case.get("packed"):
        n = r.permutation(np.resize(np.arange(1, rows + 1), B))  # as many rows in all, whatever the seed
    s["row_off"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).to(DEV)
    s["seq"] = torch.from_numpy(np.repeat(np.arange(B), n)).to(DEV)
    s["place"] = torch.from_numpy(np.concatenate([np.arange(k) for k in n])).to(DEV)
    s["logits"] = torch.empty((int(n.sum()), V), dtype=dt, device=DEV).normal_(0.0, 2.0, generator=g)
    if op == "process":
        s.update(_rules(case, g, r, B, rows, case["row0"], V))
    else:
        _masks(case, s, g, r, B, rows, V)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        _prepare_own(case, s)
    return s


# ------------------------------------------------------------------ the library's calls

def _prepare_own(case, s):
    """What a user's program keeps: the handle, the packed weights, the output
    buffers, and the argument structs that name them."""
    from draft_verification_amd import binding as B
    op, V = case["op"], case["V"]
    kind = B.SV_BF16 if case.get("bf16", True) else B.SV_F32
    if op == "history":
        s["sv"] = B.SpecVerify(case["B"], 1, V, kind)
        state = dict(slots=s["slots"], counts=s["counts"], seen=s["seen"], n_slots=case["slots"])
        s["args"] = [B.make_history_args(case["B"], tokens=s["prompt"], token_offsets=s["prompt_off"],
                                         n_tokens=s["prompt"].numel(), max_tokens=s["most"], kind=B.SV_HISTORY_PROMPT, reset=s["reset"], **state),
                     B.make_history_args(case["B"], tokens=s["output"], token_stride=case["output"],
                                         max_tokens=case["output"], kind=B.SV_HISTORY_OUTPUT, **state)]
        return
    if op in ("head", "step"):
        M, H = s["x"].shape
        fmt = B.SV_W4_FP4 if case["fmt"] == "fp4" else B.SV_W4_INT4
        s["sv"] = B.SpecVerify(M, max(1, case.get("row0", 0)), V, kind)
        packed = torch.empty(s["sv"].head_packed_bytes(H, fmt, case["group"]), dtype=torch.uint8, device=DEV)
        s["sv"].head_pack(B.make_head_pack_args(hidden=H, format=fmt, group=case["group"], weights=s["w"],
                                                weight_stride=H // 2, scales=s["scale"],
                                                scale_stride=H // case["group"], packed=packed))
        s["packed"] = packed
        s["out"] = torch.empty((M, V), dtype=s["dt"], device=DEV)
        s["head_args"] = B.make_head_args(M, hidden=H, format=fmt, group=case["group"], packed=packed,
                                          hidden_states=s["x"], hidden_stride=H, logits=s["out"], logits_stride=V)
        if op == "head":
            return
    Bn, rows = case["B"], case.get("rows", 1)
    row0 = case.get("row0", 0)
    if op != "step":
        s["sv"] = B.SpecVerify(Bn, max(1, row0 + rows - 1), V, kind)
    src = s["logits"] if op != "step" else s["out"]
    dst = torch.empty_like(src) if op == "process" else src
    s["out"] = dst
    s["live"] = torch.empty((Bn, rows), dtype=torch.int32, device=DEV)
    rules = {}
    if op != "mask":
        rules = dict(draft_tokens=s["draft"], draft_stride=s["draft"].shape[1], history_counts=s["counts"],
                     history_seen=s["seen"], n_slots=s["counts"].shape[0], slots=s["slots"], repetition=s["rep"],
                     frequency=s["freq"], presence=s["pres"])
        if s["bias_tok"].numel():
            rules.update(bias_offsets=s["bias_off"], bias_tokens=s["bias_tok"], bias_values=s["bias_val"],
                         n_biases=s["bias_tok"].numel())
    packed = s["row_off"] if case.get("packed") else None
    s["args"] = B.make_process_args(Bn, rows, row0=row0, logits_in=src, in_strides=(rows * V, V), logits_out=dst,
                                    out_strides=(rows * V, V), row_offsets=packed, masks=s["masks"],
                                    mask_stride=s["masks"].shape[1], n_masks=s["masks"].shape[0],
                                    mask_index=s["mask_idx"], live_tokens=s["live"], **rules)


def _run_own(s):
    op = s["case"]["op"]
    if op == "history":
        s["sv"].history(s["args"][0])
        s["sv"].history(s["args"][1])
        return [s["counts"], s["seen"]]
    if op in ("head", "step"):
        s["sv"].head(s["head_args"])
        if op == "head":
            return [s["out"]]
    s["sv"].process(s["args"])
    return [s["out"], s["live"]]


# ------------------------------------------------------------------ the plain forms

def _plain_weights(s):
    """The 4-bit weights as float32 [V][H]."""
    w, scale = s["w"], s["scale"]
    if s["case"]["fmt"] == "fp4":
        value = torch.tensor(FP4, device=DEV)
        scale = torch.exp2(scale.float() - 127.0)
    else:
        value = torch.arange(16, device=DEV, dtype=torch.float32) - 8.0
        scale = scale.float()
    pair = torch.arange(256, device=DEV)
    table = torch.stack([value[pair & 15], value[pair >> 4]], 1)  # both values of a byte
    V, G = w.shape[0], scale.shape[1]
    full = table.index_select(0, w.reshape(-1).to(torch.int32)).view(V, G, -1)
    return full.mul_(scale.unsqueeze(-1)).view(V, -1)


def _plain_process(s, logits):
    case = s["case"]
    V, seq, place = case["V"], s["seq"], s["place"]
    l = logits.float()
    if case["op"] != "mask":
        slot = s["slots"].long()
        has = (slot >= 0)[:, None]
        at = slot.clamp(min=0)
        counts = torch.where(has, s["counts"].index_select(0, at), 0)
        seen = _bits(s["seen"], V).index_select(0, at) & has
        draft = s["draft"].index_select(0, seq).long()
        in_prefix = torch.arange(draft.shape[1], device=DEV) < (place + case["row0"])[:, None]
        c = counts.index_select(0, seq).scatter_add_(1, draft, in_prefix.to(torch.int32))
        marked = torch.zeros_like(l, dtype=torch.int32).scatter_add_(1, draft, in_prefix.to(torch.int32)) > 0
        marked |= seen.index_select(0, seq)
        rep, freq, pres = (s[k].index_select(0, seq)[:, None] for k in ("rep", "freq", "pres"))
        l = torch.where(marked, torch.where(l > 0, l / rep, l * rep), l)
        l = l - (freq * c + pres * (c > 0))
        bias = torch.zeros((case["B"], V), device=DEV)
        bias.index_put_((s["bias_seq"], s["bias_tok"].long()), s["bias_val"])
        l = l + bias.index_select(0, seq)
    which = s["mask_idx"][seq, place].long()
    allowed = _bits(s["masks"], V).index_select(0, which.clamp(min=0)) | (which < 0)[:, None]
    out = torch.where(allowed, l, -math.inf).to(s["dt"])
    left = torch.where(which < 0, -1, (out > -math.inf).sum(1)).to(torch.int32)
    live = torch.full((case["B"], case.get("rows", 1)), -1, dtype=torch.int32, device=DEV)
    live[seq, place] = left
    return [out, live]


def _run_plain(s):
    case = s["case"]
    op, V = case["op"], case["V"]
    if op == "history":
        slot = s["slots"].long()
        counts = s["counts"].index_fill(0, slot, 0)
        seen = _bits(s["seen"], V).index_fill(0, slot, False)
        n = s["prompt_off"][1:] - s["prompt_off"][:-1]
        seen[torch.repeat_interleave(slot, n, output_size=s["prompt"].numel()), s["prompt"].long()] = True
        there = s["output"] >= 0
        rows = slot[:, None].expand_as(s["output"])
        tok = s["output"].clamp(min=0).long()
        counts.index_put_((rows, tok), there.to(torch.int32), accumulate=True)
        seen |= counts > 0
        return [counts, _words(seen)]
    if op in ("head", "step"):
        y = (s["x"].float() @ _plain_weights(s).t()).to(s["dt"])
        if op == "head":
            return [y]
        return _plain_process(s, y)
    return _plain_process(s, s["logits"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, V = case["op"], case["V"]
    words = 4 * ((V + 31) // 32)
    if op == "history":
        tokens = case["B"] * (0.75 * case["prompt"] + 0.5 * case["output"])
        return {"bytes": case["B"] * (4 * V + words) + 12.0 * tokens, "flops": tokens}
    es = 2 if case["bf16"] else 4
    head = {"bytes": 0.0, "flops": 0.0}
    if op in ("head", "step"):
        M, H, G = case["rows"] if op == "head" else case["B"], case["H"], case["group"]
        head["bytes"] = V * H / 2 + V * (H // G) * (1 if case["fmt"] == "fp4" else 2) + 2.0 * M * H + float(M) * V * es
        head["flops"] = 2.0 * M * V * H
        if op == "head":
            return head
    B, rows = case["B"], case.get("rows", 1)
    n = B * (rows + 1) / 2 if case.get("packed") else B * rows
    masked = n * case["masked"]
    if op == "mask":  # rows without a mask need no access; the others' allowed logits are read, the rest written
        return {"bytes": masked * (V * es + words), "flops": masked * V}
    kept = min(V, 0.6 * case["history"])  # tokens that the history holds, about
    rules = B * (words + 4.0 * kept + 8.0 * case["biases"] / 2) + masked * words
    if op == "step":  # in place: what the head wrote is changed where a rule says so
        return {"bytes": head["bytes"] + rules + masked * V * es, "flops": head["flops"] + 5.0 * n * V}
    return {"bytes": 2.0 * n * V * es + rules, "flops": 5.0 * n * V}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_head(s, case):
    value = torch.tensor(FP4 if case["fmt"] == "fp4" else [q - 8.0 for q in range(16)], dtype=torch.float64, device=DEV)
    x = s["x"].double()
    parts = []
    for v0 in range(0, case["V"], 16384):
        w = s["w"][v0:v0 + 16384]
        q = torch.empty((w.shape[0], case["H"]), dtype=torch.int32, device=DEV)
        q[:, 0::2] = (w & 15).to(torch.int32)
        q[:, 1::2] = (w >> 4).to(torch.int32)
        scale = s["scale"][v0:v0 + 16384]
        scale = torch.ldexp(torch.ones((), dtype=torch.float64, device=DEV), scale.int() - 127) if case["fmt"] == "fp4" else scale.double()
        parts.append(x @ (value[q] * scale.repeat_interleave(case["group"], 1)).t())
    return torch.cat(parts, 1)


def exact(case, seed):
    s = _inputs(case, seed)
    op, V = case["op"], case["V"]
    if op == "history":
        off = s["prompt_off"].tolist()
        for b, slot in enumerate(s["slots"].tolist()):
            mine = s["output"][b][s["output"][b] >= 0].long()
            s["counts"][slot] = torch.bincount(mine, minlength=V).int()
            bits = torch.zeros(((V + 31) // 32) * 32, dtype=torch.int64, device=DEV)
            bits[s["prompt"][off[b]:off[b + 1]].long()] = 1
            bits[mine] = 1
            w = (bits.view(-1, 32) * (2 ** torch.arange(32, device=DEV))).sum(1)
            s["seen"][slot] = torch.where(w > 2 ** 31 - 1, w - 2 ** 32, w).int()
        return [s["counts"], s["seen"]]
    if op in ("head", "step"):
        l = _exact_head(s, case)
        if op == "head":
            return [l]
    else:
        l = s["logits"].double()
    live = torch.full((case["B"], case.get("rows", 1)), -1, dtype=torch.int32, device=DEV)
    token = torch.arange(V, device=DEV)
    shift = (token % 32).int()
    slots = s["slots"].tolist() if op != "mask" else None
    which = s["mask_idx"].tolist()
    off = s["bias_off"].tolist() if op != "mask" else None
    now, held, count = -1, None, None
    for n, (b, j) in enumerate(zip(s["seq"].tolist(), s["place"].tolist())):
        row = l[n]
        if op != "mask":
            if b != now:
                now = b
                if slots[b] >= 0:
                    count = s["counts"][slots[b]].double()
                    held = ((s["seen"][slots[b]][token // 32] >> shift) & 1) == 1
                else:
                    count = torch.zeros(V, dtype=torch.float64, device=DEV)
                    held = torch.zeros(V, dtype=torch.bool, device=DEV)
            prefix = torch.bincount(s["draft"][b][:case["row0"] + j].long(), minlength=V).double()
            c, rep = count + prefix, s["rep"][b].double()
            row = torch.where(held | (prefix > 0), torch.where(row > 0, row / rep, row * rep), row)
            row = row - s["freq"][b].double() * c - s["pres"][b].double() * (c > 0).double()
            mine = slice(off[b], off[b + 1])
            row[s["bias_tok"][mine].long()] += s["bias_val"][mine].double()
        if which[b][j] >= 0:
            bit = (s["masks"][which[b][j]][token // 32] >> shift) & 1
            row = torch.where(bit == 1, row, -math.inf)
            live[b, j] = (row > -math.inf).sum()
        l[n] = row
    return [l, live]
