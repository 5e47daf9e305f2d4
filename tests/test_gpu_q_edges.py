"""Further edges of the calls around verification."""
import numpy as np
import pytest

from oracle import rules as R
from tests import test_gpu_n_head as N

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"


def _lib():
    from draft_verification_amd import binding
    return binding


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("inplace", [False, True])
def test_bias_lists_up_to_the_last_32_bit_index(inplace):
    # three turns of 64 biases, two turns, and one, the last of them ending at 2^31 - 1
    B = _lib()
    Bn, V, N = 3, 1000, 2 ** 31 - 1
    off = np.array([N - 250, N - 120, N - 20, N], np.int32)
    rng = np.random.default_rng(5)
    l = (3 * rng.standard_normal((Bn, V))).astype(np.float32)
    ids, values = rng.integers(0, V, 250).astype(np.int32), (2 * rng.standard_normal(250)).astype(np.float32)
    tok, val = torch.empty(N, dtype=torch.int32, device=DEV), torch.empty(N, dtype=torch.float32, device=DEV)
    tok[-250:], val[-250:] = torch.from_numpy(ids).to(DEV), torch.from_numpy(values).to(DEV)
    src = torch.from_numpy(l).to(DEV)
    out = src if inplace else torch.zeros_like(src)
    status = torch.full((1,), -9, dtype=torch.int32, device=DEV)
    B.SpecVerify(Bn, 1, V, B.SV_F32).process(B.make_process_args(
        Bn, 1, logits_in=src, in_strides=(V, V), logits_out=out, out_strides=(V, V), bias_offsets=torch.from_numpy(off).to(DEV),
        bias_tokens=tok, bias_values=val, n_biases=N, device_status=status))
    assert int(status) == 0
    got = out.cpu().numpy().astype(np.float64)
    for b in range(Bn):
        at = slice(off[b] - (N - 250), off[b + 1] - (N - 250))
        want, _, size = R.process_row(l[b].astype(np.float64), [], None, None, 1.0, 0.0, 0.0,
                                      list(zip(ids[at], values[at].astype(float))), None)
        # one rounding for each bias added, and the sum with the logit
        assert (np.abs(got[b] - want) <= (at.stop - at.start + 1) * 2.0 ** -24 * size).all()
        named = np.zeros(V, bool)
        named[ids[at]] = True
        assert np.array_equal(got[b][~named], l[b][~named])


@pytest.mark.parametrize("off", [[-2, 0, 2, 3], [-1, 1, 3, 4], [-3, -1, 2, 3], [-2 ** 63, 0, 1, 3], [0, 2, -1, 1]])
@pytest.mark.parametrize("inplace", [False, True])
def test_rows_before_the_first_are_left_alone(off, inplace):
    # the buffers go on before the call's first row, so that what lies there can be looked at
    B = _lib()
    V, before, rows = 600, 4, 3
    src = torch.full((before + 6, V), 2.0, device=DEV)
    out = src if inplace else torch.full((before + 6, V), 55.0, device=DEV)
    was = out.clone()
    live, status = torch.full((3, rows), -9, dtype=torch.int32, device=DEV), torch.full((1,), -9, dtype=torch.int32, device=DEV)
    mask = torch.full((1, (V + 31) // 32), 0x0f0f0f0f, dtype=torch.int32, device=DEV)
    B.SpecVerify(3, rows, V, B.SV_F32).process(B.make_process_args(
        3, rows, logits_in=src[before:], in_strides=(0, V), logits_out=out[before:], out_strides=(0, V),
        row_offsets=torch.tensor(off, dtype=torch.int64, device=DEV), masks=mask, mask_stride=mask.shape[1], n_masks=1,
        mask_index=torch.zeros((3, rows), dtype=torch.int32, device=DEV), live_tokens=live, device_status=status))
    assert int(status) == B.SV_STATUS_BAD_INPUT
    allowed = torch.from_numpy(R.bits(mask[0].cpu().numpy().view(np.uint32), V)).to(DEV)
    row = torch.where(allowed, 2.0, -float("inf"))
    for b in range(3):
        n = off[b + 1] - off[b] if off[b] >= 0 and off[b] <= off[b + 1] <= off[b] + rows else 0
        assert live[b].tolist() == [int(allowed.sum())] * n + [-1] * (rows - n)
        for r in range(n):
            was[before + off[b] + r] = row
    assert torch.equal(out, was)


@pytest.mark.parametrize("V", [2 ** 20, 2 ** 20 - 37, 131, 33])
@pytest.mark.parametrize("output", [True, False])
def test_reset_of_a_shared_slot_over_the_whole_vocabulary(V, output):
    # sequences 0, 2 and 3 share a slot, one of them resets it; 1 and 4 have theirs, reset and not
    B = _lib()
    rng = np.random.default_rng(V)
    seqs = [(2, 700, 0), (0, 300, 1), (2, 0, 1), (2, 2000, 0), (1, 500, 0)]
    tokens = np.full((5, 2000), -1, np.int32)
    for b, (_, n, _) in enumerate(seqs):
        tokens[b, :n] = rng.integers(0, V, n)
        tokens[b, :min(n, 4)] = [0, V - 1, V // 2, 31][:min(n, 4)]
    counts = rng.integers(0, 5, (4, V)).astype(np.int32)
    flags = rng.random((4, V)) < 0.1
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    dc, ds, status = up(counts), up(R.words(flags).view(np.int32)), i32([-9])
    B.SpecVerify(5, 1, V, B.SV_BF16).history(B.make_history_args(
        5, tokens=up(tokens), token_stride=2000, max_tokens=2000, kind=B.SV_HISTORY_OUTPUT if output else B.SV_HISTORY_PROMPT,
        slots=i32([s for s, _, _ in seqs]), reset=i32([r for _, _, r in seqs]), counts=dc, seen=ds, n_slots=4,
        device_status=status))
    assert int(status) == 0
    R.history_update(counts, flags, [(s, t[:n], r) for (s, n, r), t in zip(seqs, tokens)], output)
    assert np.array_equal(dc.cpu().numpy(), counts)
    assert np.array_equal(ds.cpu().numpy().view(np.uint32), R.words(flags))


@pytest.mark.parametrize("V,M", [(4096, 8), (65536, 16)])  # split-K workgroups, and tiles
def test_every_fp4_scale_with_every_code(V, M):
    # one hidden value at a time picks one weight; where that is in bf16's normal range or zero it is exact
    B = _lib()
    H = 32
    code, s8 = np.arange(V) % 16, (np.arange(V) // 16) % 256
    w = torch.from_numpy(np.repeat((code | code << 4).astype(np.uint8)[:, None], H // 2, 1)).to(DEV)
    s = torch.from_numpy(s8.astype(np.uint8)[:, None].copy()).to(DEV)
    sv = B.SpecVerify(M, 1, V, B.SV_F32)
    packed = torch.empty(sv.head_packed_bytes(H, B.SV_W4_FP4, 32), dtype=torch.uint8, device=DEV)
    sv.head_pack(B.make_head_pack_args(hidden=H, format=B.SV_W4_FP4, group=32, weights=w, weight_stride=H // 2, scales=s,
                                       scale_stride=1, packed=packed))
    x = torch.eye(H, device=DEV)[:M].to(torch.bfloat16).contiguous()
    out = torch.empty((M, V), device=DEV)
    sv.head(B.make_head_args(M, hidden=H, format=B.SV_W4_FP4, group=32, packed=packed, hidden_states=x, hidden_stride=H,
                             logits=out, logits_stride=V))
    want = R.FP4[code] * np.ldexp(1.0, s8 - 127)
    held = (want == 0) | ((np.abs(want) >= 2.0 ** -126) & (np.abs(want) < 2.0 ** 128))
    held &= s8 < 255
    assert held[s8 == 0].sum() == 10 * (V // 4096) and held[s8 == 254].sum() == 8 * (V // 4096)
    got = out.double().cpu().numpy()
    assert np.isnan(got[:, s8 == 255]).all()
    bad = np.flatnonzero((got[:, held] != want[held]).any(0))
    assert bad.size == 0, [(code[held][i], s8[held][i], got[0, held][i], want[held][i]) for i in bad[:8]]
# what test_gpu_n_head.py leaves of the head's kernels in either logits type: split-K workgroups, one block of
# rows and several in tiles of 16 and 32 rows, tiles of 64, the last block in part, odd and even numbers of steps
HEADS = [
    (31, 33001, 288, "fp4", 32, "bf16"), (100, 20001, 160, "fp4", 32, "bf16"),
    (130, 32010, 352, "int4", 32, "f32"), (12, 164001, 96, "int4", 32, "bf16"), (100, 16003, 160, "int4", 32, "bf16"),
    (31, 82001, 288, "int4", 32, "bf16"), (70, 32010, 96, "int4", 32, "bf16"),
    (40, 19001, 320, "int4", 64, "f32"), (31, 82001, 192, "int4", 64, "f32"), (16, 164001, 128, "int4", 64, "bf16"),
    (130, 32010, 320, "int4", 64, "bf16"),
    (12, 164001, 384, "int4", 128, "f32"), (100, 8500, 256, "int4", 128, "f32"), (100, 8500, 384, "int4", 128, "f32"),
    (130, 32010, 128, "int4", 128, "f32"), (12, 7501, 384, "int4", 128, "bf16"), (40, 19001, 256, "int4", 128, "bf16"),
    (70, 12001, 640, "int4", 128, "bf16"), (31, 40001, 384, "int4", 128, "bf16"), (70, 16003, 128, "int4", 128, "bf16"),
]


@pytest.mark.parametrize("M,V,H,fmt,group,dtype", HEADS)
def test_head_kernels_in_both_types(M, V, H, fmt, group, dtype):
    print(f"[case] head M={M} V={V} H={H} {fmt} {group} {dtype}", flush=True)
    wt = N.Weights(V, H, fmt, group, seed=M + V)
    x = N._x(np.random.default_rng(M), M, H)
    got, _ = N._run(wt, x, dtype)
    N._check(wt, x, got, dtype)


@pytest.mark.parametrize("M,V", [(5, 200), (16, 164001), (70, 66001)])  # split-K workgroups, one block in tiles, several
@pytest.mark.parametrize("group", [32, 64, 128])
def test_int4_error_stays_within_the_stated_bound(M, V, group):
    # vocabulary rows of codes 8 (weights of zero), of codes 7 and 9, and of any, on hidden values with one sign
    # and channels 2^10 times the others: where the sum of (code + 16) x and 24 times that of x nearly cancel
    B = _lib()
    H = 768
    rng = np.random.default_rng(group)
    codes = rng.integers(0, 16, (V, H))
    codes[0::3] = 8
    codes[1::3] = 7 + 2 * (codes[1::3] & 1)
    scale = torch.from_numpy((0.5 + rng.random((V, H // group))).astype(np.float32)).to(torch.bfloat16)
    x = np.abs(rng.standard_normal((M, H))) + 0.5
    x[:, ::100] *= 1024
    x = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
    sv = B.SpecVerify(M, 1, V, B.SV_F32)
    packed = torch.empty(sv.head_packed_bytes(H, B.SV_W4_INT4, group), dtype=torch.uint8, device=DEV)
    w, s, xd = torch.from_numpy((codes[:, ::2] | codes[:, 1::2] << 4).astype(np.uint8)).to(DEV), scale.to(DEV), x.to(DEV)
    sv.head_pack(B.make_head_pack_args(hidden=H, format=B.SV_W4_INT4, group=group, weights=w, weight_stride=H // 2, scales=s,
                                       scale_stride=H // group, packed=packed))
    out = torch.empty((M, V), device=DEV)
    sv.head(B.make_head_args(M, hidden=H, format=B.SV_W4_INT4, group=group, packed=packed, hidden_states=xd, hidden_stride=H,
                             logits=out, logits_stride=V))
    x64, s64 = x.double().numpy(), np.repeat(scale.double().numpy(), group, 1)
    off = np.abs(out.double().cpu().numpy() - x64 @ ((codes - 8) * s64).T)
    assert (off <= (H / 32 + 40) * 2.0 ** -23 * (np.abs(x64) @ ((codes + 40) * s64).T)).all()
