"""The 4-bit output head against an fp64 product with the same weights.

Tolerance.  Every weight and every product with a bf16 hidden value is exact in
fp32; what rounds is the summation.  Products are summed 32 at a time by the
matrix core and those sums one after another (fewer than H / 32 + 40 additions
on any term's way to the result, joins of partial sums among them), each off by
at most 2^-23 of the sum of the terms' absolute values (a step: the matrix core
may truncate).  INT4 sums (code + 16) x and 24 x apart, so its terms are those
magnitudes.  fp32 sums are then rounded once to the logits' type."""
import numpy as np
import pytest

from oracle import rules as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"


def _lib():
    from draft_verification_amd import binding
    return binding


class Weights:
    def __init__(self, V, H, fmt, group, seed=0, wpad=0, spad=0):
        LB = _lib()
        rng = np.random.default_rng(seed)
        self.V, self.H, self.group, self.fp4 = V, H, group, fmt == "fp4"
        self.format = LB.SV_W4_FP4 if self.fp4 else LB.SV_W4_INT4
        self.codes = rng.integers(0, 256, (V, H // 2)).astype(np.uint8)
        G = H // group
        if self.fp4:
            s8 = rng.integers(110, 130, (V, G)).astype(np.uint8)
            self.scale = np.ldexp(1.0, s8.astype(int) - 127)
            st = torch.from_numpy(np.pad(s8, ((0, 0), (0, spad)), constant_values=255))
        else:
            sb = torch.from_numpy((0.01 * (0.1 + rng.random((V, G)))).astype(np.float32)).to(torch.bfloat16)
            self.scale = sb.double().numpy()
            st = torch.nn.functional.pad(sb.float(), (0, spad), value=float("nan")).to(torch.bfloat16)
        self.w = torch.from_numpy(np.pad(self.codes, ((0, 0), (0, wpad)), constant_values=0xff)).to(DEV)
        self.s = st.to(DEV)

    def pack(self, sv):
        LB = _lib()
        n = sv.head_packed_bytes(self.H, self.format, self.group)
        buf = torch.full((n + 64,), 0x5a, dtype=torch.uint8, device=DEV)
        sv.head_pack(LB.make_head_pack_args(hidden=self.H, format=self.format, group=self.group, weights=self.w,
                                            weight_stride=self.w.shape[1], scales=self.s, scale_stride=self.s.shape[1],
                                            packed=buf))
        assert (buf[n:] == 0x5a).all()
        return buf

    def exact(self, x):
        """(x W^T, the sum of the terms' absolute values) in fp64, x fp64 [M][H]."""
        W = R.head_weights(self.codes, self.scale, self.fp4, self.group)
        mag = np.abs(W) if self.fp4 else np.abs(R.head_weights(self.codes, self.scale, False, self.group) +
                                                24 * np.repeat(self.scale, self.group, 1)) + 24 * np.repeat(self.scale, self.group, 1)
        return x @ W.T, np.abs(x) @ mag.T


def _x(rng, M, H):
    x = rng.standard_normal((M, H))
    x[:, ::37] *= 20
    x[:, 5] += 3
    t = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
    return t


def _run(wt, x, dtype, *, xpad=0, xshift=0, lpad=0, lshift=0, max_batch=None):
    LB = _lib()
    M, H = x.shape
    sv = LB.SpecVerify(max_batch or max(M, 1), 1, wt.V, LB.SV_BF16 if dtype == "bf16" else LB.SV_F32)
    packed = wt.pack(sv)
    xs, ls = H + xpad, wt.V + lpad
    xb = torch.full((xshift + M * xs,), float("nan"), dtype=torch.bfloat16, device=DEV)  # what lies between rows is not read
    xb[xshift:].view(M, xs)[:, :H] = x.to(DEV)
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    out = torch.full((lshift + M * ls + 9,), 55.0, dtype=tdt, device=DEV)
    sv.head(LB.make_head_args(M, hidden=H, format=wt.format, group=wt.group, packed=packed, hidden_states=xb[xshift:],
                              hidden_stride=xs, logits=out[lshift:], logits_stride=ls))
    torch.cuda.synchronize()
    full = out.double().cpu().numpy()
    body = full[lshift:lshift + M * ls].reshape(M, ls)
    assert (full[:lshift] == 55).all() and (full[lshift + M * ls:] == 55).all() and (body[:, wt.V:] == 55).all()
    return body[:, :wt.V], out


def _check(wt, x, got, dtype):
    want, size = wt.exact(x.double().numpy())
    tol = (wt.H / 32 + 40) * 2.0 ** -23 * size + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
    off = np.abs(got - want)
    assert (off <= tol).all(), (np.argwhere(off > tol)[:5], (off / tol).max())
    # and as a whole far nearer than the bound of every single value
    assert np.linalg.norm(got - want) <= (2.0 ** -9 if dtype == "bf16" else 2.0 ** -17) * np.linalg.norm(want)


CASES = [
    # M, V, H, format, group, dtype, padding
    (1, 64, 128, "fp4", 32, "f32", {}), (1, 64, 128, "int4", 128, "f32", {}), (1, 1, 32, "fp4", 32, "f32", {}),
    (1, 1, 32, "int4", 32, "bf16", {}), (3, 65, 96, "fp4", 32, "bf16", {}), (2, 100, 320, "int4", 64, "f32", {}),
    (15, 257, 256, "int4", 32, "f32", {}), (16, 255, 2880, "fp4", 32, "f32", {}), (17, 1003, 2880, "int4", 32, "bf16", {}),
    (33, 4099, 640, "int4", 128, "f32", {}), (64, 1000, 4096, "fp4", 32, "bf16", {}), (65, 511, 1024, "fp4", 32, "f32", {}),
    (130, 700, 896, "int4", 64, "bf16", {}), (300, 1111, 416, "fp4", 32, "bf16", {}), (5, 20000, 7168, "int4", 128, "f32", {}),
    (4, 300, 256, "fp4", 32, "bf16", dict(xpad=8, lpad=5)), (4, 300, 256, "int4", 64, "f32", dict(xpad=3, xshift=1, lpad=1, lshift=3)),
    (70, 130, 288, "fp4", 32, "bf16", dict(xpad=1, xshift=5, lshift=1, lpad=2)), (1, 129280, 1024, "fp4", 32, "bf16", {}),
    (600, 2000, 128, "int4", 32, "f32", {}),
    # enough vocabulary and rows for the tiles of 16, 32 and 64 rows, over an odd and an even number of steps
    (9, 65700, 160, "fp4", 32, "f32", {}), (16, 65601, 352, "fp4", 32, "bf16", dict(xpad=1, xshift=3, lshift=1)),
    (12, 164000, 192, "int4", 64, "f32", {}), (16, 164100, 128, "int4", 128, "bf16", {}), (13, 164099, 96, "int4", 32, "f32", {}),
    (20, 33001, 288, "fp4", 32, "f32", {}), (31, 82100, 320, "int4", 64, "bf16", {}), (32, 82001, 384, "int4", 128, "f32", {}),
    (17, 82100, 160, "int4", 32, "f32", dict(xpad=8, lpad=3)), (64, 20000, 416, "fp4", 32, "f32", {}), (40, 20033, 128, "fp4", 32, "bf16", {}),
    (130, 20001, 640, "int4", 128, "f32", {}), (129, 20001, 192, "int4", 64, "bf16", dict(xpad=3, lpad=1)),
    (190, 20001, 160, "int4", 32, "f32", {}),
]


@pytest.mark.parametrize("M,V,H,fmt,group,dtype,pad", CASES)
def test_head_matches_the_product(M, V, H, fmt, group, dtype, pad):
    print(f"[case] head M={M} V={V} H={H} {fmt} {group} {dtype} {pad}", flush=True)
    wt = Weights(V, H, fmt, group, seed=M + V, wpad=3 if pad else 0, spad=1 if pad else 0)
    x = _x(np.random.default_rng(M), M, H)
    got, _ = _run(wt, x, dtype, **pad)
    _check(wt, x, got, dtype)


# several blocks of rows in the tiles of 16, 32 and 64 rows, the last of them in part
BLOCKS = [(100, 8000, 160, "fp4", 32, "f32"), (100, 16001, 288, "fp4", 32, "bf16"), (250, 32010, 160, "fp4", 32, "f32"),
          (70, 66001, 96, "fp4", 32, "bf16"), (500, 2001, 192, "fp4", 32, "f32"),
          (100, 16003, 160, "int4", 32, "f32"), (250, 32010, 96, "int4", 32, "bf16"), (70, 66001, 128, "int4", 32, "f32"),
          (100, 12001, 192, "int4", 64, "bf16"), (250, 32010, 128, "int4", 64, "f32"), (75, 40001, 320, "int4", 64, "f32"),
          (100, 12001, 256, "int4", 128, "f32"), (250, 32010, 128, "int4", 128, "bf16"), (90, 24001, 384, "int4", 128, "f32")]


@pytest.mark.parametrize("M,V,H,fmt,group,dtype", BLOCKS)
def test_several_blocks_of_rows(M, V, H, fmt, group, dtype):
    print(f"[case] head M={M} V={V} H={H} {fmt} {group} {dtype}", flush=True)
    wt = Weights(V, H, fmt, group, seed=M + V)
    x = _x(np.random.default_rng(M), M, H)
    got, _ = _run(wt, x, dtype)
    _check(wt, x, got, dtype)


@pytest.mark.parametrize("fmt", ["fp4", "int4"])
def test_every_code_and_scale_is_decoded(fmt):
    # one hidden value at a time picks one weight: the logits are the weights
    V, H = 256, 128
    wt = Weights(V, H, fmt, 32, seed=3)
    wt.codes[:] = np.arange(V)[:, None]
    if fmt == "fp4":
        s8 = (1 + np.arange(V) % 250).astype(np.uint8)  # from 2^-126 to 2^123: 6 times it is in range
        wt.s = torch.from_numpy(np.repeat(s8[:, None], 4, 1)).to(DEV)
        wt.scale = np.repeat(np.ldexp(1.0, s8.astype(int) - 127)[:, None], 4, 1)
    wt.w = torch.from_numpy(wt.codes).to(DEV)
    x = torch.eye(H).to(torch.bfloat16)
    got, _ = _run(wt, x, "f32")
    want, size = wt.exact(x.double().numpy())
    # a single term: exact; INT4 takes 24 s from (code + 16) s, whose rounding is of that size;
    # what is below fp32's normal range may be flushed
    tol = (0 if fmt == "fp4" else 2.0 ** -23) * size + 2.0 ** -126
    assert (np.abs(got - want) <= tol).all(), np.argwhere(np.abs(got - want) > tol)[:5]


def test_nan_scale_reaches_its_row_only():
    wt = Weights(200, 256, "fp4", 32, seed=4)
    wt.s[77, 3] = 255
    x = _x(np.random.default_rng(5), 3, 256)
    got, _ = _run(wt, x, "f32")
    assert np.isnan(got[:, 77]).all() and np.isfinite(np.delete(got, 77, 1)).all()


@pytest.mark.parametrize("fmt,V,H", [("fp4", 1000, 512), ("int4", 1000, 512), ("fp4", 20000, 160), ("int4", 50000, 160)])
def test_rows_do_not_depend_on_each_other(fmt, V, H):
    wt = Weights(V, H, fmt, 32, seed=6)
    x = _x(np.random.default_rng(7), 40, H)
    got, raw = _run(wt, x, "f32")
    again, _ = _run(wt, x, "f32")
    assert np.array_equal(got, again)
    y = x.clone()
    y[7] = float("nan")
    y[20] = float("inf")
    other, _ = _run(wt, y, "f32")
    keep = [m for m in range(40) if m not in (7, 20)]
    assert np.array_equal(other[keep], got[keep])
    assert not np.isfinite(other[[7, 20]]).any()
