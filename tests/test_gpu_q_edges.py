"""Further edges of the calls around verification."""
import numpy as np
import pytest

from oracle import rules as R

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
