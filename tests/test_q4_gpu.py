"""GPU parity of the products with 4-bit weights (ssm_q4_*) against the 64-bit
references, through the C ABI.

Bars, from the arithmetic: the operands are exact, so only fp32 sums round.  A
group's product sums up to 128 terms x (16 + code), at most 31 |x| each, in the
matrix cores and takes (16 + zero) sum x away: 128 + 20 roundings of 2^-24 of 62
sum |x|; the groups add up in fp32, k / 32 roundings more of sums that are no
larger.  Relative to scale sum |x| over a row: 62 * 148 * 2^-24 = 5.5e-4 at the
worst; roundings are as often up as down and grow with the square root of their
number: held to 62 * 4 * sqrt(148 + k / 32) * 2^-24 of max(scale) sum |x|.  A bf16
result adds 2^-8 of itself.
"""
import numpy as np
import pytest

import block_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


def pair(a, dtype):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dtype)
    return t.cuda(), (t.double().numpy() if t.is_floating_point() else t.numpy())


def weights(r, n, k, group, scale_dt, zeros):
    codes = pair(r.integers(0, 256, (n, k // 2)), torch.uint8)
    scales = pair(r.uniform(0.5, 1.5, (n, k // group)) / np.sqrt(k), scale_dt)
    z = pair(r.integers(0, 16, (n, k // group)), torch.uint8) if zeros else (None, None)
    return codes, scales, z


def near(got, x, w, top, bias=None):
    want = x @ w.T + (0.0 if bias is None else bias)
    bar = 62 * 4 * np.sqrt(148 + x.shape[1] / 32) * 2.0 ** -24 * top * np.abs(x).sum(1, keepdims=True) + 2.0 ** -22 * np.abs(want)
    if got.dtype == BF16:
        bar = bar + 2.0 ** -8 * np.abs(want)
    y = got.double().cpu().numpy()
    assert y.shape == want.shape and not np.isnan(y).any()
    off = np.abs(y - want)
    assert (off <= bar).all(), f"off {off.max():.3e}, bar {bar.min():.3e}"


@pytest.mark.parametrize("m", [1, 2, 5, 6, 16, 17, 21, 22, 48, 64, 65, 130])
@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (33, 96, 32), (64, 128, 128), (31, 1024, 64), (100, 1152, 128), (257, 544, 32),
                                       (65, 64, 64)])
def test_matvec(m, n, k, group):
    say(f"q4 m {m} n {n} k {k} group {group}")
    r = np.random.default_rng(m * 131 + n)
    zeros, scale_dt = (n + m) % 2 == 0, BF16 if m % 2 else F32
    (c, ce), (s, se), (z, ze) = weights(r, n, k, group, scale_dt, zeros)
    w = ref.q4_weights(ce, se, ze, group)
    b, be = pair(r.standard_normal(n), F32) if m % 3 else (None, None)
    for dt in (BF16, F32):
        x, xe = pair(r.standard_normal((m, k)), dt)
        near(ssm.ssm_q4_matvec(x, c, s, z, b, out_dtype=F32), xe, w, se.max(), be)
    near(ssm.ssm_q4_matvec(x.bfloat16(), c, s, z, b), x.bfloat16().double().cpu().numpy(), w, se.max(), be)


def test_wide_and_many_columns():
    say("q4: more columns than one workgroup per CU, long rows")
    r = np.random.default_rng(3)
    n, k = 16500, 4128
    (c, ce), (s, se), (z, ze) = weights(r, n, k, 32, BF16, True)
    x, xe = pair(r.standard_normal((3, k)), BF16)
    near(ssm.ssm_q4_matvec(x, c, s, z, out_dtype=F32), xe, ref.q4_weights(ce, se, ze, 32), se.max())


def test_strided_rows_leading_dimensions_and_empty():
    say("q4: x as a slice, leading dimensions, no rows, no columns")
    r = np.random.default_rng(4)
    (c, ce), (s, se), (z, ze) = weights(r, 40, 256, 64, F32, True)
    w = ref.q4_weights(ce, se, ze, 64)
    wide, we = pair(r.standard_normal((2, 3, 512)), BF16)
    out = ssm.ssm_q4_matvec(wide[..., 128:384], c, s, z, out_dtype=F32)
    assert out.shape == (2, 3, 40)
    near(out.reshape(6, 40), we[..., 128:384].reshape(6, 256), w, se.max())
    assert ssm.ssm_q4_matvec(wide[:0, 0, :256], c, s, z).shape == (0, 40)
    out = ssm.ssm_q4_matvec(wide[0, :, :256].contiguous(), c[:0], s[:0])
    assert out.shape == (3, 0)


def test_values_that_are_not_finite_stay_in_their_row():
    say("q4: a row with NaN or infinity")
    r = np.random.default_rng(5)
    (c, _), (s, _), _ = weights(r, 70, 128, 64, F32, False)
    for dt in (BF16, F32):
        x = torch.randn(20, 128, device="cuda").to(dt)
        clean = ssm.ssm_q4_matvec(x, c, s)
        x[7, 5], x[9, 100] = float("nan"), float("inf")
        out = ssm.ssm_q4_matvec(x, c, s)
        keep = [i for i in range(20) if i not in (7, 9)]
        assert torch.equal(out[keep], clean[keep]) and not torch.isfinite(out[[7, 9]]).any()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt,scale_dt", [(F32, F32), (BF16, BF16), (BF16, F32)])
def test_quantize(group, dt, scale_dt):
    say(f"q4 quantize group {group} {dt} {scale_dt}")
    r = np.random.default_rng(group)
    a = r.standard_normal((37, 256))
    a[3] = 0.0                                  # a row of zeros
    a[4] = np.abs(a[4])                         # one sign only
    a[5] = -np.abs(a[5])
    w, we = pair(a, dt)
    c, s, z = ssm.ssm_q4_quantize(w, group, scale_dt)
    assert c.shape == (37, 128) and s.dtype == scale_dt and int(z.max()) <= 15
    se = s.double().cpu().numpy()
    got = ref.q4_weights(c.cpu().numpy(), se, z.cpu().numpy(), group)
    g = we.reshape(37, -1, group)
    span = np.maximum(g.max(-1), 0) - np.minimum(g.min(-1), 0)
    np.testing.assert_allclose(se, span / 15, rtol=2.0 ** -8 if scale_dt == BF16 else 1e-6)
    # half a step of the code and half of the zero point, and where a bf16 scale
    # was rounded down, 15 steps of 2^-9 past the range's end
    lim = (1.0 + (15 * 2.0 ** -8 if scale_dt == BF16 else 1e-5)) * np.repeat(se, group, 1)
    assert (np.abs(got - we) <= lim + 1e-12).all()
    assert not got[3].any()
    # the product with what was quantised
    x, xe = pair(r.standard_normal((2, 256)), BF16)
    near(ssm.ssm_q4_matvec(x, c, s, z, out_dtype=F32), xe, got, se.max())


def test_repeats_bitwise():
    say("q4: the same bits twice")
    r = np.random.default_rng(6)
    (c, _), (s, _), (z, _) = weights(r, 1000, 1024, 128, F32, True)
    x = torch.randn(40, 1024, device="cuda")
    assert torch.equal(ssm.ssm_q4_matvec(x, c, s, z), ssm.ssm_q4_matvec(x, c, s, z))
