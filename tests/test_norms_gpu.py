"""GPU parity of the norms around a block (ssm_add_norm_*, ssm_gated_norm_*)
against the 64-bit references, through the C ABI.

Bars, from the arithmetic: the statistics are fp32 sums of at most 16 terms per
lane, then a tree over the lanes and up to 16 wavefronts: below 40 roundings of
2^-24 each, the square root's reciprocal, the exponential and the reciprocal of
the gate add a few units in the last place (and |z| 2^-23 through the
exponent), so a value is within 40 * 2^-24 + 12 * 2^-23 < 4e-6 of its row's largest;
held to 1e-5 of it.  A bf16 result adds its rounding, 2^-9 of the value (held to
2^-8).  A column sum adds the rounding of a chain of at most 120 terms (rows of one
workgroup, then the workgroups): 120 * 2^-24 = 7.2e-6 of the sum of magnitudes, plus
the terms' own 4e-6, which for a factor that comes out of the norm is 4e-6 of its
row's largest: held to 2e-5 of the sum of those magnitudes.
"""
import numpy as np
import pytest

import block_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5
ROW, ROUND, COL = 1e-5, 2.0 ** -8, 2e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


class Draw:
    """Seeded tensors on the GPU, with their exact values in 64 bits."""

    def __init__(self, seed):
        self.r = np.random.default_rng(seed)

    def __call__(self, shape, dtype=F32, std=1.0, lo=None, hi=None, pad=None):
        """``pad``: a slice of a wider tensor, as a packed projection gives."""
        a = self.r.standard_normal(shape) * std if lo is None else self.r.uniform(lo, hi, shape)
        t = torch.from_numpy(a).to(dtype)
        exact = t.double().numpy()
        if pad:
            wide = torch.full((*shape[:-1], shape[-1] + pad), float("nan"), dtype=dtype)
            wide[..., 1:1 + shape[-1]] = t
            return wide.cuda()[..., 1:1 + shape[-1]], exact
        return t.cuda(), exact


def near(got, want, name, groups=1):
    """Rows within ROW of their largest value, and the type's rounding."""
    y = got.double().cpu().numpy()
    assert y.shape == want.shape, name
    if not want.size:
        return
    w = want.reshape(*want.shape[:-1], groups, -1)
    top = np.repeat(np.abs(w).max(-1, keepdims=True), w.shape[-1], -1).reshape(want.shape)
    bar = ROW * top + (ROUND * np.abs(want) if got.dtype == BF16 else 0.0)
    bad = np.abs(y - want) - bar
    assert not np.isnan(y).any() and bad.max() <= 0, f"{name}: {np.abs(y - want).max():.3e} off, bar {bar.max():.3e}"


def near_sum(got, rows, factor, name, groups=1):
    """``rows``: the terms; ``factor``: what of each does not come out of the norm."""
    rest = np.divide(rows, factor, out=np.zeros_like(rows), where=factor != 0).reshape(rows.shape[0], groups, -1)
    top = np.repeat(np.abs(rest).max(-1, keepdims=True), rest.shape[-1], -1).reshape(rows.shape)
    off = np.abs(got.double().cpu().numpy() - rows.sum(0))
    bar = COL * (np.abs(factor) * top).sum(0)
    assert (off <= bar).all(), f"{name}: {off.max():.3e} off"


WIDTHS = [(3, 1), (5, 2), (9, 7), (7, 8), (70, 9), (33, 64), (6, 130), (17, 512), (5, 513), (4, 1000), (3, 1024), (3, 1025),
          (1, 2560), (700, 2563), (2, 5120), (2, 8192)]


@pytest.mark.parametrize("rows,width", WIDTHS)
@pytest.mark.parametrize("x_dt,res_dt", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)])
def test_add_norm(rows, width, x_dt, res_dt):
    say(f"add_norm rows {rows} width {width} x {x_dt} residual {res_dt}")
    d = Draw(rows * 10007 + width)
    center, full = width % 2 == 1, width % 3 != 0
    x, xe = d((rows, width), x_dt, pad=5 if width > 8 else None)
    res, rese = d((rows, width), res_dt, 3.0)
    w, we = d((width,), lo=0.5, hi=1.5)
    b, be = d((width,), std=0.1) if full else (None, None)
    sc, sce = d((width,), lo=0.1, hi=1.0) if full else (None, None)
    out, r = ssm.ssm_add_norm_fwd(x, res, w, b, sc, alpha=0.75, eps=EPS, center=center)
    assert out.dtype == x_dt and r.dtype == res_dt
    want, rr = ref.add_norm(xe, rese, we, be, sce, 0.75, EPS, center)
    if width > 1 or not center:
        near(out, want, "out")
    near(r, rr, "residual_out")
    # backward from the stored r
    re_ = r.double().cpu().numpy()
    dout, de = d((rows, width), x_dt)
    dres, dre = d((rows, width), res_dt)
    g = ssm.ssm_add_norm_bwd(dout, r, w, dres, x=x, scale=sc, alpha=0.75, eps=EPS, center=center, want_bias=True,
                             want_scale=True)
    dx, dr, dw, db, ds = ref.add_norm_grad(de, re_, we, dre, xe, sce, 0.75, EPS, center)
    if width == 1 and center:
        return  # every norm is 0 / sqrt(eps): the gradients are those of the residual alone, up to cancellation
    near(g["dx"], dx, "dx")
    near(g["dresidual"], dr, "dresidual")
    near_sum(g["dweight"], dw, de, "dweight")
    near_sum(g["dbias"], db, de, "dbias")
    near_sum(g["dscale"], ds, xe, "dscale")


@pytest.mark.parametrize("rows,width", [(4, 96), (9, 1500), (5, 77)])
def test_add_norm_without_options_and_in_place(rows, width):
    say(f"add_norm plain and in place, rows {rows} width {width}")
    d = Draw(width)
    x, xe = d((rows, width), BF16)
    res, rese = d((rows, width))
    out, r = ssm.ssm_add_norm_fwd(x, out_dtype=F32)   # no residual, weight, bias, scale
    assert r.dtype == F32
    near(out, ref.norm(xe, None, None, EPS, False), "out")
    near(r, xe, "r")
    want = ssm.ssm_add_norm_fwd(x, res)
    kept = res.clone()
    got = ssm.ssm_add_norm_fwd(x, kept, residual_out=kept)
    assert got[1].data_ptr() == kept.data_ptr()
    assert torch.equal(got[0], want[0]) and torch.equal(kept, want[1])
    dout, de = d((rows, width), BF16)
    g = ssm.ssm_add_norm_bwd(dout, r, want_weight=False)
    assert set(g) == {"dx", "dresidual"}
    near(g["dx"], ref.add_norm_grad(de, xe, None, None, None, None, 1.0, EPS, False)[0], "dx")


@pytest.mark.parametrize("rows,width,groups", [(3, 6, 3), (5, 64, 8), (2, 40, 1), (7, 5120, 80), (40, 330, 10), (1, 513, 1),
                                               (9, 1040, 2), (3, 2600, 2), (2, 8192, 1), (600, 1536, 1), (1030, 192, 3)])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("gate_first", [True, False])
def test_gated_norm(rows, width, groups, dt, gate_first):
    say(f"gated_norm rows {rows} width {width} groups {groups} {dt} gate_first {gate_first}")
    d = Draw(rows + width * 31)
    center = groups % 2 == 0
    x, xe = d((rows, width), dt, 2.0, pad=8)
    z, ze = d((rows, width), dt, 2.0, pad=3)
    w, we = d((width,), lo=0.5, hi=1.5)
    b, be = d((width,), std=0.1) if groups % 3 else (None, None)
    out = ssm.ssm_gated_norm_fwd(x, z, w, b, ngroups=groups, gate_first=gate_first, eps=EPS, center=center)
    near(out, ref.gated_norm(xe, ze, we, be, groups, gate_first, EPS, center), "out", groups)
    dout, de = d((rows, width), dt)
    g = ssm.ssm_gated_norm_bwd(dout, x, z, w, b, ngroups=groups, gate_first=gate_first, eps=EPS, center=center)
    dx, dz, dw, db = ref.gated_norm_grad(de, xe, ze, we, be, groups, gate_first, EPS, center)
    dw, db = dw.reshape(rows, width), db.reshape(rows, width)
    near(g["dx"], dx, "dx", groups)
    near(g["dz"], dz, "dz", groups)
    gated = de if gate_first else de * ref.silu(ze)   # what the norm's output gets
    near_sum(g["dweight"], dw, gated, "dweight", groups)
    assert ("dbias" in g) == (b is not None)
    if b is not None:
        near_sum(g["dbias"], db, gated, "dbias", groups)


def test_gated_norm_without_a_gate_and_types():
    say("gated_norm: no gate, fp32 out of bf16, three dimensions")
    d = Draw(5)
    x, xe = d((2, 3, 256), BF16)
    w, we = d((256,), lo=0.5, hi=1.5)
    out = ssm.ssm_gated_norm_fwd(x, weight=w, ngroups=4, out_dtype=F32)
    assert out.dtype == F32 and out.shape == (2, 3, 256)
    near(out, ref.gated_norm(xe, None, we, None, 4, True, EPS, False), "out", 4)
    dout, de = d((2, 3, 256))
    g = ssm.ssm_gated_norm_bwd(dout, x, weight=w, ngroups=4)
    assert set(g) == {"dx", "dweight"}
    near(g["dx"], ref.gated_norm_grad(de, xe, None, we, None, 4, True, EPS, False)[0], "dx", 4)


def test_empty_and_special_rows():
    say("norms: no rows, zero rows, infinities and NaN stay in their row")
    w = torch.ones(64, device="cuda")
    out, r = ssm.ssm_add_norm_fwd(torch.empty(0, 64, device="cuda"), weight=w)
    assert out.shape == (0, 64)
    g = ssm.ssm_add_norm_bwd(torch.empty(0, 64, device="cuda"), r, w)
    assert torch.equal(g["dweight"], torch.zeros(64, device="cuda"))
    for width in (64, 1500):
        x = torch.randn(5, width, device="cuda")
        clean, _ = ssm.ssm_add_norm_fwd(x)
        x[1] = 0.0
        x[2, 3] = float("inf")
        x[3, 5] = float("nan")
        out, _ = ssm.ssm_add_norm_fwd(x)
        assert torch.equal(out[0], clean[0]) and torch.equal(out[4], clean[4])
        assert torch.equal(out[1], torch.zeros_like(out[1]))
        assert torch.isnan(out[3]).all() and torch.isnan(out[2, 3])


def test_results_repeat_bitwise():
    say("norms: the same bits twice, on another stream too")
    x, res = torch.randn(1000, 2560, device="cuda").bfloat16(), torch.randn(1000, 2560, device="cuda")
    w = torch.rand(2560, device="cuda")
    a = ssm.ssm_add_norm_bwd(x, res, w, res)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = ssm.ssm_add_norm_bwd(x, res, w, res, stream=s)
    s.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]), n
