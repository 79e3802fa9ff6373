"""Norms without an epsilon over rows whose squares lie below fp32's smallest normal number.
The square root's reciprocal has to take them as they are.  Rows are exact powers of two
times small integers, so that sums of squares are exact also where they are denormal; the bar is the
norms' own (1e-5 of a row's largest value)."""
import numpy as np
import pytest

import block_ref as ref
from gpu_util import say
from test_norms_gpu import near

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32 = torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


def rows(width, power):
    r = np.random.default_rng(width)
    return r.choice([-3.0, -2.0, -1.0, 1.0, 2.0, 3.0], (3, width)) * 2.0 ** power


@pytest.mark.parametrize("width", [4, 64, 1000, 2048])
@pytest.mark.parametrize("power", [-64, -66])
@pytest.mark.parametrize("center", [False, True])
def test_small_rows(width, power, center):
    """(mean squares between 2^-132 and 2^-125: the smallest normal number is 2^-126)"""
    say(f"norms of width {width}, rows of 2^{power}, center {center}")
    x = rows(width, power)
    if center:
        x[:, 1::2] = -x[:, ::2]         # (a mean of zero, exactly)
    t = torch.from_numpy(x).float().cuda()
    want = ref.norm(x, None, None, 0.0, center)
    out, _ = ssm.ssm_add_norm_fwd(t, eps=0.0, center=center)
    near(out, want, "add norm")
    near(ssm.ssm_gated_norm_fwd(t, eps=0.0, center=center), want, "norm")
    dy = np.random.default_rng(1).choice([-1.0, 0.5, 2.0], x.shape) * 2.0 ** -40      # (gradients grow by the reciprocal)
    d = torch.from_numpy(dy).float().cuda()
    wd, ww, _ = ref.norm_grad(dy, x, None, 0.0, center)
    g = ssm.ssm_add_norm_bwd(d, t, eps=0.0, center=center)
    near(g["dx"], wd, "dx of the add norm")
    near(g["dweight"], ww.sum(0), "dweight")
    g = ssm.ssm_gated_norm_bwd(d, t, eps=0.0, center=center)
    near(g["dx"], wd, "dx of the norm")
