"""The losses over a vocabulary where rows of weights end, against the 64-bit reference."""
import numpy as np
import pytest

import model_ref as ref
from gpu_util import say
from test_vocab_gpu import draw, near, pair

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32 = torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


@pytest.mark.parametrize("T", [1, 5, 16, 17])
@pytest.mark.parametrize("D", [8, 64, 72, 120, 2056, 4088])
@pytest.mark.parametrize("K", [None, 3])
def test_words_masked_by_a_weight(T, D, K):
    """A column of x that is 1 and whose weight is minus infinity for some words, first in its row: their logits are
    minus infinity, whatever the width, and everything else is as without those words."""
    say(f"masked words {T} x {D}, {K}")
    V = 300
    r, x, w = draw(T, D, V)
    x[0][:, 0] = 1
    x[1][:, 0] = 1
    masked = r.random(V) < 0.3
    masked[0], masked[7], masked[V - 1] = False, True, False
    w[0][torch.from_numpy(masked).cuda(), 0] = float("-inf")
    kept = np.flatnonzero(~masked)
    h = ref.Head(x[1], w[1][kept])
    dloss = pair(r.standard_normal(T), F32)
    if K is None:
        target = r.integers(0, len(kept), T)
        t = torch.from_numpy(kept[target]).cuda()
        loss, off, soft, hard = h.xent(target)
        got, lse = ssm.ssm_xent_fwd(x[0], w[0], t)
        g = ssm.ssm_xent_bwd(dloss[0], x[0], w[0], t, lse)
    else:
        index = np.stack([r.permutation(len(kept))[:K] for _ in range(T)])
        teacher = np.float32(r.standard_normal((T, K)))
        t, tt = torch.from_numpy(kept[index]).cuda(), torch.from_numpy(teacher).cuda()
        loss, off, soft, hard = h.distill(index, teacher)
        got, lse, z = ssm.ssm_distill_fwd(x[0], w[0], t, tt)
        g = ssm.ssm_distill_bwd(dloss[0], x[0], w[0], t, tt, lse, z)
    near(lse, h.lse, h.lse_off, "lse")
    near(got, loss, off, "loss")
    dx, dw = h.grad(dloss[1], soft, hard, np.ones(T, bool))
    near(g["dweight"][torch.from_numpy(kept).cuda()], *dw, "dweight")
    assert not g["dweight"][torch.from_numpy(masked).cuda()].any()
    # (dx of the column itself sums 0 times minus infinity)
    near(g["dx"][:, 1:], dx[0][:, 1:], dx[1][:, 1:], "dx")
