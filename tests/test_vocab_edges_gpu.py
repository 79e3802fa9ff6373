"""The losses over a vocabulary where rows of weights end, and at their smallest and largest sizes, against
the 64-bit reference."""
import numpy as np
import pytest

import model_ref as ref
from gpu_util import say
from test_vocab_gpu import check_distill, check_xent, draw, far, near, pair

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32, BF16 = torch.float32, torch.bfloat16


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


@pytest.mark.parametrize("T", [1, 5, 16])
@pytest.mark.parametrize("D", [8, 72, 2056])
def test_few_rows_of_slices(T, D):
    """Rows of packed tensors between values that are NaN."""
    check_xent(T, D, 333, -1.5, 1e-2, place=far)
    check_distill(T, D, 333, 5, 2.0, 0.7, place=far)


@pytest.mark.parametrize("T", [1, 16, 17, 300])
@pytest.mark.parametrize("V", [1, 2, 9])
def test_small_vocabularies(T, V):
    check_xent(T, 72, V, z_loss=1e-2)
    check_distill(T, 72, V, 3)


def test_few_rows_past_32_bits():
    """Weights and their gradient of more than 2^32 bytes, streamed to registers: the last rows'."""
    say("few rows past 32 bits")
    V, D, T = 600001, 4088, 3
    w = torch.empty(V, D, device="cuda", dtype=BF16)
    assert w.numel() * 2 > 1 << 32
    w.normal_(std=0.02, generator=torch.Generator(device="cuda").manual_seed(0))
    x = torch.randn(T, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    target = torch.tensor([V - 1, V - 300, 0], device="cuda")
    loss, lse = ssm.ssm_xent_fwd(x, w, target)
    parts = [(x.double() @ part.double().t(), x.double().abs() @ part.double().abs().t()) for part in w.chunk(32)]
    z, size = (torch.cat(p, -1) for p in zip(*parts))
    want, top = torch.logsumexp(z, -1), z.amax(-1)
    z_off = 2 * (D + 4) * ref.U * size
    off = z_off.amax(-1) + ref.U * (300 + 8 * top.abs() + 8 * want.abs())
    assert ((lse.double() - want).abs() <= off * 1.01).all()
    mine = z.gather(1, target[:, None])[:, 0]
    assert ((loss.double() - (want - mine)).abs() <= (off + z_off.gather(1, target[:, None])[:, 0] + 4 * ref.U * (want + mine.abs())) * 1.01).all()
    d = torch.ones(T, device="cuda")
    g = ssm.ssm_xent_bwd(d, x, w, target, lse)
    dz = torch.exp(z - want[:, None])
    p_off = dz * (z_off + off[:, None] + 8 * ref.U * (z.abs() + want[:, None] + 4))
    dz[torch.arange(T), target] -= 1
    # dz: what its exponential's argument is off by, its factors, its rounding; the products' sums and rounding
    dz_off = p_off + 60 * ref.U * (dz.abs() + 1e-30) + 2.0 ** -8 * 1.01 * dz.abs()
    last = slice(V - 400, V)
    v = dz[:, last].t() @ x.double()
    bar = dz_off[:, last].t() @ x.double().abs() + 2 * (T + 8) * ref.U * (dz[:, last].abs().t() @ x.double().abs()) + 2.0 ** -8 * 1.01 * v.abs()
    assert ((g["dweight"][last].double() - v).abs() <= bar + 1e-37).all()
    v, bar = torch.zeros(T, D, device="cuda", dtype=torch.float64), torch.zeros(T, D, device="cuda", dtype=torch.float64)
    for at in range(0, V, 20000):
        part = w[at:at + 20000].double()
        v += dz[:, at:at + 20000] @ part
        bar += (dz_off + 2 * (V + 8) * ref.U * dz.abs())[:, at:at + 20000] @ part.abs()
    assert ((g["dx"].double() - v).abs() <= bar + 2.0 ** -8 * 1.01 * v.abs()).all()
