"""Gradients of the losses over several pieces of the vocabulary, in slices and not (the cuts:
test_vocab_pieces.py), every column of dx and dweight against 64 bits on the GPU."""
import pytest

import model_ref as ref
from gpu_util import say
from test_vocab_pieces import CUTS

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

U = ref.U


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    assert torch.cuda.get_device_properties(0).multi_processor_count == 256, "the cuts are those of 256 CUs"
    ssm.library()


@pytest.mark.parametrize("T,D,V", list(CUTS))
@pytest.mark.parametrize("K", [None, 12])
def test_gradients_over_pieces(T, D, V, K):
    """Both gradients in one call, and each alone (which is cut otherwise).  Bars as in model_ref.Head."""
    say(f"pieces {T} x {D} x {V}, {K}")
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(T, D, device="cuda", generator=g).bfloat16()
    w = (torch.randn(V, D, device="cuda", generator=g) * 2 / D ** 0.5).bfloat16()
    dloss = torch.randn(T, device="cuda", generator=g)
    xd, wd, d = x.double(), w.double(), dloss.double()[:, None]
    z = xd @ wd.t()
    lse = torch.logsumexp(z, -1, keepdim=True)
    z_off = 2 * (D + 4) * U * (xd.abs() @ wd.abs().t())
    lse_off = z_off.amax(-1, keepdim=True) + U * (300 + 8 * z.amax(-1, keepdim=True).abs() + 8 * lse.abs())
    if K is None:
        target = torch.randint(0, V, (T,), device="cuda", generator=g)
        target[:4] = torch.tensor([0, V - 1, V // 2, 8191], device="cuda")
        target[torch.rand(T, device="cuda", generator=g) < 0.1] = -1
        takes, at = target >= 0, target.clamp(min=0)[:, None]
        q = torch.ones_like(at, dtype=torch.float64)
        loss, got_lse = ssm.ssm_xent_fwd(x, w, target)
        want = torch.where(takes, (lse - z.gather(1, at))[:, 0], 0.0)
        off = (lse_off + z_off.gather(1, at))[:, 0] + 4 * U * (lse.abs() + z.gather(1, at).abs())[:, 0]

        def call(**kw):
            return ssm.ssm_xent_bwd(dloss, x, w, target, got_lse, **kw)
    else:
        # evenly apart in a row, from a place of its own: each piece has some, none twice
        at = (torch.randint(0, V, (T, 1), device="cuda", generator=g) + torch.arange(K, device="cuda") * (V // K)) % V
        takes = torch.ones(T, dtype=torch.bool, device="cuda")
        teacher = torch.randn(T, K, device="cuda", generator=g) * 3
        logq = torch.log_softmax(teacher.double(), -1)
        q = logq.exp()
        loss, got_lse, logits = ssm.ssm_distill_fwd(x, w, at, teacher)
        mine = z.gather(1, at)
        want = (q * (logq - mine + lse)).sum(-1)
        size = (q * (logq.abs() + mine.abs() + lse.abs())).sum(-1)
        off = (q * z_off.gather(1, at)).sum(-1) + lse_off[:, 0] + U * (size * (200 + K) + 100)

        def call(**kw):
            return ssm.ssm_distill_bwd(dloss, x, w, at, teacher, got_lse, logits, **kw)
    assert ((got_lse.double() - lse[:, 0]).abs() <= lse_off[:, 0] * 1.01).all()
    assert ((loss.double() - want).abs() <= off * 1.01).all()
    # dz (in place of z) and what it is off by (in place of z_off): its exponential's argument, its factors, its rounding
    f = torch.where(takes[:, None], d, 0.0)
    z_off += lse_off + 8 * U * (lse.abs() + 4)
    z_off += 8 * U * z.abs()
    p = z.sub_(lse).exp_()
    z_off *= p
    z_off += 60 * U * p
    z_off.scatter_add_(1, at, 60 * U * q)
    z_off *= f.abs() * 1.01
    dz = p.scatter_add_(1, at, -q).mul_(f)
    dz_off = z_off.add_(2.0 ** -8 * 1.01 * dz.abs())
    bars = {}
    for name, a, a_off, b in (("dx", dz, dz_off, wd), ("dweight", dz.t(), dz_off.t(), xd)):
        v = a @ b
        bars[name] = v, (a_off @ b.abs() + 2 * (a.shape[1] + 8) * U * (a.abs() @ b.abs()) + 2.0 ** -8 * v.abs() * 1.01) * 1.01 + 1e-37
    del z, p, z_off, dz, dz_off
    for wants in (dict(), dict(want_weight=False), dict(want_x=False)):
        got = call(**wants)
        assert set(got) == {n for n, k in (("dx", "want_x"), ("dweight", "want_weight")) if wants.get(k, True)}
        for name, t in got.items():
            v, bar = bars[name]
            worst = ((t.double() - v).abs() / bar).max().item()
            say(f"{name} {wants}: {worst:.2f} of its bar")
            assert worst <= 1, (name, wants, worst)
        if "dx" in got:
            assert not got["dx"][~takes].any()
