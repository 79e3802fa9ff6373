"""GPU parity of the losses over a vocabulary (ssm_xent_*, ssm_distill_*) against the 64-bit
reference, to the bars that model_ref.py derives."""
import numpy as np
import pytest

import model_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


def pair(a, dtype=BF16):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to("cuda", dtype)
    return t, t.double().cpu().numpy()


def draw(T, D, V, seed=0, size=2.0):
    r = np.random.default_rng([seed, T, D, V])
    return r, pair(r.standard_normal((T, D))), pair(r.standard_normal((V, D)) * size / np.sqrt(D))


def near(got, want, off, what):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    bad = np.where(np.isnan(want), -1.0, np.abs(got - want) - (off * 1.01 + 1e-37))
    assert bad.max(initial=-1) <= 0, (what, float(bad.max()), np.unravel_index(bad.argmax(), bad.shape))


def targets(r, T, V):
    t = r.integers(0, V, T)
    t[0], t[-1] = V - 1, 0
    if T > 4:
        t[r.random(T) < 0.2] = -100
    return t


def check_xent(T, D, V, scale=1.0, z_loss=0.0, seed=0, place=None, target=None, grads=True):
    say(f"xent {T} x {D} x {V}")
    r, x, w = draw(T, D, V, seed)
    target = targets(r, T, V) if target is None else target
    tx, tw, tt = x[0], w[0], torch.from_numpy(target).cuda()
    if place:
        tx, tw = place(tx), place(tw)
    h = ref.Head(x[1], w[1], scale)
    loss, off, soft, hard = h.xent(target, z_loss)
    got_loss, got_lse = ssm.ssm_xent_fwd(tx, tw, tt, scale, z_loss)
    near(got_lse, h.lse, h.lse_off, "lse")
    near(got_loss, loss, off, "loss")
    if not grads:
        return
    dloss = pair(r.standard_normal(T), F32)
    g = ssm.ssm_xent_bwd(dloss[0], tx, tw, tt, got_lse, scale, z_loss)
    takes = (target >= 0) & (target < V)
    for n, (v, o) in zip(("dx", "dweight"), h.grad(dloss[1], soft, hard, takes)):
        near(g[n], v, o, n)
    assert not g["dx"][torch.from_numpy(~takes).cuda()].any()


SIZES = [(1, 8, 1), (1, 64, 300), (3, 72, 257), (5, 256, 1000), (17, 136, 255), (64, 64, 256), (100, 320, 50), (129, 512, 513),
         (255, 200, 700), (256, 64, 512), (257, 128, 1025), (300, 1000, 90), (600, 96, 2000), (33, 2560, 1111)]


@pytest.mark.parametrize("T,D,V", SIZES)
def test_xent(T, D, V):
    check_xent(T, D, V)


@pytest.mark.parametrize("scale,z_loss", [(0.25, 0.0), (-1.5, 1e-2), (1.0, 1e-4), (0.0, 0.0)])
def test_xent_scale_and_z_loss(scale, z_loss):
    check_xent(70, 128, 600, scale, z_loss)


def far(t):
    """The same rows, apart, between others' values."""
    big = torch.full((t.shape[0], t.shape[1] + 72), float("nan"), device="cuda", dtype=t.dtype)
    big[:, 8:8 + t.shape[1]].copy_(t)
    return big[:, 8:8 + t.shape[1]]


@pytest.mark.parametrize("T,D,V", [(70, 72, 300), (300, 136, 600)])
def test_xent_of_slices(T, D, V):
    check_xent(T, D, V, place=far)


def distill_inputs(r, T, V, K, holes=True):
    index = np.stack([r.permutation(V)[:K] if K <= V else r.integers(0, V, K) for _ in range(T)])
    teacher = np.float32(r.standard_normal((T, K)) * 3)
    if holes:
        index[r.random((T, K)) < 0.1] = -1
        teacher[r.random((T, K)) < 0.1] = -np.inf
        index[0, 0], teacher[0, 0] = V - 1, 1.0
    return index, teacher


def check_distill(T, D, V, K, temperature=1.0, scale=1.0, seed=0, place=None, given=None):
    say(f"distill {T} x {D} x {V}, {K}")
    r, x, w = draw(T, D, V, seed)
    index, teacher = given or distill_inputs(r, T, V, K)
    tx, tw, ti, tt = x[0], w[0], torch.from_numpy(index).cuda(), torch.from_numpy(teacher).cuda()
    if place:
        tx, tw = place(tx), place(tw)
    h = ref.Head(x[1], w[1], scale, temperature)
    loss, off, soft, hard = h.distill(index, teacher)
    got_loss, got_lse, logits = ssm.ssm_distill_fwd(tx, tw, ti, tt, temperature, scale)
    near(got_lse, h.lse, h.lse_off, "lse")
    near(got_loss, loss, off, "loss")
    rows, at = np.arange(T)[:, None], np.clip(index, 0, V - 1)
    inside = (index >= 0) & (index < V)
    near(logits, np.where(inside, h.z[rows, at], 0.0), np.where(inside, h.z_off[rows, at], 0.0), "logits")
    dloss = pair(r.standard_normal(T), F32)
    g = ssm.ssm_distill_bwd(dloss[0], tx, tw, ti, tt, got_lse, logits, temperature, scale)
    takes = soft > 0
    for n, (v, o) in zip(("dx", "dweight"), h.grad(dloss[1], soft, hard, takes)):
        near(g[n], v, o, n)
    assert not g["dx"][torch.from_numpy(~takes).cuda()].any()


@pytest.mark.parametrize("T,D,V", SIZES)
@pytest.mark.parametrize("K", [1, 5])
def test_distill(T, D, V, K):
    check_distill(T, D, V, K)


@pytest.mark.parametrize("K,V", [(64, 1000), (65, 300), (130, 400), (1024, 1500), (300, 20)])
def test_distill_many(K, V):
    """More indices than a wavefront, and more than the vocabulary has (the same index often)."""
    check_distill(40, 64, V, K, 2.0)


@pytest.mark.parametrize("temperature,scale", [(0.5, 1.0), (4.0, 1.0), (2.0, -0.7)])
def test_distill_temperature(temperature, scale):
    check_distill(50, 128, 500, 20, temperature, scale)


def test_distill_of_slices():
    check_distill(300, 136, 600, 9, place=far)


def test_distill_holes():
    """Rows without an index, with the same one throughout, without weight, with one past the vocabulary."""
    V, K = 300, 6
    index = np.array([[-1] * K, [7] * K, [0, 1, 2, 3, 4, 5], [299, 0, 0, 1, -5, 299], [0, 1, 300, 2, 3, 4], [256, 255, 257, 1, 2, 3]])
    teacher = np.float32(np.random.default_rng(0).standard_normal((6, K)))
    teacher[2] = -np.inf
    check_distill(6, 64, V, K, given=(index, teacher))


def test_targets_past_the_vocabulary():
    check_xent(6, 64, 300, target=np.array([0, 300, 299, 1 << 40, -1, -(1 << 62)]))


@pytest.mark.parametrize("kind", ["xent", "distill"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_padding_may_hold_anything(kind, bad):
    """Rows without a target do not reach the gradients, even where they are not finite; their loss is 0."""
    T, D, V = 300, 64, 520
    r, x, w = draw(T, D, V)
    tx, tw = x[0].clone(), w[0]
    none = torch.from_numpy(r.random(T) < 0.3).cuda()
    if kind == "xent":
        target = torch.from_numpy(r.integers(0, V, T)).cuda()
        target[none] = -1

        def run(x):
            loss, lse = ssm.ssm_xent_fwd(x, tw, target)
            return loss, ssm.ssm_xent_bwd(torch.ones(T, device="cuda"), x, tw, target, lse)
    else:
        index = torch.from_numpy(r.integers(0, V, (T, 4))).cuda()
        index[none] = -1
        teacher = torch.randn(T, 4, device="cuda")

        def run(x):
            loss, lse, z = ssm.ssm_distill_fwd(x, tw, index, teacher)
            return loss, ssm.ssm_distill_bwd(torch.ones(T, device="cuda"), x, tw, index, teacher, lse, z)
    loss, g = run(tx)
    tx[none] = bad
    loss2, g2 = run(tx)
    assert torch.equal(loss, loss2) and not loss[none].any()
    for n in g:
        assert torch.equal(g[n], g2[n]), n


def test_large_logits():
    """Logits in the hundreds: the softmax is one row's maximum, its gradient exact zeros elsewhere."""
    T, D, V = 40, 64, 700
    r, x, w = draw(T, D, V, size=200.0)
    target = r.integers(0, V, T)
    h = ref.Head(x[1], w[1])
    loss, off, soft, hard = h.xent(target)
    got, lse = ssm.ssm_xent_fwd(x[0], w[0], torch.from_numpy(target).cuda())
    near(lse, h.lse, h.lse_off, "lse")
    near(got, loss, off, "loss")
    dloss = pair(r.standard_normal(T), F32)
    g = ssm.ssm_xent_bwd(dloss[0], x[0], w[0], torch.from_numpy(target).cuda(), lse)
    for n, (v, o) in zip(("dx", "dweight"), h.grad(dloss[1], soft, hard, np.ones(T, bool))):
        near(g[n], v, o, n)


def test_values_that_are_not_finite_stay_in_their_row():
    T, D, V = 40, 64, 700
    r, x, w = draw(T, D, V)
    target = torch.from_numpy(r.integers(0, V, T)).cuda()
    clean = ssm.ssm_xent_fwd(x[0], w[0], target)
    x[0][7, 3] = float("nan")
    loss, lse = ssm.ssm_xent_fwd(x[0], w[0], target)
    other = torch.arange(T, device="cuda") != 7
    assert torch.isnan(loss[7]) and torch.isnan(lse[7])
    assert torch.equal(loss[other], clean[0][other]) and torch.equal(lse[other], clean[1][other])
    g = ssm.ssm_xent_bwd(torch.ones(T, device="cuda"), x[0], w[0], target, lse)
    assert torch.isnan(g["dx"][7]).all() and torch.isfinite(g["dx"][other]).all()


def test_one_gradient_alone():
    r, x, w = draw(100, 64, 300)
    target = torch.from_numpy(r.integers(0, 300, 100)).cuda()
    _, lse = ssm.ssm_xent_fwd(x[0], w[0], target)
    d = torch.ones(100, device="cuda")
    both = ssm.ssm_xent_bwd(d, x[0], w[0], target, lse)
    for n, kw in (("dx", {"want_weight": False}), ("dweight", {"want_x": False})):
        g = ssm.ssm_xent_bwd(d, x[0], w[0], target, lse, **kw)
        assert list(g) == [n] and torch.equal(g[n], both[n])
    assert ssm.ssm_xent_bwd(d, x[0], w[0], target, lse, want_x=False, want_weight=False) == {}


def test_no_rows():
    x, w, t = torch.empty(0, 64, device="cuda", dtype=BF16), torch.randn(30, 64, device="cuda").bfloat16(), torch.empty(0, device="cuda", dtype=torch.int64)
    loss, lse = ssm.ssm_xent_fwd(x, w, t)
    assert loss.shape == lse.shape == (0,)
    g = ssm.ssm_xent_bwd(loss, x, w, t, lse)
    assert g["dx"].shape == (0, 64) and not g["dweight"].any()


def test_leading_dimensions():
    r, x, w = draw(24, 64, 300)
    target = torch.from_numpy(r.integers(0, 300, 24)).cuda()
    a = ssm.ssm_xent_fwd(x[0], w[0], target)
    b = ssm.ssm_xent_fwd(x[0].view(2, 12, 64), w[0], target.view(2, 12))
    assert torch.equal(a[0], b[0].flatten()) and b[1].shape == (2, 12)
    g = ssm.ssm_xent_bwd(torch.ones(2, 12, device="cuda"), x[0].view(2, 12, 64), w[0], target.view(2, 12), b[1])
    assert g["dx"].shape == (2, 12, 64)


def test_pieces_of_the_vocabulary():
    """Rows so many that dz of the whole vocabulary takes several pieces: sampled rows and columns."""
    T, D, V = 40000, 64, 8300
    say("xent in pieces")
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(T, D, device="cuda", generator=g).bfloat16()
    w = (torch.randn(V, D, device="cuda", generator=g) / 4).bfloat16()
    target = torch.randint(0, V, (T,), device="cuda", generator=g)
    dloss = torch.randn(T, device="cuda", generator=g)
    loss, lse = ssm.ssm_xent_fwd(x, w, target)
    got = ssm.ssm_xent_bwd(dloss, x, w, target, lse)
    some = np.r_[0:40, 20000:20040, T - 40:T]
    h = ref.Head(x[some].double().cpu().numpy(), w.double().cpu().numpy())
    want, off, soft, hard = h.xent(target[some].cpu().numpy())
    near(loss[some], want, off, "loss")
    near(lse[some], h.lse, h.lse_off, "lse")
    near(got["dx"][some], *h.grad(dloss[some].double().cpu().numpy(), soft, hard, np.ones(len(some), bool))[0], "dx")
    # columns of the vocabulary at the pieces' borders, from the logits in 64 bits on the GPU
    cols = torch.tensor([0, 1, 3327, 3328, 3329, 6655, 6656, 8191, 8299], device="cuda")
    z = x.double() @ w[cols].double().t()
    p = torch.exp(z - torch.logsumexp(x.double() @ w.double().t(), -1, keepdim=True))
    dz = (p - (target[:, None] == cols).double()) * dloss.double()[:, None]
    want = dz.t() @ x.double()
    size = dz.abs().t() @ x.double().abs()
    # dz: its rounding, and an exponential whose argument is off by 2^-18; T products in fp32
    bar = (2.0 ** -8 + 2.0 ** -17 + 2 * T * 2.0 ** -24) * size + 2.0 ** -8 * want.abs() + \
        2.0 ** -17 * (dloss.double().abs()[:, None] * p).t() @ x.double().abs()
    assert ((got["dweight"][cols].double() - want).abs() <= bar).all()


# ------------------------------------------- sizes of many tiles, in 64 bits on the GPU


def check_many_tiles(T, D, V, K=None, place=lambda t: t, seed=0):
    """As check_xent and check_distill (K indices), with the reference and its bars on the GPU."""
    say(f"many tiles {T} x {D} x {V}, {K}")
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = place(torch.randn(T, D, device="cuda", generator=g).bfloat16())
    w = place((torch.randn(V, D, device="cuda", generator=g) * 2 / D ** 0.5).bfloat16())
    dloss = torch.randn(T, device="cuda", generator=g)
    xd, wd, dd, U = x.double(), w.double(), dloss.double()[:, None], ref.U
    z = xd @ wd.t()
    z_off = 2 * (D + 4) * U * (xd.abs() @ wd.abs().t())
    lse = torch.logsumexp(z, -1)
    lse_off = z_off.amax(-1) + U * (300 + 8 * z.amax(-1).abs() + 8 * lse.abs())
    if K is None:
        target = torch.randint(0, V, (T,), device="cuda", generator=g)
        target[torch.rand(T, device="cuda", generator=g) < 0.2] = -1
        takes = target >= 0
        at = target.clamp(min=0)[:, None]
        loss, got_lse = ssm.ssm_xent_fwd(x, w, target)
        want = torch.where(takes, lse - z.gather(1, at)[:, 0], 0.0)
        off = lse_off + z_off.gather(1, at)[:, 0] + 4 * U * (lse.abs() + z.gather(1, at)[:, 0].abs())
        hard = torch.zeros_like(z).scatter_(1, at, 1.0)
        got = ssm.ssm_xent_bwd(dloss, x, w, target, got_lse)
    else:
        index = torch.rand(T, V, device="cuda", generator=g).topk(K, -1).indices
        teacher = torch.randn(T, K, device="cuda", generator=g) * 3
        takes = torch.ones(T, dtype=torch.bool, device="cuda")
        loss, got_lse, logits = ssm.ssm_distill_fwd(x, w, index, teacher)
        logq = torch.log_softmax(teacher.double(), -1)
        mine = z.gather(1, index)
        assert ((logits.double() - mine).abs() <= z_off.gather(1, index) * 1.01).all()
        want = (logq.exp() * (logq - mine + lse[:, None])).sum(-1)
        size = (logq.exp() * (logq.abs() + mine.abs() + lse[:, None].abs())).sum(-1)
        off = (logq.exp() * z_off.gather(1, index)).sum(-1) + lse_off + U * (size * (200 + K) + 100)
        hard = torch.zeros_like(z).scatter_(1, index, logq.exp())
        got = ssm.ssm_distill_bwd(dloss, x, w, index, teacher, got_lse, logits)
    assert ((got_lse.double() - lse).abs() <= lse_off * 1.01).all()
    assert ((loss.double() - want).abs() <= off * 1.01).all()
    p = torch.exp(z - lse[:, None])
    f = torch.where(takes[:, None], dd, 0.0)
    dz = f * (p - hard)
    dz_off = f.abs() * (p * (z_off + lse_off[:, None] + 8 * U * (z.abs() + lse.abs()[:, None] + 4)) + 60 * U * (p + hard)) * 1.01
    dz_off = dz_off + 2.0 ** -8 * (dz.abs() + dz_off)
    for name, a, a_off, b in (("dx", dz, dz_off, wd), ("dweight", dz.t(), dz_off.t(), xd)):
        v = a @ b
        bar = a_off @ b.abs() + 2 * (a.shape[1] + 8) * U * (a.abs() @ b.abs()) + 2.0 ** -8 * v.abs() * 1.01
        worst = ((got[name].double() - v).abs() / (bar * 1.01 + 1e-37)).max().item()
        assert worst <= 1, (name, worst)
    assert not got["dx"][~takes].any()


# (large tiles in one piece, in several, with a ragged end of each dimension; rows in slices; columns in slices)
@pytest.mark.parametrize("T,D,V", [(1100, 1160, 21003), (2100, 72, 9000), (6100, 304, 1341), (40, 1032, 30001), (700, 2056, 4099)])
@pytest.mark.parametrize("K", [None, 12])
def test_many_tiles(T, D, V, K):
    check_many_tiles(T, D, V, K)


@pytest.mark.parametrize("T,D,V", [(13000, 264, 12100)])
def test_many_tiles_in_pieces(T, D, V):
    check_many_tiles(T, D, V)


@pytest.mark.parametrize("T,D,V,K", [(2100, 72, 19000, 128), (1100, 136, 21003, 300), (700, 64, 4099, 1024), (1500, 64, 2570, 1024),
                                     (40, 1032, 30001, 100), (400, 72, 30001, 1000), (8, 64, 5000, 1024)])
def test_many_indices_of_many_tiles(T, D, V, K):
    check_many_tiles(T, D, V, K)


def test_many_indices_in_one_place():
    """1024 indices of which most are one column, and none elsewhere; others are past the vocabulary or negative."""
    T, D, V, K = 1500, 64, 3001, 1024
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = torch.randn(T, D, device="cuda", generator=g).bfloat16(), torch.randn(V, D, device="cuda", generator=g).bfloat16() / 8
    index = torch.full((T, K), V - 1, device="cuda")
    index[:, ::3] = -1
    index[:, 5] = 255
    index[7, 9], index[8] = V, -1
    teacher = torch.zeros(T, K, device="cuda")
    loss, lse, z = ssm.ssm_distill_fwd(x, w, index, teacher)
    wide = x.double() @ w.double().t()
    at = index.clamp(0, V - 1)
    has = ((index >= 0) & (index < V)).double()
    assert ((z.double() - wide.gather(1, at) * has).abs() <= 2 * (D + 4) * ref.U * (x.double().abs() @ w.double().abs().t()).gather(1, at) * 1.01).all()
    q = has / has.sum(-1, keepdim=True)
    assert torch.isnan(loss[7]) and loss[8] == 0
    d = torch.ones(T, device="cuda")
    got = ssm.ssm_distill_bwd(d, x, w, index, teacher, lse, z)
    assert not got["dx"][7:9].any()
    takes = torch.ones(T, dtype=torch.bool, device="cuda")
    takes[7:9] = False
    p = torch.softmax(wide, -1)
    dz = torch.where(takes[:, None], p.scatter_add(1, at, -q.nan_to_num()), 0.0)
    # dz is rounded once and the result once; its own error, some 300 roundings of fp32, is below a sixteenth of that
    bar = 2.0 ** -8 * 1.07 * (dz.abs().t() @ x.double().abs()) + 2.0 ** -8 * (dz.t() @ x.double()).abs() + 1e-6
    assert ((got["dweight"].double() - dz.t() @ x.double()).abs() <= bar).all()


def test_many_tiles_of_slices():
    check_many_tiles(1100, 520, 21003, place=far)


@pytest.mark.parametrize("T", [1, 3, 16])
@pytest.mark.parametrize("D", [8, 72, 2048, 2056, 4096, 4104])
def test_few_rows(T, D):
    """Weights streamed, x in LDS for either of its sizes, and the width past it."""
    check_many_tiles(T, D, 2600)
    check_many_tiles(T, D, 33, 5)


def test_bits_repeat():
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = torch.randn(700, 264, device="cuda", generator=g).bfloat16(), torch.randn(9000, 264, device="cuda", generator=g).bfloat16() / 8
    index, teacher = torch.randint(0, 9000, (700, 20), device="cuda", generator=g), torch.randn(700, 20, device="cuda", generator=g)
    d, first = torch.randn(700, device="cuda", generator=g), None
    for _ in range(4):
        loss, lse, z = ssm.ssm_distill_fwd(x, w, index, teacher, 2.0)
        now = [loss, lse, z, *ssm.ssm_distill_bwd(d, x, w, index, teacher, lse, z, 2.0).values()]
        loss, lse = ssm.ssm_xent_fwd(x, w, index[:, 0].contiguous())
        now += [loss, lse, *ssm.ssm_xent_bwd(d, x, w, index[:, 0].contiguous(), lse).values()]
        first = first or now
        for a, b in zip(now, first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,V", [(5, 3000), (200, 3000), (2100, 9000)])
def test_logits_of_minus_infinity(T, V):
    """Whole tiles of them beside logits far below zero; rows of nothing else have lse minus infinity."""
    D = 64
    x = torch.ones(T, D, device="cuda", dtype=torch.bfloat16)
    w = torch.full((V, D), -60.0, device="cuda", dtype=torch.bfloat16)
    w[:2000], w[2500:] = float("-inf"), float("-inf")
    target = torch.full((T,), 2100, device="cuda")
    loss, lse = ssm.ssm_xent_fwd(x, w, target)
    want = -60.0 * D + np.log(500.0)
    # 64 sums of 60, a conversion of base there and back, and a logarithm
    bar = 400 * ref.U * 60 * D
    assert ((lse.double() - want).abs() <= bar).all() and ((loss.double() - np.log(500.0)).abs() <= 2 * bar).all()
    index = target[:, None].expand(T, 3).contiguous()
    loss, lse, z = ssm.ssm_distill_fwd(x, w, index, torch.zeros(T, 3, device="cuda"))
    assert ((lse.double() - want).abs() <= bar).all() and (z == -60.0 * D).all()
    w[:] = float("-inf")
    assert torch.isneginf(ssm.ssm_xent_fwd(x, w, target)[1]).all()


@pytest.mark.parametrize("T,K", [(10, 4), (300, 4), (1500, 1024)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.4e38])
def test_what_stands_beside_no_index(T, K, bad):
    """Teacher's logits without an index, and x and dloss of rows without any, may be anything: same bits."""
    D, V = 64, 3001
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = torch.randn(T, D, device="cuda", generator=g).bfloat16(), torch.randn(V, D, device="cuda", generator=g).bfloat16() / 8
    index = torch.randint(0, V, (T, K), device="cuda", generator=g)
    index[torch.rand(T, K, device="cuda", generator=g) < 0.3] = -1
    none = torch.rand(T, device="cuda", generator=g) < 0.3
    none[0], none[1], index[1, 0] = True, False, 5
    index[none] = -7
    teacher, d = torch.randn(T, K, device="cuda", generator=g), torch.randn(T, device="cuda", generator=g)

    def run():
        loss, lse, z = ssm.ssm_distill_fwd(x, w, index, teacher, 2.0)
        grads = ssm.ssm_distill_bwd(d, x, w, index, teacher, lse, z, 2.0)
        return [loss, z, grads["dx"], grads["dweight"]]
    first = run()
    teacher[index < 0] = bad
    empty = (index < 0).all(-1)
    x[empty], d[empty] = bad, bad
    for a, b in zip(run(), first):
        assert torch.equal(a, b) and torch.isfinite(a).all()
    assert not first[0][empty].any() and not first[2][empty].any()


@pytest.mark.parametrize("T", [10, 300])
def test_gradients_beside_no_target(T):
    """dloss of rows without a target may be anything."""
    x, w = torch.randn(T, 64, device="cuda").bfloat16(), torch.randn(500, 64, device="cuda").bfloat16() / 8
    target = torch.arange(T, device="cuda") % 400
    target[::3] = -1
    _, lse = ssm.ssm_xent_fwd(x, w, target)
    d = torch.randn(T, device="cuda")
    first = ssm.ssm_xent_bwd(d, x, w, target, lse)
    d[::3], lse[::3] = float("nan"), float("inf")
    again = ssm.ssm_xent_bwd(d, x, w, target, lse)
    for n in first:
        assert torch.equal(first[n], again[n]) and torch.isfinite(first[n]).all()


@pytest.mark.parametrize("temperature", [0.5, 1.0, 3.0])
def test_teachers_of_the_lowest_value(temperature):
    """Logits of fp32's lowest value are without weight beside others, and equal ones alone."""
    T, D, V, K = 40, 64, 500, 6
    x, w = torch.randn(T, D, device="cuda").bfloat16(), torch.randn(V, D, device="cuda").bfloat16() / 8
    index = torch.rand(T, V, device="cuda").topk(K, -1).indices
    teacher = torch.randn(T, K, device="cuda")
    lowest = torch.finfo(F32).min
    some = teacher.clone()
    some[:, 2:4] = lowest
    some[::2] = lowest
    plain = some.clone()
    plain[:, 2:4] = float("-inf")
    plain[::2] = 1.5
    d = torch.randn(T, device="cuda")
    results = []
    for t in (some, plain):
        loss, lse, z = ssm.ssm_distill_fwd(x, w, index, t, temperature)
        assert (loss > 0).all()
        results.append([loss, *ssm.ssm_distill_bwd(d, x, w, index, t, lse, z, temperature).values()])
    for a, b in zip(*results):
        assert torch.equal(a, b)
