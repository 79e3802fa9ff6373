"""Training steps of several operators, held to the same steps in 64 bits with bf16 roundings at
the same places: what is left is where a value lies so near a rounding's border that fp32's
errors decide it.

Bars, by the norm of the difference over the norm: a rounding to bf16 is off by at most 2^-8 of a
value, by 2^-8 / sqrt(3) of it in the mean square over a binade's values; two results whose roundings
have come out entirely independent of each other differ by sqrt(2) of that, 3.2e-3, a rounding.
Counted are those between a result and what is given."""
import os
import sys

import pytest

from gpu_util import say
from test_model_gpu import ROOT, randn, train_step

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F = torch.nn.functional
F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
EACH = (2 / 3) ** 0.5 * 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


def rb(t):
    return t.to(BF16).double()


def stage(f, inputs, dout=None):
    """f's outputs for detached inputs, and a function from their gradients to the inputs'."""
    leaves = [t.detach().clone().requires_grad_() for t in inputs]
    out = f(*leaves)

    def back(*grads):
        outs = out if isinstance(out, tuple) else (out,)
        return torch.autograd.grad(outs, leaves, [g.expand_as(o) for g, o in zip(grads, outs)])
    return (tuple(t.detach() for t in out) if isinstance(out, tuple) else out.detach()), back


def norm(r, w):
    return r / torch.sqrt((r * r).mean(-1, keepdim=True) + 1e-5) * w


def head(y, w, target, dloss, teacher=None, t=1.0):
    """(loss, dy, dweight) of rows y."""
    z = y @ w.t() / t
    lse = torch.logsumexp(z, -1, keepdim=True)
    p = torch.exp(z - lse)
    if teacher is None:
        takes, at = target >= 0, target.clamp(min=0)[..., None]
        loss = torch.where(takes, (lse - z.gather(-1, at))[..., 0], 0.0)
        dz = p.scatter_add(-1, at, -torch.ones_like(at, dtype=F64)) * torch.where(takes, dloss, 0.0)[..., None]
    else:
        logq = torch.log_softmax(teacher[1].double() / t, -1)
        loss = t * t * (logq.exp() * (logq - z.gather(-1, teacher[0]) + lse)).sum(-1)
        dz = p.scatter_add(-1, teacher[0], -logq.exp()) * (t * dloss)[..., None]
    dz = rb(dz)
    return loss, rb(dz @ w), rb(dz.flatten(0, -2).t() @ y.flatten(0, -2))


def errors(got, want):
    return {n: ((got[n].double() - want[n]).norm() / want[n].norm()).item() for n in want}


def recurrence(xs, rs, ins, rate):
    a = torch.exp(-rate * torch.sigmoid(rs))
    b = torch.sqrt(-torch.expm1(-2 * rate * torch.sigmoid(rs))) * torch.sigmoid(ins) * xs
    h, hs = torch.zeros_like(b[:, 0]), []
    for t in range(b.shape[1]):
        h = a[:, t] * h + b[:, t]
        hs.append(h)
    return torch.stack(hs, 1)


@pytest.mark.parametrize("kind", ["xent", "distill"])
def test_recurrence_norm_and_loss(kind):
    say(f"training step's roundings: {kind}")
    B, L, D, V, K = 2, 200, 128, 777, 10
    x, w_in, w_out = randn(B, L, D), randn(3 * D, D, seed=1) / 12, randn(V, D, seed=2) / 8
    rate, w_norm = randn(D, dtype=F32, seed=3).abs() + 0.05, 1 + 0.1 * randn(D, dtype=F32, seed=4)
    gen = torch.Generator(device="cuda").manual_seed(0)
    target = torch.randint(0, V, (B, L), device="cuda", generator=gen)
    target[0, :20] = -1
    teacher = None
    if kind == "distill":
        teacher = torch.rand(B, L, V, device="cuda", generator=gen).topk(K, -1).indices, randn(B, L, K, dtype=F32, seed=5) * 2
    got = train_step(x, w_in, rate, w_norm, w_out, target, teacher)

    xd, wi, ra, wn, wo = (t.double() for t in (x, w_in, rate, w_norm, w_out))
    gates = rb(xd @ wi.t()).chunk(3, -1)
    h, h_back = stage(recurrence, (*gates, ra))
    r = xd + rb(h)
    y, res = rb(norm(r, wn)), rb(r)
    loss, dy, dweight = head(y, wo, target, torch.full((B, L), 1.0 / target.numel(), device="cuda", dtype=F64), teacher,
                             1.0 if teacher is None else 2.0)
    _, n_back = stage(norm, (res, wn))
    dres, dnorm = n_back(dy)
    dres = rb(dres)
    *dgates, drate = h_back(dres)
    dproj = torch.cat([rb(t) for t in dgates], -1)
    want = {"loss": loss, "dweight": dweight, "dnorm": dnorm, "drate": drate,
            "dw_in": dproj.flatten(0, 1).t() @ xd.flatten(0, 1), "dx": dproj @ wi + dres}
    found = errors(got, want)
    say(str(found))
    # the projection, the states, the norm; back dz, dy, the norm's gradient, the gates'; a weight's gradient
    counts = {"loss": 3, "dweight": 5, "dnorm": 6, "drate": 6, "dw_in": 7, "dx": 7}
    for n, e in found.items():
        assert e <= counts[n] * EACH, (n, e, counts[n] * EACH)


def test_example_block():
    """The example's block, as above: its norm, projection, linear attention, gated norm, output and last norm
    are six roundings; back there are dz, dy, the last norm's gradient, the product's, the gated norm's, linear
    attention's, the projection's and the first norm's."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import linattn_block
    finally:
        sys.path.pop(0)
    say("example's roundings")
    block = linattn_block.LinAttnBlock(width=512, heads=6, groups=3, dim=64, group=64)
    B, L, D, V = 2, 96, 512, 1000
    gen = torch.Generator(device="cpu").manual_seed(2)
    x = torch.randn(B, L, D, generator=gen).to("cuda", BF16)
    res = torch.randn(B, L, D, generator=gen).to("cuda")
    vocab = (torch.randn(V, D, generator=gen) * D ** -0.5).to("cuda", BF16)
    target = torch.randint(-1, V, (B, L), generator=gen).to("cuda")
    loss, got = block.train(x, res, vocab, target)

    H, G, d = block.H, block.G, block.d
    nw, wi, hw, wo, bias, lw = (t.double() for t in (block.norm_weight, block.w_in, block.head_weight, block.w_out, block.decay_bias,
                                                     block.last_weight))

    def attention(q, k, v, a, bias):
        q, k = (t.unflatten(-1, (G, d)).repeat_interleave(H // G, -2) for t in (q, k))
        v, decay = v.unflatten(-1, (H, d)), torch.exp(-F.softplus(a + bias))
        S, ys = x.new_zeros(B, H, d, d, dtype=F64), []
        for t in range(L):
            S = decay[:, t, :, None, None] * S + v[:, t, :, :, None] * k[:, t, :, None, :]
            ys.append((S * q[:, t, :, None, :]).sum(-1) * d ** -0.5)
        return torch.stack(ys, 1).flatten(2)

    def gated(y, z, hw):
        return norm(y.unflatten(-1, (H, d)), hw.view(H, d)).flatten(2) * F.silu(z)

    r, r_back = stage(lambda x, res: res + x, (x.double(), res.double()))
    un, u_back = stage(norm, (r, nw))
    u = rb(un)
    p = rb(u @ wi.t())
    q, k, v, z, a = p[..., :sum(block.sizes)].split(block.sizes, -1)
    yn, y_back = stage(attention, (q, k, v, a, bias))
    y = rb(yn)
    on, o_back = stage(gated, (y, z, hw))
    o = rb(on)
    out = rb(o @ wo.t())
    last, l_back = stage(norm, (r + out, lw))
    dloss = (target >= 0) / (target >= 0).sum().double()
    want_loss, dy, dhead = head(rb(last), vocab.double(), target, dloss)
    dlast, dlw = l_back(dy)
    dout = rb(dlast)
    dyn, dz, dhw = o_back(rb(dout @ wo))
    dq, dk, dv, da, dbias = y_back(rb(dyn))
    dp = torch.cat([*(rb(t) for t in (dq, dk, dv, dz, da)), p.new_zeros(B, L, p.shape[-1] - sum(block.sizes))], -1)
    dr, dnw = u_back(rb(dp @ wi))
    dr = dr + dlast
    want = {"loss": want_loss, "norm_weight": dnw, "head_weight": dhw, "decay_bias": dbias, "last_weight": dlw, "head": dhead, "x": dr,
            "residual": dr, "w_in": dp.flatten(0, 1).t() @ u.flatten(0, 1), "w_out": dout.flatten(0, 1).t() @ o.flatten(0, 1)}
    found = errors({**got, "loss": loss}, want)
    say(str(found))
    counts = {"loss": 6, "head": 8, "last_weight": 8, "w_out": 10, "head_weight": 10, "decay_bias": 11, "w_in": 13, "norm_weight": 13,
              "x": 14, "residual": 14}
    assert set(counts) == set(want) and set(got) == set(want) - {"loss"}
    for n, e in found.items():
        assert e <= counts[n] * EACH, (n, e, counts[n] * EACH)
