"""The model operators (include/ssmmodel.h) as a program uses them: together, captured in
HIP graphs, on other streams, refused calls, tensors past 2^31 elements."""
import os
import sys

import numpy as np
import pytest

import model_ref as ref
from gpu_util import say
from test_graph_gpu import _capture

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32, BF16 = torch.float32, torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


def randn(*shape, dtype=BF16, seed=0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return torch.randn(*shape, generator=g).to("cuda", dtype)


def operators():
    """name -> a call without arguments; its outputs are new tensors on every call."""
    x, r, i = (randn(3, 700, 130, seed=s) for s in range(3))
    rate, S = randn(130, dtype=F32, seed=3).abs(), randn(3, 130, dtype=F32, seed=4)
    dout = randn(3, 700, 130, seed=5)
    states = torch.empty(3, 22, 130, device="cuda")
    ssm.ssm_gscan_fwd(x, r, i, rate, initial_state=S, states=states)
    h, w = randn(300, 136, seed=6), randn(1000, 136, seed=7) / 8
    few = h[:5].contiguous()
    t = torch.randint(-1, 1000, (300,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(0))
    index = torch.randint(0, 1000, (300, 9), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    teacher, d = randn(300, 9, dtype=F32, seed=8), randn(300, dtype=F32, seed=9)
    _, lse = ssm.ssm_xent_fwd(h, w, t)
    _, warm, z = ssm.ssm_distill_fwd(h, w, index, teacher, 2.0)

    def forward():
        last, kept = torch.empty_like(S), torch.empty_like(states)
        return ssm.ssm_gscan_fwd(x, r, i, rate, initial_state=S, last_state=last, states=kept), last, kept
    return {
        "gscan_fwd": forward,
        "gscan_fwd, one tile": lambda: (ssm.ssm_gscan_fwd(x[:, :100].contiguous(), r[:, :100].contiguous()),),
        "gscan_bwd": lambda: ssm.ssm_gscan_bwd(x, r, i, rate, dout, states, dlast_state=S, want_dinitial_state=True).values(),
        "gscan_update": lambda: (ssm.ssm_gscan_update(S.clone(), x[:, 0].contiguous(), r[:, 0].contiguous(), i[:, 0].contiguous(), rate),),
        "xent_fwd": lambda: ssm.ssm_xent_fwd(h, w, t),
        "xent_fwd, few rows": lambda: ssm.ssm_xent_fwd(few, w, t[:5].contiguous()),
        "xent_bwd": lambda: ssm.ssm_xent_bwd(d, h, w, t, lse).values(),
        "xent_bwd, few rows": lambda: ssm.ssm_xent_bwd(d[:5].contiguous(), few, w, t[:5].contiguous(), lse[:5].contiguous()).values(),
        "distill_fwd": lambda: ssm.ssm_distill_fwd(h, w, index, teacher, 2.0),
        "distill_bwd": lambda: ssm.ssm_distill_bwd(d, h, w, index, teacher, warm, z, 2.0).values(),
    }


NAMES = ("gscan_fwd", "gscan_fwd, one tile", "gscan_bwd", "gscan_update", "xent_fwd", "xent_fwd, few rows", "xent_bwd", "xent_bwd, few rows",
         "distill_fwd", "distill_bwd")


@pytest.mark.parametrize("name", NAMES)
def test_graph_replays(name):
    say(f"graph: {name}")
    call = operators()[name]
    want = [t.clone() for t in call()]
    got = []

    def run():
        got[:] = call()
    g = _capture(run)
    for r in range(4):
        for t in got:
            t.fill_(float("nan"))
        call()          # eager work between the replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), f"replay {r}: output {i} differs from the eager result"


@pytest.mark.parametrize("name", NAMES)
def test_graph_of_a_shape_not_met_before(name):
    """Captured calls whose workspace is the library's own, part of the graph."""
    from sequence_scan_amd import block
    say(f"graph, own workspace: {name}")
    call = operators()[name]
    want = [t.clone() for t in call()]
    got = []

    def run():
        block._wanted.clear()
        got[:] = call()
    g = _capture(run)
    for r in range(3):
        for t in got:
            t.fill_(float("nan"))
        call()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), f"replay {r}: output {i} differs from the eager result"


def test_two_graphs_in_turn():
    """Two captured chains, replayed in turn and on two streams at once, keep apart."""
    say("two graphs")
    calls = operators()
    want = {n: [t.clone() for t in calls[n]()] for n in ("gscan_fwd", "gscan_bwd")}
    got, graphs = {}, {}
    for n in want:
        def run(n=n):
            got[n] = list(calls[n]())
        graphs[n] = _capture(run)
    for _ in range(3):
        for n in want:
            for t in got[n]:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in want]
        for s, g in zip(streams, graphs.values()):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for n in want:
            for a, b in zip(got[n], want[n]):
                assert torch.equal(a, b), n


@pytest.mark.parametrize("name", NAMES)
def test_another_stream(name):
    say(f"stream: {name}")
    call = operators()[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        busy = torch.ones(1 << 26, device="cuda")
        for _ in range(8):
            busy.mul_(1.5)
        got = [t.clone() for t in call()]
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_several_streams_at_once():
    """The same calls on four streams without waiting: chains that run side by side."""
    say("four streams")
    x, r = randn(2, 4000, 256), randn(2, 4000, 256, seed=1)
    want = ssm.ssm_gscan_fwd(x, r)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(4)], []
    for _ in range(6):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(ssm.ssm_gscan_fwd(x, r))
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g, want)


def test_given_stream():
    x, r = randn(1, 300, 66), randn(1, 300, 66, seed=1)
    want = ssm.ssm_gscan_fwd(x, r)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.empty_like(want)
    ssm.ssm_gscan_fwd(x, r, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_workspace_from_either_side():
    """A shape's first call takes its workspace from the library, later ones from PyTorch."""
    from sequence_scan_amd import block
    for name, call in operators().items():
        block._wanted.clear()
        first = [t.clone() for t in call()]
        assert any(block._wanted.values()) == (name not in ("gscan_fwd, one tile", "gscan_update")), name
        for _ in range(2):
            torch.empty(1 << 20, device="cuda").fill_(float("nan"))
            for a, b in zip(call(), first):
                assert torch.equal(a, b), name


def test_refused_calls_write_nothing():
    x, r = randn(2, 40, 64), randn(2, 40, 64, seed=1)
    S = torch.full((2, 64), 7.0, device="cuda")
    out, states = torch.full_like(x, 7), torch.full((2, 2, 64), 7.0, device="cuda")
    wide = torch.empty(1, 1, (1 << 24) + 8, device="cuda", dtype=BF16)
    cases = {
        "shape": (ValueError, lambda: ssm.ssm_gscan_fwd(x, r[:, :39], out=out, last_state=S, states=states)),
        "type": (TypeError, lambda: ssm.ssm_gscan_fwd(x, r.float(), out=out, last_state=S, states=states)),
        "rate": (ValueError, lambda: ssm.ssm_gscan_fwd(x, r, None, randn(63, dtype=F32), out=out, last_state=S, states=states)),
        "states": (ValueError, lambda: ssm.ssm_gscan_fwd(x, r, out=out, last_state=S, states=states[:, :1])),
        "out on x": (ssm.SSMError, lambda: ssm.ssm_gscan_fwd(out, r, out=out, last_state=S)),
        "width": (ssm.SSMError, lambda: ssm.ssm_gscan_fwd(wide, wide)),
        "rate wanted": (ssm.SSMError, lambda: ssm.ssm_gscan_bwd(x, r, None, None, x, states, want_rate=True)),
        "update": (ssm.SSMError, lambda: ssm.ssm_gscan_update(S, out[:, 0], r[:, 0].contiguous(), out=out.view(-1, 64)[:2])),
    }
    for name, (error, call) in cases.items():
        say(f"refusal: {name}")
        with pytest.raises(error):
            call()
        torch.cuda.synchronize()
        for t in (out, S, states):
            assert torch.all(t == 7), f"{name}: a refused call wrote an output"
    h, w, t = randn(8, 64), randn(100, 64), torch.zeros(8, dtype=torch.int64, device="cuda")
    for error, call in ((ssm.SSMError, lambda: ssm.ssm_xent_fwd(h.float(), w.float(), t)),
                        (ssm.SSMError, lambda: ssm.ssm_xent_fwd(h[:, :60], w[:, :60], t)),
                        (ssm.SSMError, lambda: ssm.ssm_xent_fwd(randn(8, 67)[:, 3:], w, t)),
                        (ssm.SSMError, lambda: ssm.ssm_xent_fwd(h, w, t, scale=float("nan"))),
                        (ValueError, lambda: ssm.ssm_xent_fwd(h, w, t[:7])),
                        (ssm.SSMError, lambda: ssm.ssm_distill_fwd(h, w, t[:, None], randn(8, 1, dtype=F32), temperature=0.0))):
        with pytest.raises(error):
            call()


# ------------------------------------------------------------------------- together


def train_step(x, w_in, rate, w_norm, w_out, target, teacher=None):
    """A recurrent layer between two projections, its norm, and the loss; all gradients, by hand."""
    B, L, D = x.shape
    proj = torch.matmul(x, w_in.t())                                    # x, r, i of the layer, packed
    gates = proj.chunk(3, -1)
    states = torch.empty(B, -(-L // ssm.SSM_GSCAN_SEGMENT), D, device="cuda")
    h = ssm.ssm_gscan_fwd(*gates, rate, states=states)
    y, res = ssm.ssm_add_norm_fwd(h, x, w_norm)
    n = target.numel()
    dloss = torch.full(target.shape, 1.0 / n, device="cuda")
    if teacher is None:
        loss, lse = ssm.ssm_xent_fwd(y, w_out, target)
        g = ssm.ssm_xent_bwd(dloss, y, w_out, target, lse)
    else:
        loss, lse, z = ssm.ssm_distill_fwd(y, w_out, *teacher, temperature=2.0)
        g = ssm.ssm_distill_bwd(dloss, y, w_out, *teacher, lse, z, temperature=2.0)
    gn = ssm.ssm_add_norm_bwd(g["dx"], res, w_norm, x=h)
    gs = ssm.ssm_gscan_bwd(*gates, rate, gn["dx"], states)
    dproj = torch.cat([gs["dx"], gs["dr"], gs["di"]], -1)
    return {"loss": loss, "dweight": g["dweight"], "dnorm": gn["dweight"], "drate": gs["drate"],
            "dw_in": torch.matmul(dproj.flatten(0, 1).t().contiguous().float(), x.flatten(0, 1).float()),
            "dx": torch.matmul(dproj.float(), w_in.float()) + gn["dresidual"].float()}


@pytest.mark.parametrize("kind", ["xent", "distill"])
def test_a_training_step(kind):
    """Recurrence, norm and loss with all gradients, against float64 autograd of the same formulas.  About six
    roundings to bf16 (2^-8 each) lie between the input and a loss, and as many again back to a gradient, of
    values up to about four times those they are summed with: 12 * 4 * 2^-8 = 0.19 of the largest; the loss is
    held to 6 * 4 * 2^-8."""
    say(f"training step {kind}")
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
    leaves = [t.double().requires_grad_() for t in (x, w_in, rate, w_norm, w_out)]
    xd, wi, ra, wn, wo = leaves
    xs, rs, ins = (xd @ wi.t()).chunk(3, -1)
    a = torch.exp(-ra * torch.sigmoid(rs))
    b = torch.sqrt(1 - a * a) * torch.sigmoid(ins) * xs
    h, hs = torch.zeros(B, D, device="cuda", dtype=torch.float64), []
    for t in range(L):
        h = a[:, t] * h + b[:, t]
        hs.append(h)
    res = torch.stack(hs, 1) + xd
    y = res / torch.sqrt((res * res).mean(-1, keepdim=True) + 1e-5) * wn
    if teacher is None:
        loss = torch.nn.functional.cross_entropy((y @ wo.t()).flatten(0, 1), target.flatten(), ignore_index=-1, reduction="none").view(B, L)
    else:
        logp = torch.log_softmax(y @ wo.t() / 2.0, -1).gather(-1, teacher[0])
        logq = torch.log_softmax(teacher[1].double() / 2.0, -1)
        loss = 4.0 * (logq.exp() * (logq - logp)).sum(-1)
    (loss.sum() / target.numel()).backward()
    worst = ((got["loss"].double() - loss).abs().max() / loss.abs().max()).item()
    assert worst <= 6 * 4 * 2.0 ** -8, worst
    for name, leaf in zip(("dx", "dw_in", "drate", "dnorm", "dweight"), leaves):
        e = ((got[name].double() - leaf.grad).abs().max() / leaf.grad.abs().max()).item()
        say(f"{name} {e:.2e}")
        assert e <= 12 * 4 * 2.0 ** -8, (name, e)


def test_example_training_step():
    """The example's block with a vocabulary behind it, against plain float32.  About eight roundings to bf16
    (2^-8) lie between the input and a loss and as many back to a gradient, each of values up to about four times
    those they are summed with: 8 * 4 * 2^-8 = 0.125 of the largest, and twice that."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import linattn_block
    finally:
        sys.path.pop(0)
    errors = linattn_block.check_training(linattn_block.LinAttnBlock(width=512, heads=6, groups=3, dim=64, group=64))
    say(str(errors))
    assert len(errors) == 10
    for name, e in errors.items():
        assert e <= (0.25 if name.startswith("d ") else 0.125), (name, e)


def test_tokens_continue_a_prompt():
    """A prompt, then single tokens from its last state, give what the whole sequence gives."""
    B, L, D = 3, 150, 200
    x, r, i = (randn(B, L, D, dtype=F32, seed=s) for s in range(3))
    rate = randn(D, dtype=F32, seed=3).abs()
    whole = ssm.ssm_gscan_fwd(x, r, i, rate)
    S = torch.empty(B, D, device="cuda")
    head = [t[:, :140].contiguous() for t in (x, r, i)]
    ssm.ssm_gscan_fwd(*head, rate, last_state=S)
    want = ref.Gscan(*[t.double().cpu().numpy() for t in (x, r, i)], rate.double().cpu().numpy())
    for t in range(140, L):
        out = ssm.ssm_gscan_update(S, *[v[:, t].contiguous() for v in (x, r, i)], rate)
        for got in (out, whole[:, t]):
            assert np.all(np.abs(got.double().cpu().numpy() - want.h[:, t]) <= 1.01 * want.h_off[:, t])


# ----------------------------------------------------------------- past 2^31 elements


def test_recurrence_past_32_bits():
    """Rows of packed tensors that span more than 2^32 bytes, and tensors of more than 2^31 elements."""
    say("recurrence past 32 bits")
    big = torch.empty(1, 300, 1 << 23, device="cuda", dtype=BF16)
    assert big.numel() > 1 << 31
    parts = [big[..., (j << 21) + 5:(j << 21) + 5 + 130] for j in range(3)]
    for j, p in enumerate(parts):
        p.copy_(randn(1, 300, 130, seed=j))
    flat = [p.contiguous() for p in parts]
    states = [torch.empty(1, 10, 130, device="cuda") for _ in range(2)]
    assert torch.equal(ssm.ssm_gscan_fwd(*parts, states=states[0]), ssm.ssm_gscan_fwd(*flat, states=states[1]))
    dout = randn(1, 300, 130, seed=7)
    for a, b in zip(ssm.ssm_gscan_bwd(*parts, None, dout, states[0]).values(), ssm.ssm_gscan_bwd(*flat, None, dout, states[1]).values()):
        assert torch.equal(a, b)
    del big, parts
    B, L, D = 2, 70000, 15400
    x, r = torch.empty(B, L, D, device="cuda", dtype=BF16), torch.empty(B, L, D, device="cuda", dtype=BF16)
    assert x.numel() > 1 << 31
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(0))
    r.normal_(1.0, generator=torch.Generator(device="cuda").manual_seed(1))
    out = ssm.ssm_gscan_fwd(x, r, lerp=True)
    at = slice(D - 66, D)
    want = ssm.ssm_gscan_fwd(x[1:, :, at].contiguous(), r[1:, :, at].contiguous(), lerp=True, out_dtype=F32)
    # chains cut into other groups: two roundings of fp32 apart for each of some ten compositions, and bf16's own
    assert ((out[1:, :, at].float() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19).all()


def test_head_past_32_bits():
    """Weights and their gradient of more than 2^32 bytes: the last rows' against the same rows alone."""
    say("head past 32 bits")
    V, D, T = 262144, 8200, 20
    w = torch.empty(V, D, device="cuda", dtype=BF16)
    assert w.numel() * 2 > 1 << 32
    w.normal_(std=0.01, generator=torch.Generator(device="cuda").manual_seed(0))
    x = randn(T, D)
    target = torch.full((T,), V - 1, device="cuda")
    loss, lse = ssm.ssm_xent_fwd(x, w, target)
    z = torch.cat([x.double() @ part.double().t() for part in w.chunk(16)], -1)
    want = torch.logsumexp(z, -1)
    off = 2 * (D + 4) * ref.U * (x.double().abs() @ w[-4096:].double().abs().t()).amax() * 2
    assert ((lse.double() - want).abs() <= off + 500 * ref.U * want.abs()).all()
    assert ((loss.double() - (want - z[:, -1])).abs() <= 2 * off + 500 * ref.U * want.abs()).all()
    d = randn(T, dtype=F32, seed=1)
    g = ssm.ssm_xent_bwd(d, x, w, target, lse)
    dz = torch.exp(z[:, -300:] - want[:, None])
    dz[:, -1] -= 1
    dz *= d.double()[:, None]
    v, size = dz.t() @ x.double(), dz.abs().t() @ x.double().abs()
    assert ((g["dweight"][-300:].double() - v).abs() <= (2.0 ** -8 + 2.0 ** -12) * size + 2.0 ** -8 * v.abs() + 1e-30).all()
    dx = -d.double()[:, None] * w[-1].double() + d.double()[:, None] * sum(
        torch.exp(z[:, j:j + 16384] - want[:, None]) @ w[j:j + 16384].double() for j in range(0, V, 16384))
    assert ((g["dx"].double() - dx).abs().max() <= 3 * 2.0 ** -8 * dx.abs().max())
