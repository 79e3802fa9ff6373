"""The block operators (include/ssmblock.h) as a program uses them: captured in HIP graphs,
on other streams, refused calls, tensors past 2^31 elements, the forms of the 4-bit
product that other tests' sizes do not reach, and the example that runs them together."""
import os
import sys

import numpy as np
import pytest

import block_ref as ref
from gpu_util import say
from test_graph_gpu import _capture, _poison, _replay_and_check
from test_linattn_gpu import CHUNKED, draw, near, pair

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
    x, z, r = randn(70, 640), randn(70, 640, seed=1), randn(70, 640, dtype=F32, seed=2)
    w, s = randn(640, dtype=F32, seed=3), randn(640, dtype=F32, seed=4)
    q, k = randn(2, 2100, 2, 64, seed=5), randn(2, 2100, 2, 64, seed=6)
    v, g = randn(2, 2100, 4, 64, seed=7), -randn(2, 2100, 4, dtype=F32, seed=8).abs() * 0.1
    S = randn(2, 4, 64, 64, dtype=F32, seed=9)
    codes, scales, zeros = ssm.ssm_q4_quantize(randn(520, 640, seed=10), 64)
    few = {"chunk_len": 512}
    return {
        "add_norm": lambda: ssm.ssm_add_norm_fwd(x, r, w, scale=s),
        "add_norm_bwd": lambda: ssm.ssm_add_norm_bwd(z, r, w, r, x, s).values(),
        "gated_norm": lambda: (ssm.ssm_gated_norm_fwd(x, z, w, ngroups=10),),
        "gated_norm_bwd": lambda: ssm.ssm_gated_norm_bwd(z, x, z, w, ngroups=10).values(),
        "linattn": lambda: (ssm.ssm_linattn_fwd(q, k, v, g, initial_state=S),),
        "linattn in time chunks": lambda: (ssm.ssm_linattn_fwd(q, k, v, g, initial_state=S, plan=few),),
        "linattn_bwd": lambda: ssm.ssm_linattn_bwd(q, k, v, g, v, initial_state=S, want_dinitial_state=True).values(),
        "linattn_bwd, fixed decay": lambda: ssm.ssm_linattn_bwd(q, k, v, g[0, 0], v).values(),
        "linattn step": lambda: (ssm.ssm_linattn_state_update(S, q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(),
                                                              g[:, 0].contiguous(), state_out=torch.empty_like(S)),),
        "q4, one row": lambda: (ssm.ssm_q4_matvec(x[:1], codes, scales, zeros),),
        "q4, rows laid out": lambda: (ssm.ssm_q4_matvec(x, codes, scales, zeros),),
        "q4_quantize": lambda: ssm.ssm_q4_quantize(x),
    }


NAMES = ("add_norm", "add_norm_bwd", "gated_norm", "gated_norm_bwd", "linattn", "linattn in time chunks", "linattn_bwd",
         "linattn_bwd, fixed decay", "linattn step", "q4, one row", "q4, rows laid out", "q4_quantize")


@pytest.mark.parametrize("name", NAMES)
def test_graph_replays(name):
    say(f"graph: {name}")
    call = operators()[name]
    want = [t.clone() for t in call()]
    got = []

    def run():
        got[:] = call()
    g = _capture(run)

    def reset():
        for t in got:
            t.fill_(0 if t.dtype == torch.uint8 else float("nan"))
        call()          # eager work between the replays
    for r in range(4):
        reset()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), f"replay {r}: output {i} differs from the eager result"


def test_state_updates_in_place_in_a_graph():
    S = randn(2, 4, 64, 32, dtype=F32)
    start = S.clone()
    q, k, v, g = randn(2, 4, 32), randn(2, 4, 32, seed=1), randn(2, 4, 64, seed=2), -randn(2, 4, dtype=F32, seed=3).abs()
    out = ssm.ssm_linattn_state_update(S, q, k, v, g)
    want = out.clone(), S.clone()
    graph = _capture(lambda: ssm.ssm_linattn_state_update(S, q, k, v, g, out=out))

    def reset():
        S.copy_(start)
        _poison(out)
    _replay_and_check(graph, reset, (out, S), want)


@pytest.mark.parametrize("name", NAMES)
def test_another_stream(name):
    """A call on a side stream, behind that stream's own work, gives what it gives on the
    current one."""
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


def test_workspace_from_either_side():
    """A shape's first call takes its workspace from the library, later ones from PyTorch."""
    from sequence_scan_amd import block
    for name, call in operators().items():
        block._wanted.clear()
        first = [t.clone() for t in call()]
        wants = any(block._wanted.values())
        assert wants == (name in ("add_norm_bwd", "gated_norm_bwd", "linattn", "linattn in time chunks", "linattn_bwd",
                                  "linattn_bwd, fixed decay", "q4, rows laid out")), name
        for _ in range(2):
            torch.empty(1 << 20, device="cuda").fill_(float("nan"))
            for a, b in zip(call(), first):
                assert torch.equal(a, b), name


def test_given_stream():
    x, w = randn(64, 256), randn(256, dtype=F32, seed=1)
    want, _ = ssm.ssm_add_norm_fwd(x, None, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.empty_like(want)
    ssm.ssm_add_norm_fwd(x, None, w, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_refused_calls_write_nothing():
    x, z = randn(8, 64), randn(8, 64, seed=1)
    q, v, g = randn(1, 40, 2, 64), randn(1, 40, 2, 64, seed=1), -randn(1, 40, 2, dtype=F32, seed=2).abs()
    S = torch.full((1, 2, 64, 64), 7.0, device="cuda")
    codes, scales, _ = ssm.ssm_q4_quantize(randn(24, 64), 32)
    out, res = torch.full_like(x, 7), torch.full_like(x, 7)
    la, step, y = torch.full_like(v, 7), torch.full_like(v[:, 0], 7), torch.full((8, 24), 7.0, device="cuda", dtype=BF16)
    cases = {
        "width": (ValueError, lambda: ssm.ssm_add_norm_fwd(x, z, randn(60, dtype=F32), out=out, residual_out=res)),
        "eps": (ssm.SSMError, lambda: ssm.ssm_add_norm_fwd(x, z, eps=-1.0, out=out, residual_out=res)),
        "out on x": (ssm.SSMError, lambda: ssm.ssm_add_norm_fwd(out, z, out=out, residual_out=res)),
        "groups": (ssm.SSMError, lambda: ssm.ssm_gated_norm_fwd(x, z, ngroups=5, out=out)),
        "gate type": (TypeError, lambda: ssm.ssm_gated_norm_fwd(x, z.float(), out=out)),
        "fp32 prompt": (ssm.SSMError, lambda: ssm.ssm_linattn_fwd(q.float(), q.float(), v.float(), g, out=la, last_state=S)),
        "plan": (ssm.SSMError, lambda: ssm.ssm_linattn_fwd(q, q, v, g, out=la, last_state=S, plan={"chunk_len": 33})),
        "scale": (ssm.SSMError, lambda: ssm.ssm_linattn_fwd(q, q, v, g, float("nan"), out=la, last_state=S)),
        "decay shape": (ValueError, lambda: ssm.ssm_linattn_fwd(q, q, v, g[:, :39], out=la, last_state=S)),
        "state shape": (ValueError, lambda: ssm.ssm_linattn_state_update(S[..., :32].contiguous(), q[:, 0].contiguous(),
                                                                         q[:, 0].contiguous(), v[:, 0].contiguous(), g[:, 0].contiguous(), out=step)),
        "strided step": (ValueError, lambda: ssm.ssm_linattn_state_update(S, q.transpose(2, 3)[:, 0], q[:, 0].contiguous(),
                                                                          v[:, 0].contiguous(), g[:, 0].contiguous(), out=step)),
        "columns": (ValueError, lambda: ssm.ssm_q4_matvec(x[:, :32], codes, scales, out=y)),
        "row stride": (ssm.SSMError, lambda: ssm.ssm_q4_matvec(randn(8, 67)[:, :64], codes, scales, out=y)),
        "bias type": (TypeError, lambda: ssm.ssm_q4_matvec(x, codes, scales, bias=randn(24), out=y)),
    }
    for name, (error, call) in cases.items():
        say(f"refusal: {name}")
        with pytest.raises(error):
            call()
        torch.cuda.synchronize()
        for t in (out, res, la, S, step, y):
            assert torch.all(t == 7), f"{name}: a refused call wrote an output"


# ------------------------------------------------------------- past 2^31 elements


def test_rows_far_apart():
    """Rows of packed tensors that span more than 2^32 bytes give the packed rows' bits."""
    rows, width = 300, 1 << 23
    big = torch.empty(1, rows, width, device="cuda", dtype=BF16)
    assert big.numel() > 1 << 31
    parts = [big[..., i * 1024:i * 1024 + 128] for i in range(4)]
    for i, p in enumerate(parts):
        p.copy_(randn(1, rows, 128, seed=i))
    flat = [p.contiguous() for p in parts]

    def heads(ts):
        return [t.unflatten(-1, (2, 64)) for t in ts[:3]]
    g = -randn(1, rows, 2, dtype=F32, seed=9).abs() * 0.1
    assert torch.equal(ssm.ssm_linattn_fwd(*heads(parts), g), ssm.ssm_linattn_fwd(*heads(flat), g))
    dout = randn(1, rows, 2, 64, seed=11)
    for a, b in zip(ssm.ssm_linattn_bwd(*heads(parts), g, dout).values(), ssm.ssm_linattn_bwd(*heads(flat), g, dout).values()):
        assert torch.equal(a, b)
    for a, b in zip(ssm.ssm_add_norm_fwd(parts[0], flat[1]), ssm.ssm_add_norm_fwd(flat[0], flat[1])):
        assert torch.equal(a, b)
    assert torch.equal(ssm.ssm_gated_norm_fwd(parts[0], parts[1], ngroups=2), ssm.ssm_gated_norm_fwd(flat[0], flat[1], ngroups=2))
    gates = [ssm.ssm_gated_norm_bwd(flat[2], a, b, ngroups=2) for a, b in (parts[:2], flat[:2])]
    for a, b in zip(gates[0].values(), gates[1].values()):
        assert torch.equal(a, b)
    codes, scales, zeros = ssm.ssm_q4_quantize(randn(100, 128, seed=5), 32)
    for m in (1, rows):
        a = ssm.ssm_q4_matvec(parts[0][0, rows - m:], codes, scales, zeros)
        assert torch.equal(a, ssm.ssm_q4_matvec(flat[0][0, rows - m:], codes, scales, zeros))


def test_states_and_codes_past_32_bits():
    B, H, d = 4128, 32, 128
    S = torch.empty(B, H, d, d, device="cuda")
    assert S.numel() > 1 << 31
    S[-2:].copy_(randn(2, H, d, d, dtype=F32))
    q, k, v = randn(B, H, d), randn(B, H, d, seed=1), randn(B, H, d, seed=2)
    g = -randn(B, H, dtype=F32, seed=3).abs()
    tail = S[-2:].clone()
    want = ssm.ssm_linattn_state_update(tail, q[-2:].contiguous(), k[-2:].contiguous(), v[-2:].contiguous(), g[-2:].contiguous())
    out = ssm.ssm_linattn_state_update(S, q, k, v, g)
    assert torch.equal(out[-2:], want) and torch.equal(S[-2:], tail)
    del S
    n, kk = 140000, 65536
    codes = torch.randint(0, 256, (n, kk // 2), device="cuda", dtype=torch.uint8)
    assert codes.numel() > 1 << 32
    scales = torch.full((n, kk // 128), 2.0 ** -8, device="cuda")
    for m in (1, 20):
        x = randn(m, kk, seed=m)
        y = ssm.ssm_q4_matvec(x, codes, scales, out_dtype=F32)
        xd = x.double().cpu().numpy()
        w = ref.q4_weights(codes[-40:].cpu().numpy(), scales[-40:].double().cpu().numpy(), None, 128)
        # sums of 65536 products of up to 23 |x| scale, 512 groups' sums and 8 parts' joins
        size = np.abs(xd).sum(-1, keepdims=True) * 24 * 2.0 ** -8
        assert np.all(np.abs(y[:, -40:].double().cpu().numpy() - xd @ w.T) <= (128 + 512 + 8) * 2.0 ** -24 * size)


# ------------------------------------------------------- forms of the 4-bit product


@pytest.mark.parametrize("m,n,k,group", [(16, 40, 8192, 64), (13, 50, 16384, 128), (9, 33, 20000, 32), (1, 40000, 160, 32),
                                         (3, 33000, 384, 128), (2, 70000, 96, 32), (16, 35, 3968, 128), (5, 20, 12800, 64)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_few_rows_in_slabs(m, n, k, group, dt):
    """Up to 16 rows whose x does not fit the LDS at once, and many columns.  The bar: an
    output sums k products of at most 31 |x| scale in fp32, in parts (16 products a matrix
    instruction, k / group groups, 8 wavefronts), held to (group + k / group + 8) * 2^-24
    of the sum of their magnitudes, bf16 outputs to 2^-8 of themselves more."""
    if dt == F32:
        m = min(m, 5)
    say(f"q4 slabs: {m} x {n} x {k}, group {group}, {dt}")
    r = np.random.default_rng(k)
    codes = torch.from_numpy(r.integers(0, 256, (n, k // 2), dtype=np.uint8)).cuda()
    scales, se = pair(r.uniform(0.01, 0.02, (n, k // group)), F32)
    zeros = torch.from_numpy(r.integers(0, 16, (n, k // group), dtype=np.uint8)).cuda()
    x, xe = pair(r.standard_normal((m, k)), dt)
    w = ref.q4_weights(codes.cpu().numpy(), se, zeros.cpu().numpy(), group)
    y = ssm.ssm_q4_matvec(x, codes, scales, zeros).double().cpu().numpy()
    want = xe @ w.T
    size = np.abs(xe).sum(-1, keepdims=True) * 31 * 0.02
    bar = (group + k // group + 8) * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(want) if dt == BF16 else 0)
    assert np.all(np.abs(y - want) <= bar)


# -------------------------------------------------------------- gradients and NaN


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_backward_keeps_bad_values_in_their_head(bad):
    """A bad value of dout: its own dq row and, back in time, dk and dv of its head are not
    finite; later steps, other rows of dq, other heads and batch rows keep their bits."""
    d = draw(2, 150, 4, 4, 64, 64, seed=5)
    q, k, v, g, dout = (d[n][0] for n in ("q", "k", "v", "g", "dout"))
    clean = ssm.ssm_linattn_bwd(q, k, v, g, dout)
    t, h = 70, 2
    dout[1, t, h, 9] = bad
    got = ssm.ssm_linattn_bwd(q, k, v, g, dout)
    assert not torch.isfinite(got["dq"][1, t, h]).any()
    assert not torch.isfinite(got["dv"][1, :t + 1, h, 9]).any()
    assert not torch.isfinite(got["dk"][1, :t + 1, h]).any()
    assert not torch.isfinite(got["dlog_decay"][1, 1:t + 1, h]).any()
    for name in ("dq", "dk", "dv", "dlog_decay"):
        a, b = got[name], clean[name]
        assert torch.equal(a[0], b[0]), name
        for j in (0, 1, 3):
            assert torch.equal(a[1, :, j], b[1, :, j]), name
    for name in ("dk", "dv"):
        assert torch.equal(got[name][1, t + 1:, h], clean[name][1, t + 1:, h]), name
    for s in (slice(0, t), slice(t + 1, None)):
        assert torch.equal(got["dq"][1, s, h], clean["dq"][1, s, h])


@pytest.mark.parametrize("L", [1, 2, 31, 33])
def test_short_sequences_with_states(L):
    d = draw(3, L, 6, 2, 40, 24, seed=L)
    args = [d[n] for n in ("q", "k", "v", "g")]
    got = ssm.ssm_linattn_bwd(*[a[0] for a in args], d["dout"][0], 0.5, d["S0"][0], d["dlast"][0], True, F32)
    want = ref.linattn_grad(*[a[1] for a in args], 0.5, d["dout"][1], d["S0"][1], d["dlast"][1])
    size = ref.linattn_grad(*[np.abs(a[1]) if i < 3 else a[1] for i, a in enumerate(args)], 0.5, np.abs(d["dout"][1]),
                            np.abs(d["S0"][1]), np.abs(d["dlast"][1]))
    for name in ("dq", "dk", "dv", "dinitial_state"):
        near(got[name], want[name], size[name], CHUNKED, name)
    top = np.broadcast_to(size["dlog_decay"].max(1, keepdims=True), want["dlog_decay"].shape)
    near(got["dlog_decay"], want["dlog_decay"], top, CHUNKED + 2 * 2.0 ** -18, "dlog_decay")


# -------------------------------------------------------------------- the example


def test_example_block():
    """The example's prompt, tokens and gradients against plain float32.  Six roundings to
    bf16 lie between the input and an output (the norm, the projection, linear attention,
    its norm, the product, the output), 2^-9 each, of values up to about four times those
    they are summed with: 6 * 4 * 2^-9 = 4.7e-2 of the largest; the gradients pass about as
    many again."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import linattn_block
    finally:
        sys.path.pop(0)
    errors = linattn_block.check(linattn_block.LinAttnBlock(width=512, heads=6, groups=3, dim=64, group=64))
    say(str(errors))
    assert errors["residual"] == 0.0
    for name, e in errors.items():
        assert e <= (9.4e-2 if name.startswith("d ") else 4.7e-2), (name, e)


@pytest.mark.parametrize("plan", [None, {"chunk_len": 64}])
@pytest.mark.parametrize("which", ["decay", "q", "k"])
def test_values_that_are_not_finite_reach_their_head_only(which, plan):
    """A NaN of a decay or of k at step t of one head: its outputs are NaN from there on
    (of q: that step's alone); earlier steps and other heads and batch rows keep their bits."""
    d = draw(2, 200, 3, 3, 64, 72, seed=9)
    q, k, v, g = (d[n][0] for n in ("q", "k", "v", "g"))
    clean = ssm.ssm_linattn_fwd(q, k, v, g, plan=plan)
    b, t, h = 1, 77, 1
    if which == "decay":
        g[b, t, h] = float("nan")
    else:
        (q if which == "q" else k)[b, t, h, 5] = float("nan")
    got = ssm.ssm_linattn_fwd(q, k, v, g, plan=plan)
    hit = torch.zeros(got.shape[:3], dtype=torch.bool, device="cuda")
    hit[b, t:t + 1 if which == "q" else None, h] = True
    assert torch.isnan(got[hit]).all()
    assert torch.equal(got[~hit], clean[~hit])
