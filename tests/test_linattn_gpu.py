"""GPU parity of linear attention with a decay for each head (ssm_linattn_*)
against the 64-bit references, through the C ABI.

Bars, from the arithmetic.  Inputs are the same bits on both sides.  In the
chunked form a computed operand enters the matrix cores as two bf16 terms, within
2^-18 of itself; sums of up to 64 + 128 fp32 terms round within 192 * 2^-24; a
decay is the exponential of a difference of sums below 256 in magnitude, whose
rounding moves it by 2 * 256 * 2^-24.  Each of these is relative to the sum of the
magnitudes of an output's terms, which is the same operator on absolute values:
3.8e-6 + 1.2e-5 + 3.1e-5, held to 6e-5 of it (and 2^-8 of a bf16 value).  The
decay's gradient carries <S, dS> across the matrix chunks of a time chunk, at most
32, two sums of split products each: 2 * n * 2^-18 of its largest more.  The
single-token step is fp32 throughout: 256 * 2^-24 and the exponential, held to 2e-5.
"""
import numpy as np
import pytest

import block_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32, BF16 = torch.float32, torch.bfloat16
CHUNKED, STEP, ROUND = 6e-5, 2e-5, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


def pair(a, dtype=BF16):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dtype)
    return t.cuda(), t.double().numpy()


def draw(B, L, H, G, dk, dv, seed, fixed=False, rate=16.0, packed=False):
    r = np.random.default_rng(seed)
    d = {}
    if packed:   # one projection's output: q | k | v side by side, and some more
        n = [G * dk, G * dk, H * dv, 24]
        t, e = pair(r.standard_normal((B, L, sum(n))))
        cut = np.cumsum([0] + n)
        for i, (name, h, w) in enumerate((("q", G, dk), ("k", G, dk), ("v", H, dv))):
            sl = slice(cut[i], cut[i + 1])
            d[name] = t[..., sl].unflatten(-1, (h, w)), e[..., sl].reshape(B, L, h, w)
    else:
        for name, h, w in (("q", G, dk), ("k", G, dk), ("v", H, dv)):
            d[name] = pair(r.standard_normal((B, L, h, w)))
    rates = np.exp(r.uniform(0, np.log(rate), H))
    step = np.exp(r.uniform(np.log(1e-3), np.log(0.1), (B, L, H)))
    d["g"] = pair(-rates * 0.02 if fixed else -rates * step, F32)
    for name in ("S0", "dlast"):
        d[name] = pair(r.standard_normal((B, H, dv, dk)), F32)
    d["dout"] = pair(r.standard_normal((B, L, H, dv)))
    return d


def near(got, want, size, bar, name):
    y = got.double().cpu().numpy()
    assert y.shape == want.shape, name
    lim = bar * size + (ROUND * np.abs(want) if got.dtype == BF16 else 0.0)
    off = np.abs(y - want)
    assert not np.isnan(y).any() and (off <= lim).all(), f"{name}: {np.max(off - lim):.3e} past the bar, off {off.max():.3e}"


def check_forward(d, out, last, scale, S0=None):
    q, k, v, g = (d[n][1] for n in ("q", "k", "v", "g"))
    want, S = ref.linattn(q, k, v, g, scale, S0)
    size, Ssize = ref.linattn(abs(q), abs(k), abs(v), g, scale, None if S0 is None else abs(S0))
    near(out, want, size, CHUNKED, "out")
    near(last, S, Ssize, CHUNKED, "last_state")


SHAPES = [(1, 1, 1, 1, 8, 8), (2, 2, 2, 1, 64, 64), (1, 63, 3, 3, 16, 40), (2, 64, 2, 2, 128, 128), (1, 65, 4, 2, 96, 72),
          (1, 127, 2, 1, 64, 128), (3, 200, 2, 2, 128, 64), (1, 1000, 2, 1, 128, 8), (2, 130, 5, 1, 32, 128)]


@pytest.mark.parametrize("B,L,H,G,dk,dv", SHAPES)
@pytest.mark.parametrize("fixed", [False, True])
def test_forward(B, L, H, G, dk, dv, fixed):
    say(f"linattn forward {B} x {L}, heads {H}/{G}, dk {dk} dv {dv}, fixed {fixed}")
    d = draw(B, L, H, G, dk, dv, L + dk, fixed, packed=L % 2 == 0)
    last = torch.full((B, H, dv, dk), float("nan"), device="cuda")
    out = ssm.ssm_linattn_fwd(d["q"][0], d["k"][0], d["v"][0], d["g"][0], last_state=last, out_dtype=F32)
    check_forward(d, out, last, dk ** -0.5)
    o16 = ssm.ssm_linattn_fwd(d["q"][0], d["k"][0], d["v"][0], d["g"][0])
    assert torch.equal(o16, out.bfloat16())


@pytest.mark.parametrize("chunk_len,in_place", [(None, False), (None, True), (64, False), (64, True), (192, False), (4096, True)])
def test_forward_from_a_state_and_plans(chunk_len, in_place):
    say(f"linattn from a state, time chunks of {chunk_len}, in place {in_place}")
    d = draw(2, 333, 4, 2, 80, 136 - 8, 7)
    S0 = d["S0"][0].clone()
    last = S0 if in_place else torch.empty_like(S0)
    out = ssm.ssm_linattn_fwd(d["q"][0], d["k"][0], d["v"][0], d["g"][0], scale=0.3, initial_state=S0, last_state=last,
                              out_dtype=F32, plan={"chunk_len": chunk_len} if chunk_len else None)
    check_forward(d, out, last, 0.3, d["S0"][1])


def test_forward_planned_chunks():
    say("linattn: one long head, the planner's time chunks")
    plan = ssm.ssm_linattn_plan_query(1, 3000, 1, 64, 64)
    assert plan["n_chunks"] > 1
    d = draw(1, 3000, 1, 1, 64, 64, 11)
    last = torch.empty(1, 1, 64, 64, device="cuda")
    out = ssm.ssm_linattn_fwd(d["q"][0], d["k"][0], d["v"][0], d["g"][0], last_state=last, out_dtype=F32)
    check_forward(d, out, last, 64 ** -0.5)


@pytest.mark.parametrize("B,L,H,G,dk,dv", SHAPES + [(1, 2100, 2, 1, 64, 96), (1, 700, 1, 1, 128, 128)])
@pytest.mark.parametrize("fixed,states", [(False, True), (True, True), (False, False)])
def test_backward(B, L, H, G, dk, dv, fixed, states):
    say(f"linattn backward {B} x {L}, heads {H}/{G}, dk {dk} dv {dv}, fixed {fixed}, states {states}")
    d = draw(B, L, H, G, dk, dv, 3 * L + dv, fixed, packed=L % 2 == 1)
    t, e = {n: x[0] for n, x in d.items()}, {n: x[1] for n, x in d.items()}
    S0, dl = (t["S0"], t["dlast"]) if states else (None, None)
    g = ssm.ssm_linattn_bwd(t["q"], t["k"], t["v"], t["g"], t["dout"], initial_state=S0, dlast_state=dl,
                            want_dinitial_state=True, grad_dtype=F32)
    S0e, dle = (e["S0"], e["dlast"]) if states else (None, None)
    scale = dk ** -0.5
    want = ref.linattn_grad(e["q"], e["k"], e["v"], e["g"], scale, e["dout"], S0e, dle)
    size = ref.linattn_grad(abs(e["q"]), abs(e["k"]), abs(e["v"]), e["g"], scale, abs(e["dout"]),
                            None if S0e is None else abs(S0e), None if dle is None else abs(dle))
    for n in ("dq", "dk", "dv", "dinitial_state"):
        near(g[n], want[n], size[n], CHUNKED, n)
    top = size["dlog_decay"] if fixed else np.broadcast_to(size["dlog_decay"].max(1, keepdims=True), want["dlog_decay"].shape)
    n_chunks = min(32, -(-L // 64))
    near(g["dlog_decay"], want["dlog_decay"], top, CHUNKED + 2 * n_chunks * 2.0 ** -18, "dlog_decay")
    if not fixed and states:
        b = ssm.ssm_linattn_bwd(t["q"], t["k"], t["v"], t["g"], t["dout"], initial_state=S0, dlast_state=dl)
        assert "dinitial_state" not in b and b["dq"].dtype == BF16
        for n in ("dq", "dk", "dv"):
            assert torch.equal(b[n], g[n].bfloat16()), n
        assert torch.equal(b["dlog_decay"], g["dlog_decay"])


def test_resets():
    """A decay of minus infinity cuts the sequence: what follows equals a fresh start, and no gradient crosses."""
    say("linattn: decays of minus infinity")
    d = draw(1, 150, 2, 1, 64, 64, 21)
    cuts = [40, 41, 128]
    for n in (0, 1):
        d["g"][n][:, cuts] = -float("inf")
    t, e = {n: x[0] for n, x in d.items()}, {n: x[1] for n, x in d.items()}
    last = torch.empty(1, 2, 64, 64, device="cuda")
    out = ssm.ssm_linattn_fwd(t["q"], t["k"], t["v"], t["g"], initial_state=t["S0"], last_state=last, out_dtype=F32)
    check_forward(d, out, last, 0.125, e["S0"])
    g = ssm.ssm_linattn_bwd(t["q"], t["k"], t["v"], t["g"], t["dout"], initial_state=t["S0"], want_dinitial_state=True,
                            grad_dtype=F32)
    want = ref.linattn_grad(e["q"], e["k"], e["v"], e["g"], 0.125, e["dout"], e["S0"])
    size = ref.linattn_grad(abs(e["q"]), abs(e["k"]), abs(e["v"]), e["g"], 0.125, abs(e["dout"]), abs(e["S0"]))
    for n in ("dq", "dk", "dv", "dinitial_state"):
        near(g[n], want[n], size[n], CHUNKED, n)
    near(g["dlog_decay"], want["dlog_decay"], size["dlog_decay"].max(), CHUNKED + 6 * 2.0 ** -18, "dlog_decay")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_stay_behind(bad):
    say(f"linattn: {bad} in v, k and q reaches later steps only")
    for name, col in (("v", 5), ("k", None), ("q", None)):
        d = draw(1, 200, 2, 2, 64, 64, 31)
        t = {n: x[0].clone() for n, x in d.items()}
        clean = ssm.ssm_linattn_fwd(t["q"], t["k"], t["v"], t["g"])
        t[name][0, 100, 1, 5] = bad
        out = ssm.ssm_linattn_fwd(t["q"], t["k"], t["v"], t["g"])
        assert torch.equal(out[0, :, 0], clean[0, :, 0]) and torch.equal(out[0, :100, 1], clean[0, :100, 1])
        if name == "q":
            assert torch.equal(out[0, 101:, 1], clean[0, 101:, 1]) and not torch.isfinite(out[0, 100, 1]).any()
        elif name == "k":
            assert not torch.isfinite(out[0, 100:, 1]).any()
        else:
            keep = [i for i in range(64) if i != col]
            assert torch.equal(out[0, :, 1][:, keep], clean[0, :, 1][:, keep])
            assert not torch.isfinite(out[0, 100:, 1, col]).any()


@pytest.mark.parametrize("B,H,G,dk,dv", [(1, 1, 1, 4, 1), (2, 4, 2, 64, 64), (3, 6, 1, 128, 37), (1, 5, 5, 20, 130), (2, 2, 1, 256, 16),
                                         (70, 3, 3, 96, 48)])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("fixed", [False, True])
def test_step(B, H, G, dk, dv, dt, fixed):
    say(f"linattn step batch {B}, heads {H}/{G}, dk {dk} dv {dv}, {dt}, fixed {fixed}")
    r = np.random.default_rng(dk + dv)
    (q, qe), (k, ke) = pair(r.standard_normal((B, G, dk)), dt), pair(r.standard_normal((B, G, dk)), dt)
    v, ve = pair(r.standard_normal((B, H, dv)), dt)
    g, ge = pair(-r.uniform(0, 2, (H,) if fixed else (B, H)), F32)
    S, Se = pair(r.standard_normal((B, H, dv, dk)), F32)
    kept = S.clone()
    new = torch.empty_like(S)
    out = ssm.ssm_linattn_state_update(S, q, k, v, g, scale=0.5, state_out=new, out_dtype=F32)
    assert torch.equal(S, kept)
    args = [a[:, None] for a in (qe, ke, ve)] + [ge if fixed else ge[:, None]]
    want, Sw = ref.linattn(*args, 0.5, Se)
    size, Ss = ref.linattn(*[abs(a) for a in args[:3]], args[3], 0.5, abs(Se))
    near(out, want[:, 0], size[:, 0], STEP, "out")
    near(new, Sw, Ss, STEP, "state")
    again = ssm.ssm_linattn_state_update(S, q, k, v, g, scale=0.5)   # in place
    assert torch.equal(S, new) and torch.equal(again, out.to(dt))


def test_steps_follow_a_prompt():
    say("linattn: a prompt's last state, then single tokens, against the whole at once")
    d = draw(2, 90, 4, 2, 64, 64, 41)
    t = {n: x[0] for n, x in d.items()}
    S = torch.empty(2, 4, 64, 64, device="cuda")
    cut = lambda a, s: a[:, s].contiguous()  # noqa: E731
    first = slice(0, 77)
    outs = [ssm.ssm_linattn_fwd(*(cut(t[n], first) for n in ("q", "k", "v", "g")), last_state=S, out_dtype=F32)]
    for i in range(77, 90):
        outs.append(ssm.ssm_linattn_state_update(S, *(cut(t[n], i) for n in ("q", "k", "v", "g")), out_dtype=F32)[:, None])
    check_forward(d, torch.cat(outs, 1), S, 0.125)


def test_empty_and_repeat():
    say("linattn: no steps, no rows, the same bits twice and on another stream")
    S0 = torch.randn(2, 4, 64, 64, device="cuda")
    z = lambda *s: torch.empty(s, device="cuda", dtype=BF16)  # noqa: E731
    last = torch.empty_like(S0)
    g0 = torch.empty(2, 0, 4, device="cuda")
    assert ssm.ssm_linattn_fwd(z(2, 0, 2, 64), z(2, 0, 2, 64), z(2, 0, 4, 64), g0, initial_state=S0, last_state=last).numel() == 0
    assert torch.equal(last, S0)
    ssm.ssm_linattn_fwd(z(2, 0, 2, 64), z(2, 0, 2, 64), z(2, 0, 4, 64), g0, last_state=last)
    assert not last.any()
    b = ssm.ssm_linattn_bwd(z(2, 0, 2, 64), z(2, 0, 2, 64), z(2, 0, 4, 64), torch.zeros(4, device="cuda"), z(2, 0, 4, 64),
                            dlast_state=S0, want_dinitial_state=True)
    assert torch.equal(b["dinitial_state"], S0) and not b["dlog_decay"].any()
    assert ssm.ssm_linattn_fwd(z(0, 5, 2, 64), z(0, 5, 2, 64), z(0, 5, 4, 64), torch.empty(0, 5, 4, device="cuda")).shape[0] == 0
    d = draw(2, 700, 4, 2, 128, 128, 51)
    t = {n: x[0] for n, x in d.items()}
    run = lambda **kw: ssm.ssm_linattn_bwd(t["q"], t["k"], t["v"], t["g"], t["dout"], dlast_state=t["dlast"],  # noqa: E731
                                           want_dinitial_state=True, **kw)
    a = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = run(stream=s)
    s.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]), n
