"""GPU parity of the gated linear recurrence (ssm_gscan_*) against the 64-bit reference, to
the bars that model_ref.py derives."""
import numpy as np
import pytest

import model_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32, BF16 = torch.float32, torch.bfloat16
SEG = 32
HALF = {F32: 0.0, BF16: 2.0 ** -8}      # an output's own rounding (fp32: among the counts)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


def pair(a, dtype):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to("cuda", dtype)
    return t, t.double().cpu().numpy()


def draw(B, L, D, dtype, gate, rate, seed=0, out_dtype=None):
    """name -> (tensor, its values in 64 bits), absent ones (None, None)."""
    r = np.random.default_rng([seed, B, L, D])
    n = r.standard_normal
    out = {"x": pair(n((B, L, D)), dtype), "r": pair(n((B, L, D)) * 1.5 + (0 if rate else 1), dtype),
           "i": pair(n((B, L, D)), dtype) if gate else (None, None),
           "rate": pair(np.exp(r.uniform(np.log(1e-3), np.log(8.0), D)), F32) if rate else (None, None),
           "S0": pair(n((B, D)), F32), "dout": pair(n((B, L, D)), out_dtype or dtype), "dlast": pair(n((B, D)), F32)}
    return out


def near(got, want, off, half, what):
    got = got.double().cpu().numpy()
    bad = np.abs(got - want) - (off * 1.01 + half * np.abs(want) * 1.01 + 1e-37)
    assert not np.isnan(got).any(), what
    assert bad.max(initial=-1) <= 0, (what, float(bad.max()), np.unravel_index(bad.argmax(), bad.shape))


def states_for(B, L, D):
    return torch.full((B, -(-L // SEG), D), float("nan"), device="cuda")


def check(B, L, D, dtype, gate, rate, lerp, state, out_dtype=None, seed=0, tensors=None):
    out_dtype = out_dtype or dtype
    d = draw(B, L, D, dtype, gate, rate, seed, out_dtype)
    t = {n: v[0] for n, v in d.items()}
    if tensors:
        t.update(tensors(t))
    S0 = d["S0"] if state else (None, None)
    want = ref.Gscan(d["x"][1], d["r"][1], d["i"][1], d["rate"][1], lerp, S0[1])
    last, states = torch.full((B, D), float("nan"), device="cuda"), states_for(B, L, D)
    out = ssm.ssm_gscan_fwd(t["x"], t["r"], t["i"], t["rate"], lerp, S0[0], last_state=last, states=states, out_dtype=out_dtype)
    assert out.dtype == out_dtype
    near(out, want.h, want.h_off, HALF[out_dtype], "out")
    near(last, want.last, want.last_off, 0, "last_state")
    near(states, want.before[:, ::SEG], want.before_off[:, ::SEG], 0, "states")
    dlast = d["dlast"] if state else (None, None)
    g = ssm.ssm_gscan_bwd(t["x"], t["r"], t["i"], t["rate"], t["dout"], states, lerp, dlast[0], want_dinitial_state=state)
    wg = want.grad(d["dout"][1], dlast[1])
    assert set(g) == {"dx", "dr"} | ({"di"} if gate else set()) | ({"drate"} if rate else set()) | ({"dinitial_state"} if state else set())
    for n, v in g.items():
        near(v, *wg[n], HALF[dtype] if n in ("dx", "dr", "di") else 0, n)


CHOICES = [(g, r, l) for g in (True, False) for r in (True, False) for l in (True, False)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate,rate,lerp", CHOICES)
def test_each_form(gate, rate, lerp, dtype):
    say(f"gscan forms: {gate} {rate} {lerp} {dtype}")
    check(2, 150, 130, dtype, gate, rate, lerp, True)


@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 256, 257, 1000, 2500])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_lengths(L, dtype):
    say(f"gscan length {L} {dtype}")
    check(2, L, 96, dtype, True, True, False, L % 2 == 0)


@pytest.mark.parametrize("D", [1, 2, 3, 7, 63, 64, 65, 127, 128, 129, 255, 1023])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_widths(D, dtype):
    say(f"gscan width {D} {dtype}")
    check(3, 300, D, dtype, D % 3 != 0, D % 2 == 1, True, True)


@pytest.mark.parametrize("dtype,out_dtype", [(F32, BF16), (BF16, F32)])
def test_mixed_types(dtype, out_dtype):
    say(f"gscan {dtype} to {out_dtype}")
    check(2, 200, 70, dtype, True, True, False, True, out_dtype)


@pytest.mark.parametrize("shape", [(40, 37, 50), (1, 20000, 8), (300, 3, 5), (5, 700, 258)])
def test_batches(shape):
    say(f"gscan shape {shape}")
    check(*shape, BF16, True, False, False, True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 65, 96])
def test_slices_of_a_packed_projection(dtype, D):
    """x, r and i as slices of one tensor whose rows are odd or even elements apart."""
    say(f"gscan packed {dtype} {D}")

    def packed(t):
        B, L, _ = t["x"].shape
        out = {}
        big = torch.full((B, L, 3 * D + 5), float("nan"), device="cuda", dtype=dtype)
        for j, n in enumerate(("x", "i", "r")):
            part = big[..., 1 + j * D:1 + (j + 1) * D]
            part.copy_(t[n])
            out[n] = part
        return out
    check(2, 140, D, dtype, True, True, True, True, tensors=packed)


def test_states_in_place_and_across_calls():
    """A sequence in two calls joined by the state, the second in place, gives the whole one's bits."""
    say("gscan continued")
    d = draw(2, 384, 66, BF16, True, True)
    t = {n: v[0] for n, v in d.items()}
    last = torch.empty(2, 66, device="cuda")
    whole = ssm.ssm_gscan_fwd(t["x"], t["r"], t["i"], t["rate"], initial_state=t["S0"], last_state=last, out_dtype=F32)
    want = ref.Gscan(d["x"][1], d["r"][1], d["i"][1], d["rate"][1], False, d["S0"][1])
    S = t["S0"].clone()
    parts = []
    for at in (slice(0, 300), slice(300, 384)):
        cut = [t[n][:, at].contiguous() for n in ("x", "r", "i")]
        parts.append(ssm.ssm_gscan_fwd(*cut, t["rate"], initial_state=S, last_state=S, out_dtype=F32))
    both = torch.cat(parts, 1)
    near(whole, want.h, want.h_off, 0, "whole")
    near(both, want.h, 2 * want.h_off, 0, "parts")
    near(S, want.last, 2 * want.last_off, 0, "state")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate,rate,lerp", CHOICES)
def test_step(gate, rate, lerp, dtype):
    say(f"gscan step {gate} {rate} {lerp} {dtype}")
    for B, D in ((1, 1), (3, 130), (1, 2560), (70, 257)):
        d = draw(B, 1, D, dtype, gate, rate)
        t = {n: v[0] if v[0] is None or n in ("rate", "S0") else v[0][:, 0] for n, v in d.items()}
        want = ref.Gscan(d["x"][1], d["r"][1], d["i"][1], d["rate"][1], lerp, d["S0"][1])
        kept, S2 = t["S0"].clone(), torch.full((B, D), float("nan"), device="cuda")
        out = ssm.ssm_gscan_update(t["S0"], t["x"], t["r"], t["i"], t["rate"], lerp, state_out=S2)
        assert torch.equal(t["S0"], kept)
        near(out, want.h[:, 0], want.h_off[:, 0], HALF[dtype], "out")
        near(S2, want.last, want.last_off, 0, "state")
        out2 = ssm.ssm_gscan_update(t["S0"], t["x"], t["r"], t["i"], t["rate"], lerp)
        assert torch.equal(out, out2) and torch.equal(t["S0"], S2)


def test_step_of_slices():
    x = torch.randn(5, 300, device="cuda")
    S = torch.zeros(5, 96, device="cuda")
    a = ssm.ssm_gscan_update(S.clone(), x[:, 1:97], x[:, 101:197], x[:, 201:297])
    b = ssm.ssm_gscan_update(S.clone(), *[x[:, o:o + 96].contiguous() for o in (1, 101, 201)])
    assert torch.equal(a, b)


def test_saturated_gates():
    """Gates far out: decays of exactly 0 and 1, inputs shut and open, infinite arguments."""
    say("gscan saturated")
    B, L, D = 1, 140, 64
    d = draw(B, L, D, F32, True, False, seed=3)
    r, i = d["r"][1].copy(), d["i"][1].copy()
    r[:, 10::7], r[:, 11::7], i[:, 12::5], i[:, 13::5] = 90.0, -90.0, 60.0, -60.0
    r[:, 50], r[:, 60], i[:, 70], i[:, 80] = np.inf, -np.inf, np.inf, -np.inf
    finite = [np.clip(v, -90, 90) for v in (r, i)]
    for rate in (None, np.full(D, 1e-3, np.float32)):
        rt = None if rate is None else torch.from_numpy(rate).cuda()
        want = ref.Gscan(d["x"][1], finite[0], finite[1], rate, True, d["S0"][1])
        states = states_for(B, L, D)
        tr, ti = (torch.from_numpy(v.astype(np.float32)).cuda() for v in (r, i))
        out = ssm.ssm_gscan_fwd(d["x"][0], tr, ti, rt, True, d["S0"][0], states=states)
        near(out, want.h, want.h_off, 0, "out")
        g = ssm.ssm_gscan_bwd(d["x"][0], tr, ti, rt, d["dout"][0], states, True)
        for n, v in g.items():
            near(v, *want.grad(d["dout"][1])[n], 0, n)


def test_no_derivative_of_a_zero_coefficient():
    """A rate of 0 makes a = 1 and m = 0: h stays, and gradients stay finite."""
    d = draw(1, 70, 32, F32, True, True)
    rate = torch.zeros(32, device="cuda")
    states = states_for(1, 70, 32)
    out = ssm.ssm_gscan_fwd(*[d[n][0] for n in ("x", "r", "i")], rate, initial_state=d["S0"][0], states=states)
    assert torch.equal(out, d["S0"][0].unsqueeze(1).expand_as(out))
    g = ssm.ssm_gscan_bwd(*[d[n][0] for n in ("x", "r", "i")], rate, d["dout"][0], states)
    assert not g["dr"].any() and not g["dx"].any() and torch.isfinite(g["drate"]).all()


@pytest.mark.parametrize("name", ["x", "r", "i"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_in_their_channel(name, bad):
    """They reach their channel's later steps; earlier ones, other channels and rows keep their bits."""
    d = draw(2, 400, 70, F32, True, True)
    t = {n: d[n][0] for n in ("x", "r", "i")}
    clean = ssm.ssm_gscan_fwd(*t.values(), d["rate"][0])
    b, at, c = 1, 233, 17
    t[name][b, at, c] = bad
    got = ssm.ssm_gscan_fwd(*t.values(), d["rate"][0])
    hit = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
    hit[b, at:, c] = True
    assert torch.equal(got[~hit], clean[~hit])
    if bad != bad or name == "x":
        assert not torch.isfinite(got[b, at:at + 8, c]).any()
    else:
        assert torch.isfinite(got[hit]).all()          # an open gate


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_gradients_that_are_not_finite_reach_earlier_steps_only(bad):
    d = draw(2, 400, 70, F32, True, True)
    t = {n: d[n][0] for n in ("x", "r", "i")}
    states = states_for(2, 400, 70)
    ssm.ssm_gscan_fwd(*t.values(), d["rate"][0], states=states)
    dout = d["dout"][0]
    clean = ssm.ssm_gscan_bwd(*t.values(), d["rate"][0], dout, states)
    b, at, c = 1, 233, 17
    dout[b, at, c] = bad
    got = ssm.ssm_gscan_bwd(*t.values(), d["rate"][0], dout, states)
    hit = torch.zeros(dout.shape, dtype=torch.bool, device="cuda")
    hit[b, :at + 1, c] = True
    for n in ("dx", "dr", "di"):
        assert torch.equal(got[n][~hit], clean[n][~hit]), n
        assert not torch.isfinite(got[n][b, at, c]), n
    other = torch.arange(70, device="cuda") != c
    assert torch.equal(got["drate"][other], clean["drate"][other]) and not torch.isfinite(got["drate"][c])


def test_empty_calls():
    for shape in ((0, 5, 8), (2, 0, 8), (2, 5, 0)):
        B, L, D = shape
        x = torch.empty(shape, device="cuda")
        S, last = torch.randn(B, D, device="cuda"), torch.full((B, D), 7.0, device="cuda")
        rate = torch.ones(D, device="cuda")
        states = torch.empty(B, -(-L // SEG), D, device="cuda")
        ssm.ssm_gscan_fwd(x, x, x, rate, initial_state=S, last_state=last, states=states)
        assert torch.equal(last, S)
        g = ssm.ssm_gscan_bwd(x, x, x, rate, x, states, dlast_state=S, want_dinitial_state=True)
        assert torch.equal(g["dinitial_state"], S) and not g["drate"].any()
    ssm.ssm_gscan_fwd(torch.empty(2, 0, 8, device="cuda"), torch.empty(2, 0, 8, device="cuda"), last_state=last.new_full((2, 8), 7.0))


def test_bits_repeat():
    d = draw(3, 3000, 200, BF16, True, True)
    t = [d[n][0] for n in ("x", "r", "i", "rate")]
    states = states_for(3, 3000, 200)
    first = None
    for _ in range(4):
        out = ssm.ssm_gscan_fwd(*t, states=states, initial_state=d["S0"][0])
        g = ssm.ssm_gscan_bwd(*t, d["dout"][0], states, want_dinitial_state=True)
        now = [out, states.clone(), *g.values()]
        first = first or now
        for a, b in zip(now, first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("B,L,D", [(2047, 3, 20), (2048, 3, 20), (3000, 2, 70), (30, 5000, 20)])
def test_rates_gradient_over_many_tiles(B, L, D):
    check(B, L, D, BF16, True, True, False, False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [1, 40, 150])
def test_growing_decays(L, dtype):
    """Rates below zero, with 1 - a as the input's coefficient: a > 1."""
    d = draw(2, L, 66, dtype, True, True)
    rate, r64 = pair(np.random.default_rng(0).uniform(-1.2, 0.3, 66) * np.linspace(0.01, 1, 66), F32)
    states = states_for(2, L, 66)
    out = ssm.ssm_gscan_fwd(d["x"][0], d["r"][0], d["i"][0], rate, True, states=states)
    want = ref.Gscan(d["x"][1], d["r"][1], d["i"][1], r64, True)
    near(out, want.h, want.h_off, HALF[dtype], "out")
    g = ssm.ssm_gscan_bwd(d["x"][0], d["r"][0], d["i"][0], rate, d["dout"][0], states, True)
    for n, v in g.items():
        near(v, *want.grad(d["dout"][1])[n], HALF[dtype] if n != "drate" else 0, n)
    S = torch.zeros(2, 66, device="cuda")
    step = ssm.ssm_gscan_update(S, *(d[n][0][:, 0].contiguous() for n in "xri"), rate, True)
    near(step, want.h[:, 0], want.h_off[:, 0], HALF[dtype], "step")


@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 64, 65])
@pytest.mark.parametrize("D,dtype", [(66, BF16), (130, F32), (65, BF16)])
def test_short_sequences_of_many_rows(L, D, dtype):
    """Several rows to a workgroup, the last one's not all there."""
    check(37, L, D, dtype, True, True, False, True)
    check(5, L, D, dtype, False, False, True, False)
