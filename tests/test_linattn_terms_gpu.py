"""Linear attention's fp32 outputs, gradients and states hold fp32's precision: computed
operands enter the bf16 matrix cores with all their 24 bits.

The bar, in the 2-norm of an output's error over that of the output.  A value goes through at
most 4 + 1 products of 32 terms into an element of the score or the readout, three terms
each for four more of the readout and for one of the score: 22 instructions of at most 8
additions, below 180 roundings in a row, and a handful for the decays and factors; each is off
by 2^-24 / sqrt(3) of a partial sum in the mean, independently, and a partial sum of terms of either
sign is below the whole in norm: sqrt(180) * 3.4e-8 = 4.6e-7, held to 6e-7.  An operand in
two bf16 terms is off by up to 2^-18, 2e-6 in the mean, and does not pass.  Where one
term decides the output (one step, or one entry of the state), every element is held to 8
roundings of 2^-24 (two terms: up to 2^-18 = 64 of them).
"""
import pytest

import linattn_steps as steps
from gpu_util import say
from test_linattn_gpu import draw

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32, BF16 = torch.float32, torch.bfloat16
NORM, ONE = 6e-7, 8 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


SHAPES = [(2, 3, 4, 2, 64, 64), (1, 64, 2, 2, 128, 128), (2, 333, 4, 2, 80, 128), (1, 700, 3, 1, 32, 24)]


@pytest.mark.parametrize("B,L,H,G,dk,dv", SHAPES)
@pytest.mark.parametrize("fixed,chunk_len", [(False, None), (True, None), (False, 96)])
def test_forward_precision(B, L, H, G, dk, dv, fixed, chunk_len):
    say(f"linattn precision {B} x {L}, heads {H}/{G}, dk {dk} dv {dv}, fixed {fixed}, time chunks of {chunk_len}")
    d = {n: x[0] for n, x in draw(B, L, H, G, dk, dv, 5 * L + dk, fixed).items()}
    last = torch.empty(B, H, dv, dk, device="cuda")
    out = ssm.ssm_linattn_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["S0"], last_state=last, out_dtype=F32,
                              plan={"chunk_len": chunk_len} if chunk_len else None)
    o, S = steps.forward(d["q"], d["k"], d["v"], d["g"], dk ** -0.5, d["S0"])
    assert off(out, o) <= NORM, f"out {off(out, o):.2e}"
    assert off(last, S) <= NORM, f"last_state {off(last, S):.2e}"


@pytest.mark.parametrize("B,L,H,G,dk,dv", SHAPES)
@pytest.mark.parametrize("fixed", [False, True])
def test_gradient_precision(B, L, H, G, dk, dv, fixed):
    say(f"linattn gradients' precision {B} x {L}, heads {H}/{G}, dk {dk} dv {dv}, fixed {fixed}")
    d = {n: x[0] for n, x in draw(B, L, H, G, dk, dv, 7 * L + dv, fixed).items()}
    g = ssm.ssm_linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["dout"], initial_state=d["S0"], dlast_state=d["dlast"],
                            want_dinitial_state=True, grad_dtype=F32)
    want = steps.gradients(d["q"], d["k"], d["v"], d["g"], dk ** -0.5, d["dout"], d["S0"], d["dlast"])
    for n in ("dq", "dk", "dv", "dinitial_state"):
        assert off(g[n], want[n]) <= NORM, f"{n} {off(g[n], want[n]):.2e}"


def test_one_entry_of_the_state():
    """q picks one column of the state: out is an entry times a decay."""
    say("linattn: one entry of the state")
    B, H, dk, dv = 2, 3, 64, 64
    gen = torch.Generator(device="cpu").manual_seed(3)
    S0 = torch.randn(B, H, dv, dk, generator=gen).cuda()
    q = torch.zeros(B, dk, H, dk, device="cuda", dtype=BF16)
    q[:, range(dk), :, range(dk)] = 1.0
    z = torch.zeros(B, dk, H, dv, device="cuda", dtype=BF16)
    out = ssm.ssm_linattn_fwd(q, torch.zeros_like(q), z, torch.zeros(B, dk, H, device="cuda"), scale=1.0, initial_state=S0,
                              out_dtype=F32)
    want = S0.double().permute(0, 3, 1, 2)
    assert ((out.double() - want).abs() <= ONE * want.abs()).all(), ((out.double() - want) / want).abs().max()


def test_one_score():
    """One step from nothing: out is (q . k) scale times v, with a score of all 24 bits."""
    say("linattn: one score")
    d = {n: x[0] for n, x in draw(64, 1, 4, 4, 8, 64, 9).items()}
    out = ssm.ssm_linattn_fwd(d["q"], d["k"], d["v"], d["g"], scale=0.3, out_dtype=F32)
    qk = (d["q"].double() * d["k"].double())
    want = torch.tensor(0.3, dtype=F32).double().item() * qk.sum(-1, keepdim=True) * d["v"].double()
    size = 0.3 * qk.abs().sum(-1, keepdim=True) * d["v"].double().abs()
    assert ((out.double() - want).abs() <= ONE * size).all(), ((out.double() - want).abs() / size).max()
