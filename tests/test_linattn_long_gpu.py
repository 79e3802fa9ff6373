"""Linear attention over long time chunks (up to the backward's 64 chunks of 32 steps, and past
the forward's ring of 16), and its decay's gradient held to the gradient's own size.

Bars.  Outputs, gradients and states as in test_linattn_terms_gpu.py: 6e-7 of their norm.
dg_t is a border's <S, dS> and sums of the steps' parts from there, each part as exact as an
output (6e-7 of its size) and independent of the others, while dg_t itself adds up the same
parts: the two states of a border, the parts before it, those behind it, and the closing of the
recursion on both ends (at most the whole again) make sqrt(2 + 1 + 1 + 4 ..) < 4 times 6e-7,
held to 2.5e-6 of dg's root mean square.  A fixed decay's gradient is the sum over n = batch *
L steps.  A border's error is shared by at most 128 steps and independent of the next one's, so
the sum is off by at most 2.5e-6 sqrt(128 n) root mean squares, which are 1.25 mean magnitudes
(of normal values): 3.1e-6 sqrt(128 / n) of the sum of |dg_t| over the steps.
The readout in two bf16 terms, and one border per time chunk, do not pass.
"""
import pytest

import linattn_steps as steps
from gpu_util import say
from test_linattn_gpu import draw
from test_linattn_terms_gpu import NORM, off

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32 = torch.float32
DECAY, SHARED = 2.5e-6, 3.1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


@pytest.mark.parametrize("L,chunk_len", [(1100, 4096), (2100, 4096), (2100, 1024), (2049, 1024), (700, 4096)])
@pytest.mark.parametrize("B,H,G,dk,dv", [(2, 3, 3, 64, 40), (1, 4, 2, 128, 64)])
def test_forward_over_long_time_chunks(B, H, G, dk, dv, L, chunk_len):
    say(f"linattn {B} x {L}, heads {H}/{G}, dk {dk} dv {dv}, time chunks of {chunk_len}")
    d = {n: x[0] for n, x in draw(B, L, H, G, dk, dv, L + dk).items()}
    last = torch.empty(B, H, dv, dk, device="cuda")
    out = ssm.ssm_linattn_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["S0"], last_state=last, out_dtype=F32,
                              plan={"chunk_len": chunk_len})
    o, S = steps.forward(d["q"], d["k"], d["v"], d["g"], dk ** -0.5, d["S0"])
    assert off(out, o) <= NORM, f"out {off(out, o):.2e}"
    assert off(last, S) <= NORM, f"last_state {off(last, S):.2e}"


def workspace(B, L, H, G, dk, dv, n_chunks, chunk_len, states, fixed):
    """Bytes of workspace of the backward over so many time chunks (include/ssmblock.h)."""
    r4, k64, v64 = lambda n: -(-n // 4) * 4, -(-dk // 64), 128 if dv > 64 else 64  # noqa: E731
    state, heads = B * H * dk * dv, B * H * n_chunks
    n = 2 * r4(B * L * H * k64)
    if n_chunks > 1:
        n += 2 * r4(state * n_chunks) + 2 * r4(heads)
    n += 2 * r4(state) if states else 0
    n += 2 * r4(B * L * H * dk) if H > G else 0
    if fixed:
        n += r4(2 * heads) + 2 * r4(heads * ((-(-min(L, chunk_len) // 32) - 1) // 4) * k64 * 64 * v64)
    return 4 * n


# (more workgroups than CUs: time chunks are not cut below 2048 steps)
LONG = [(90, 2048, 1, 1, 8, 8, 1, 2048), (6, 2047, 15, 15, 8, 8, 1, 2048), (45, 1100, 2, 1, 16, 8, 1, 1120),
        (3, 2048, 15, 15, 128, 128, 1, 2048), (2, 5000, 45, 15, 64, 64, 3, 1696)]
SHORT = [(1, 700, 1, 1, 128, 128), (2, 333, 4, 2, 80, 128), (3, 200, 2, 2, 128, 64), (1, 1000, 2, 1, 128, 8)]


def check_gradients(B, L, H, G, dk, dv, states, fixed):
    d = {n: x[0] for n, x in draw(B, L, H, G, dk, dv, 11 * L + B, fixed).items()}
    S0, dl = (d["S0"], d["dlast"]) if states else (None, None)
    g = ssm.ssm_linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["dout"], initial_state=S0, dlast_state=dl,
                            want_dinitial_state=True, grad_dtype=F32)
    wanted = ssm.ssm_workspace_bytes()
    want = steps.gradients(d["q"], d["k"], d["v"], d["g"], dk ** -0.5, d["dout"], S0, dl)
    for n in ("dq", "dk", "dv", "dinitial_state"):
        assert off(g[n], want[n]) <= NORM, f"{n} {off(g[n], want[n]):.2e}"
    dg, got = want["dlog_decay"], g["dlog_decay"].double()
    if fixed:
        bar = SHARED * (128 / (B * L)) ** 0.5 * dg.abs().sum((0, 1))
        dg = dg.sum((0, 1))
        assert (dg.abs() > 2 * bar).all(), "zeros would pass"
        assert ((got - dg).abs() <= bar).all(), f"dlog_decay {((got - dg).abs() / bar).max():.2f} bars off"
    else:
        assert off(got, dg) <= DECAY, f"dlog_decay {off(got, dg):.2e}"
    return wanted


@pytest.mark.parametrize("B,L,H,G,dk,dv,n_chunks,chunk_len", LONG)
@pytest.mark.parametrize("fixed", [False, True])
@pytest.mark.parametrize("states", [False, True])
def test_gradients_over_long_time_chunks(B, L, H, G, dk, dv, n_chunks, chunk_len, states, fixed):
    say(f"linattn gradients {B} x {L}, heads {H}/{G}, dk {dk} dv {dv}, states {states}, fixed {fixed}")
    wanted = check_gradients(B, L, H, G, dk, dv, states, fixed)
    assert wanted == workspace(B, L, H, G, dk, dv, n_chunks, chunk_len, states, fixed), "time chunks are other than these"


@pytest.mark.parametrize("B,L,H,G,dk,dv", SHORT)
@pytest.mark.parametrize("fixed", [False, True])
@pytest.mark.parametrize("states", [False, True])
def test_decay_gradient_by_its_own_size(B, L, H, G, dk, dv, states, fixed):
    say(f"linattn decay gradient {B} x {L}, heads {H}/{G}, dk {dk} dv {dv}, states {states}, fixed {fixed}")
    check_gradients(B, L, H, G, dk, dv, states, fixed)
