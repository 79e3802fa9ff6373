"""The gated linear recurrence at the ends of its ranges, against the 64-bit reference."""
import numpy as np
import pytest

import model_ref as ref
from gpu_util import say
from test_gscan_gpu import SEG, near, pair, states_for

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 0.0, BF16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


def run(x, r, i, rate, lerp, dout, dtype, S0=None, dlast=None):
    """Forward and gradients held to the reference's bars; all arguments are arrays of fp32 values."""
    B, L, D = x.shape
    (x, xd), (r, rd), (dout, dd) = pair(x, dtype), pair(r, dtype), pair(dout, dtype)
    i, id_ = (None, None) if i is None else pair(i, dtype)
    rate, ra = (None, None) if rate is None else pair(rate, F32)
    S0, Sd = (None, None) if S0 is None else pair(S0, F32)
    dlast, dl = (None, None) if dlast is None else pair(dlast, F32)
    want = ref.Gscan(xd, rd, id_, ra, lerp, Sd)
    last, states = torch.full((B, D), float("nan"), device="cuda"), states_for(B, L, D)
    out = ssm.ssm_gscan_fwd(x, r, i, rate, lerp, S0, last_state=last, states=states)
    near(out, want.h, want.h_off, HALF[dtype], "out")
    near(last, want.last, want.last_off, 0, "last_state")
    near(states, want.before[:, ::SEG], want.before_off[:, ::SEG], 0, "states")
    g = ssm.ssm_gscan_bwd(x, r, i, rate, dout, states, lerp, dlast, want_dinitial_state=True)
    wg = want.grad(dd, dl)
    for n, v in g.items():
        near(v, *wg[n], HALF[dtype] if n in ("dx", "dr", "di") else 0, n)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_token_of_many_narrow_rows(dtype):
    """More rows than the sequences' grids have workgroups: the same bits as of one wide row."""
    say(f"many narrow rows {dtype}")
    B = (1 << 23) + 5
    g = torch.Generator(device="cuda").manual_seed(0)
    x, r, i = (torch.randn(B, 1, device="cuda", generator=g).to(dtype) for _ in range(3))
    S, wide = (torch.randn(B, 1, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) for _ in range(2))
    out = ssm.ssm_gscan_update(S, x, r, i)
    want = ssm.ssm_gscan_update(wide.view(1, B), *(t.view(1, B) for t in (x, r, i)))
    assert torch.equal(out.view(1, B), want) and torch.equal(S, wide)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rate", [-1.5, -30.0])
@pytest.mark.parametrize("L", [100, 400, 3000])
def test_states_of_zero_through_growing_decays(L, rate, dtype):
    """Steps with decays far above 1 and no input in front: their product leaves fp32's range, the states stay 0."""
    say(f"zeros in front {L} {rate} {dtype}")
    B, D = 2, 66
    g = np.random.default_rng(2)
    front = L - 40
    x, r = g.standard_normal((B, L, D)), np.full((B, L, D), 0.0)
    x[:, :front] = 0
    r[:, front:] = -6.0
    xt, rt, rate_t = (torch.from_numpy(np.float32(v)).cuda() for v in (x, r, np.full(D, rate)))
    xt, rt = xt.to(dtype), rt.to(dtype)
    want = ref.Gscan(xt.double().cpu().numpy(), rt.double().cpu().numpy(), None, np.full(D, rate), True)
    last, states = torch.full((B, D), float("nan"), device="cuda"), states_for(B, L, D)
    out = ssm.ssm_gscan_fwd(xt, rt, None, rate_t, True, last_state=last, states=states)
    assert not out[:, :front].any()
    near(out, want.h, want.h_off, HALF[dtype], "out")
    near(last, want.last, want.last_off, 0, "last_state")
    near(states, want.before[:, ::SEG], want.before_off[:, ::SEG], 0, "states")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rate", [-1.5, -30.0])
@pytest.mark.parametrize("L", [100, 400, 3000])
def test_gradients_of_zero_through_growing_decays(L, rate, dtype):
    """The same from behind: no gradient arrives in the last steps, whose decays' product leaves fp32's range."""
    say(f"zeros behind {L} {rate} {dtype}")
    B, D = 2, 66
    g = np.random.default_rng(3)
    x, r, dout = np.zeros((B, L, D)), np.full((B, L, D), 0.0), g.standard_normal((B, L, D))
    r[:, :40] = -6.0
    dout[:, 40:] = 0
    run(x, r, None, np.full(D, rate), True, dout, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("lerp", [True, False])
def test_closed_and_open_gates_without_a_rate(gate, lerp, dtype):
    """sigmoid(r) and 1 - sigmoid(r) down to fp32's smallest normal numbers: the gradient of r falls as they do.

    Closed gates keep no state, so dr is about g h e^r: relative to that it is held to the bars of everything else
    (a few roundings for each unit of |r|)."""
    say(f"far gates {gate} {lerp} {dtype}")
    B, L, D = 2, 150, 66
    g = np.random.default_rng(1)
    r = -g.uniform(40, 80, (B, L, D))
    r[:, :, ::3] *= -1
    r[:, ::5] = g.standard_normal(r[:, ::5].shape)
    i = g.standard_normal((B, L, D)) if gate else None
    run(g.standard_normal((B, L, D)), r, i, None, lerp, g.standard_normal((B, L, D)), dtype,
        g.standard_normal((B, D)), g.standard_normal((B, D)))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [13, 30, 60])
def test_zeros_through_growing_decays_of_short_sequences(L, dtype):
    """As above where one wavefront, or several of a workgroup, hold a sequence, of many rows."""
    say(f"zeros, short {L} {dtype}")
    B, D, rate = 21, 66, np.full(66, -30.0)
    g = np.random.default_rng(4)
    x, r, dout = g.standard_normal((B, L, D)), np.zeros((B, L, D)), g.standard_normal((B, L, D))
    front, back = x.copy(), dout.copy()
    front[:, :L - 3], back[:, 3:] = 0, 0
    late, early = r.copy(), r.copy()
    late[:, L - 3:], early[:, :3] = -6.0, -6.0
    (xt, xd), (rt, rd) = pair(front, dtype), pair(late, dtype)
    rate_t, ra = pair(rate, F32)
    want = ref.Gscan(xd, rd, None, ra, True)
    out = ssm.ssm_gscan_fwd(xt, rt, None, rate_t, True)
    near(out, want.h, want.h_off, HALF[dtype], "out")
    assert not out[:, :L - 3].any()
    run(np.zeros_like(x), early, None, rate, True, back, dtype)
