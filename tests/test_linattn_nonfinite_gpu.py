"""Values that are not finite in linear attention's gradients: what depends on such a value is
not finite, and everything else keeps its bits.  With S and dS the states and their
gradients, dq_t = S_t^T dout_t, dk_t = dS_t^T v_t and dv_t = dS_t k_t (scale aside): a value of k
or v at step t is in S from t on, one of q or dout in dS up to t, a decay in S from t on
and in dS before t; a column of k reaches that column of dq and a row of dv, and so on.
A decay may also reach dk and dv of the steps behind it in its 32, whose decays are differences
of sums over all of them (include/ssmblock.h).
The decay's gradient, whose sums are closed over a time chunk, may be lost in all of the time
chunks that the value's step and what it reaches lie in, but in no other head or batch row."""
import pytest

from gpu_util import say
from test_linattn_gpu import draw

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32 = torch.float32
COL = 5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


# what of dq, dk and dv a value at step t reaches: (steps, columns), "=" the step itself
REACH = {
    "q": {"dk": ("<=", COL), "dv": ("<=", None)},
    "k": {"dq": (">=", COL), "dv": ("=", None)},
    "v": {"dq": (">=", None), "dk": ("=", None)},
    "dout": {"dq": ("=", None), "dk": ("<=", None), "dv": ("<=", COL)},
    "g": {"dq": (">=", None), "dk": ("<", None), "dv": ("<", None)},
}


def span(rel, t, L):
    return {"<=": slice(0, t + 1), "<": slice(0, t), ">=": slice(t, L), "=": slice(t, t + 1)}[rel]


@pytest.mark.parametrize("name", list(REACH))
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("L,t", [(150, 70), (150, 149), (150, 0), (1500, 800), (1500, 1023)])
@pytest.mark.parametrize("share", [1, 2])
def test_gradients_of_values_that_are_not_finite(name, bad, L, t, share):
    say(f"linattn gradients: {bad} in {name}, step {t} of {L}, {share} heads share")
    B, G, dk, dv = 2, 2, 64, 72
    H = G * share
    d = {n: x[0].clone() for n, x in draw(B, L, H, G, dk, dv, L + t).items()}

    def run():
        return ssm.ssm_linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["dout"], initial_state=d["S0"], dlast_state=d["dlast"],
                                   want_dinitial_state=True, grad_dtype=F32)
    clean = run()
    h, grp = H - 1, G - 1                       # the head and its group
    if name == "g":
        d["g"][0, t, h] = bad
    else:
        d[name][0, t, grp if name in "qk" else h, COL] = bad
    got = run()
    heads = range(grp * share, H) if name in "qk" else [h]
    for n in ("dq", "dk", "dv"):
        own = {grp} if n != "dv" else set(heads)
        lost = torch.zeros_like(got[n], dtype=torch.bool)
        if n in REACH[name]:
            rel, col = REACH[name][n]
            for i in own:
                lost[0, span(rel, t, L), i, slice(None) if col is None else slice(col, col + 1)] = True
        same = ~lost
        if name == "g" and n != "dq":
            same[0, t:(t // 32 + 1) * 32, list(own)] = False
        assert torch.equal(got[n][same], clean[n][same]), f"{n}: what the value does not reach has changed"
        assert not torch.isfinite(got[n][lost]).any(), f"{n}: what the value reaches is finite"
    # the decay's gradient of dS S: steps up to t (of a q or dout), after t (of a k or v)
    reached = span("<=" if name in ("q", "dout") else ">=", t, L)
    first = reached.start + (0 if name in ("q", "dout", "g") else 1)
    keep = torch.ones_like(clean["dlog_decay"], dtype=torch.bool)
    for i in heads:
        keep[0, :, i] = False
        assert not torch.isfinite(got["dlog_decay"][0, first:reached.stop, i]).any(), "dlog_decay: what the value reaches is finite"
    assert torch.equal(got["dlog_decay"][keep], clean["dlog_decay"][keep]), "dlog_decay of another head or batch row has changed"
    first_state = got["dinitial_state"]
    for b in range(B):
        for i in range(H):
            if b == 0 and i in heads and name in ("q", "dout", "g"):
                part = first_state[b, i]
                part = part[:, COL] if name == "q" else part[COL] if name == "dout" else part
                assert not torch.isfinite(part).any(), "dinitial_state is finite"
            else:
                assert torch.equal(first_state[b, i], clean["dinitial_state"][b, i])
