"""The block operators' 64-bit references (block_ref.py) against differences of
their own forwards and against properties of the definitions (CPU)."""
import numpy as np
import pytest

import block_ref as ref

H = 1e-5
# A central difference of a smooth function of order one has an error of about
# H^2 (third derivative) + 2e-16 / H (rounding): 1e-10 and 2e-11, times the
# number of outputs summed; the bar leaves four orders of magnitude.
TOL = 1e-6


def difference(f, a):
    """d sum(f) / d a by central differences."""
    g = np.zeros_like(a)
    it = np.nditer(a, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = a[i]
        a[i] = old + H
        up = f()
        a[i] = old - H
        down = f()
        a[i] = old
        g[i] = (up - down) / (2 * H)
    return g


def check(got, want):
    assert np.abs(got - want).max() <= TOL * (1 + np.abs(want).max())


@pytest.mark.parametrize("center", [False, True])
def test_add_norm_gradients(center):
    r = np.random.default_rng(1)
    x, res, dout, dres = (r.standard_normal((3, 7)) for _ in range(4))
    w, b, scale = (r.uniform(0.5, 1.5, 7) for _ in range(3))
    alpha, eps = 0.7, 1e-3

    def loss():
        o, s = ref.add_norm(x, res, w, b, scale, alpha, eps, center)
        return (o * dout).sum() + (s * dres).sum()

    rr = ref.add_norm(x, res, w, b, scale, alpha, eps, center)[1]
    dx, dr, dw, db, ds = ref.add_norm_grad(dout, rr, w, dres, x, scale, alpha, eps, center)
    for got, a in ((dx, x), (dr, res), (dw.sum(0), w), (db.sum(0), b), (ds.sum(0), scale)):
        check(got, difference(loss, a))


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("gate_first", [False, True])
def test_gated_norm_gradients(gate_first, center):
    r = np.random.default_rng(2)
    x, z, dout = (r.standard_normal((3, 12)) for _ in range(3))
    w, b = (r.uniform(0.5, 1.5, 12) for _ in range(2))
    f = lambda: (ref.gated_norm(x, z, w, b, 3, gate_first, 1e-3, center) * dout).sum()  # noqa: E731
    dx, dz, dw, db = ref.gated_norm_grad(dout, x, z, w, b, 3, gate_first, 1e-3, center)
    for got, a in ((dx, x), (dz, z), (dw.sum(0), w), (db.sum(0), b)):
        check(got, difference(f, a))


@pytest.mark.parametrize("fixed", [False, True])
def test_linattn_gradients(fixed):
    r = np.random.default_rng(3)
    q, k = r.standard_normal((2, 5, 2, 3)), r.standard_normal((2, 5, 2, 3))
    v, dout = r.standard_normal((2, 5, 4, 2)), r.standard_normal((2, 5, 4, 2))
    g = -r.uniform(0.01, 1.0, (4,) if fixed else (2, 5, 4))
    S0, dl = r.standard_normal((2, 4, 2, 3)), r.standard_normal((2, 4, 2, 3))

    def loss():
        o, S = ref.linattn(q, k, v, g, 0.6, S0)
        return (o * dout).sum() + (S * dl).sum()

    got = ref.linattn_grad(q, k, v, g, 0.6, dout, S0, dl)
    for n, a in (("dq", q), ("dk", k), ("dv", v), ("dlog_decay", g), ("dinitial_state", S0)):
        check(got[n], difference(loss, a))


def test_linattn_is_the_masked_product():
    """Without a state, o = scale (Q K^T o D) V with D_ts = exp(sum of g over (s, t]) for s <= t."""
    r = np.random.default_rng(4)
    q, k, v = r.standard_normal((1, 6, 1, 3)), r.standard_normal((1, 6, 1, 3)), r.standard_normal((1, 6, 1, 2))
    g = -r.uniform(0.01, 1.0, (1, 6, 1))
    o, _ = ref.linattn(q, k, v, g, 1.0)
    for t in range(6):
        want = sum(np.exp(g[0, s + 1:t + 1, 0].sum()) * (q[0, t, 0] @ k[0, s, 0]) * v[0, s, 0] for s in range(t + 1))
        np.testing.assert_allclose(o[0, t, 0], want, rtol=1e-12)
    # a decay of minus infinity forgets everything before its step
    g[0, 3] = -np.inf
    o2, _ = ref.linattn(q, k, v, g, 1.0)
    o3, _ = ref.linattn(q[:, 3:], k[:, 3:], v[:, 3:], g[:, 3:], 1.0)
    np.testing.assert_allclose(o2[:, 3:], o3, rtol=1e-12)
