"""The 64-bit references of the model operators (model_ref.py): their gradients against
differences, and the recurrence against its closed form."""
import numpy as np
import pytest

import model_ref as ref


def draw(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("lerp", [False, True])
@pytest.mark.parametrize("with_rate", [False, True])
@pytest.mark.parametrize("with_i", [False, True])
def test_recurrence_gradients_against_differences(lerp, with_rate, with_i):
    B, L, D = 2, 5, 3
    at = {"x": draw(0, B, L, D), "r": draw(1, B, L, D), "initial": draw(2, B, D)}
    if with_i:
        at["i"] = draw(3, B, L, D)
    if with_rate:
        at["rate"] = np.abs(draw(4, D)) + 0.1
    dout, dlast = draw(5, B, L, D), draw(6, B, D)

    def value(args):
        g = ref.Gscan(lerp=lerp, **args)
        return (g.h * dout).sum() + (g.last * dlast).sum()
    got = ref.Gscan(lerp=lerp, **at).grad(dout, dlast)
    names = {"x": "dx", "r": "dr", "i": "di", "rate": "drate", "initial": "dinitial_state"}
    assert set(names[n] for n in at) == set(got)
    for n, v in at.items():
        grad = np.zeros_like(v)
        for j in np.ndindex(v.shape):
            step = np.zeros_like(v)
            step[j] = 1e-5
            grad[j] = (value({**at, n: v + step}) - value({**at, n: v - step})) / 2e-5
        # differences over 1e-5 of third derivatives of order 10: 1e-9, and roundings of 1e-16 * 30 / 1e-5
        np.testing.assert_allclose(got[names[n]][0], grad, rtol=1e-7, atol=1e-7)


def test_recurrence_against_its_closed_form():
    x, r, rate, h0 = draw(0, 1, 40, 2), draw(1, 1, 40, 2), np.array([0.3, 2.0]), draw(2, 1, 2)
    a = np.exp(-rate / (1 + np.exp(-r)))
    for lerp in (False, True):
        b = (1 - a if lerp else np.sqrt(1 - a * a)) * x
        h = [np.prod(a[:, :t + 1], 1) * h0 + sum(np.prod(a[:, s + 1:t + 1], 1) * b[:, s] for s in range(t + 1)) for t in range(40)]
        np.testing.assert_allclose(ref.Gscan(x, r, None, rate, lerp, h0).h, np.stack(h, 1), rtol=1e-12, atol=1e-13)


def head_value(x, w, loss_of, dloss, scale, t):
    return np.nansum(loss_of(ref.Head(x, w, scale, t)) * dloss)


@pytest.mark.parametrize("kind", ["xent", "xent z_loss", "distill", "distill warm"])
def test_loss_gradients_against_differences(kind):
    T, D, V, K = 5, 3, 11, 4
    x, w, dloss = draw(0, T, D), draw(1, V, D), draw(2, T)
    scale, t = 1.3, 2.0 if kind == "distill warm" else 1.0
    if kind.startswith("xent"):
        target, zl = np.array([3, 0, -1, 10, 3]), 0.1 if "z_loss" in kind else 0.0
        takes = target >= 0

        def parts(h):
            return h.xent(target, zl)
    else:
        index = np.array([[1, 2, 3, 4], [0, 0, 5, 10], [7, -1, 8, -1], [-1, -1, -1, -1], [9, 3, 9, 9]])
        teacher = draw(3, T, K)
        teacher[0, 2] = -np.inf
        takes = np.array([True, True, True, False, True])

        def parts(h):
            return h.distill(index, teacher)
    h = ref.Head(x, w, scale, t)
    loss, _, soft, hard = parts(h)
    assert np.isfinite(loss).all() and (loss[~takes] == 0).all()
    (dx, _), (dw, _) = h.grad(dloss, soft, hard, takes)
    for v, grad, other in ((x, dx, lambda a: (a, w)), (w, dw, lambda a: (x, a))):
        diff = np.zeros_like(v)
        for j in np.ndindex(v.shape):
            step = np.zeros_like(v)
            step[j] = 1e-5
            diff[j] = (head_value(*other(v + step), lambda h: parts(h)[0], dloss, scale, t) -
                       head_value(*other(v - step), lambda h: parts(h)[0], dloss, scale, t)) / 2e-5
        np.testing.assert_allclose(grad, diff, rtol=1e-7, atol=1e-7)


def test_rows_past_the_vocabulary_are_nan():
    h = ref.Head(draw(0, 2, 3), draw(1, 5, 3))
    assert np.isnan(h.xent(np.array([5, 1]))[0]).tolist() == [True, False]
    assert np.isnan(h.distill(np.array([[1, 7], [1, 2]]), draw(2, 2, 2))[0]).tolist() == [True, False]
