"""Plain 64-bit references of the model operators (include/ssmmodel.h), with the bars that
fp32 arithmetic is held to (not a test module).

``U`` is half a step of fp32 relative to a value.  A bar counts the roundings that an
element's value passes through, each times the magnitude that it rounds; the counts are
beside them."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}


def sigmoid(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


class Gscan:
    """The recurrence in 64 bits over x, r [B, L, D] (and i, rate [D]): the values, and for each how far fp32
    arithmetic may be off.

    Half steps of a coefficient: a sigmoid is an exponential (2, and 2 for its argument's rounding near 0; an
    argument v has |v| of them more, since e^v moves by v's error), a sum (1) and a reciprocal (2); a decay adds
    a product (1) and an exponential of argument y (2 + y times what y is off by); 1 - e^-w divides what e^-w <
    0.61 is off by through a difference of at least 0.39, and its square root halves that.  That is under
    ``count`` = 40 + 2 |v| for every coefficient, |v| the largest gate argument."""

    def __init__(self, x, r, i=None, rate=None, lerp=False, initial=None):
        x, r = np.asarray(x, np.float64), np.asarray(r, np.float64)
        self.x, self.rate, self.lerp, self.has_i = x, rate, lerp, i is not None
        self.pos, self.neg = sigmoid(r), sigmoid(-r)
        if rate is None:
            self.a, rest = self.pos, self.neg
        else:
            y = rate * self.pos
            self.a, rest = np.exp(-y), -np.expm1(-y)
        self.m = rest if lerp else np.sqrt(rest * (1 + self.a))
        self.ipos, self.ineg = (sigmoid(np.asarray(i, np.float64)), sigmoid(-np.asarray(i, np.float64))) if i is not None \
            else (np.ones_like(x), np.zeros_like(x))
        self.u = x * self.ipos
        biggest = max(np.abs(r).max(initial=0), 0 if i is None else np.abs(i).max(initial=0))
        self.c = (40 + 2 * biggest) * U * (1 + (0 if rate is None else np.abs(rate).max(initial=0)))
        B, L, D = x.shape
        h = np.zeros((B, D)) if initial is None else np.asarray(initial, np.float64)
        size, off = np.abs(h), np.zeros((B, D))
        self.before, self.before_off, self.h, self.h_off = (np.zeros((B, L, D)) for _ in range(4))
        self.before_size = np.zeros((B, L, D))
        b = self.m * self.u
        for t in range(L):
            self.before[:, t], self.before_off[:, t], self.before_size[:, t] = h, off, size
            a = self.a[:, t]
            # a step adds what a and b are off by, and two roundings
            off = a * off + self.c * (a * size + np.abs(b[:, t]))
            size = a * size + np.abs(b[:, t])
            h = a * h + b[:, t]
            self.h[:, t], self.h_off[:, t] = h, off
        self.last, self.last_off = h, off

    def grad(self, dout, dlast=None):
        """name -> (gradient, bar)."""
        dout = np.asarray(dout, np.float64)
        B, L, D = dout.shape
        carry = np.zeros((B, D)) if dlast is None else np.asarray(dlast, np.float64)
        size, off = np.abs(carry), np.zeros((B, D))
        g, g_off, g_size = (np.zeros((B, L, D)) for _ in range(3))
        for t in range(L - 1, -1, -1):
            g[:, t] = dout[:, t] + carry
            size = np.abs(dout[:, t]) + size
            off = off + 2 * U * size
            g_off[:, t], g_size[:, t] = off, size
            a = self.a[:, t]
            carry, off, size = a * g[:, t], a * off + self.c * a * size, a * size
        a, m, u, c = self.a, self.m, self.u, self.c
        slope = -a if self.lerp else np.where(m == 0, 0.0, -a * a / np.where(m == 0, 1.0, m))
        inner = a * self.before + u * slope
        inner_off = a * self.before_off + c * (a * self.before_size + np.abs(u * slope)) * 2
        e = g * inner
        e_off = g_off * np.abs(inner) + np.abs(g) * inner_off + g_off * inner_off + 4 * U * np.abs(e)
        by = self.neg * (1 if self.rate is None else -self.rate * self.pos)
        gm_off = (g_off + 2 * c * np.abs(g)) * np.abs(m)
        out = {"dx": (g * m * self.ipos, (gm_off + c * np.abs(g * m)) * self.ipos),
               "dr": (e * by, (e_off + 2 * c * np.abs(e)) * np.abs(by))}
        if self.has_i:
            out["di"] = (g * m * u * self.ineg, (gm_off + 2 * c * np.abs(g * m)) * np.abs(u) * self.ineg)
        if self.rate is not None:
            # a sum over B L terms, added in any order: n roundings of what has been added
            n = B * L
            out["drate"] = (-(e * self.pos).sum((0, 1)),
                            ((e_off + 2 * c * np.abs(e)) * self.pos).sum((0, 1)) + n * U * np.abs(e * self.pos).sum((0, 1)))
        out["dinitial_state"] = (carry, off)
        return out


def softmax_teacher(index, teacher, vocab, temperature):
    """q [T, K], rows that count, rows with an index past the vocabulary."""
    has = (index >= 0) & (teacher != -np.inf)
    past = (index >= vocab).any(-1)
    counts = has.any(-1) & ~past
    l = np.where(has & counts[:, None], teacher, -np.inf) / temperature
    top = np.where(counts, l.max(-1), 0.0)
    q = np.exp(l - top[:, None])
    return q / np.maximum(q.sum(-1, keepdims=True), 1e-300), counts, past


class Head:
    """z = scale x w^T / temperature of x [T, D], w [V, D] in 64 bits; their log sum of exponentials; bars: a logit
    sums D products in fp32 (D + 2 roundings of the sum of their magnitudes; matrix cores may cut where others
    round: twice that)."""

    def __init__(self, x, w, scale=1.0, temperature=1.0):
        self.x, self.w, self.scale, self.t = np.asarray(x, np.float64), np.asarray(w, np.float64), scale, temperature
        by = scale / temperature
        self.z = self.x @ self.w.T * by
        self.z_off = 2 * (x.shape[1] + 4) * U * (np.abs(self.x) @ np.abs(self.w).T) * abs(by)
        top = self.z.max(-1)
        self.lse = top + np.log(np.exp(self.z - top[:, None]).sum(-1))
        # what the logits are off by; sums of up to a thousand parts; top and the logarithm times a rounded constant
        self.lse_off = self.z_off.max(-1) + U * (300 + 8 * np.abs(top) + 8 * np.abs(self.lse))

    def xent(self, target, z_loss=0.0):
        V = self.z.shape[1]
        has = (target >= 0) & (target < V)
        rows = np.arange(len(target))
        at = np.where(has, target, 0)
        loss = np.where(has, self.lse - self.z[rows, at] + z_loss * self.lse ** 2, 0.0)
        off = np.where(has, (self.lse_off + self.z_off[rows, at] + 4 * U * (np.abs(self.lse) + np.abs(self.z[rows, at]))) +
                       abs(z_loss) * np.abs(self.lse) * (2 * self.lse_off + 8 * U * np.abs(self.lse)), 0.0)
        loss[target >= V] = np.nan
        soft = np.where(has, 1 + 2 * z_loss * self.lse, 0.0)
        hard = np.zeros_like(self.z)
        hard[rows, at] = has
        return loss, off, soft, hard

    def distill(self, index, teacher):
        V = self.z.shape[1]
        q, counts, past = softmax_teacher(index, teacher, V, self.t)
        rows = np.arange(len(index))[:, None]
        at = np.where((index >= 0) & (index < V), index, 0)
        mine = self.z[rows, at]
        with np.errstate(divide="ignore", invalid="ignore"):
            terms = np.where(q > 0, q * (np.log(q) - mine + self.lse[:, None]), 0.0)
            size = np.where(q > 0, q * (np.abs(np.log(q)) + np.abs(mine) + np.abs(self.lse[:, None])), 0.0)
        big = np.abs(np.where(np.isfinite(teacher), teacher, 0)).max(-1) / self.t
        loss = np.where(counts, self.t ** 2 * terms.sum(-1), 0.0)
        # a term: its logarithms and difference, and q through an exponential of up to big
        off = np.where(counts, self.t ** 2 * ((q * self.z_off[rows, at]).sum(-1) + self.lse_off +
                                              U * (size.sum(-1) * (40 + 8 * big + index.shape[1]) + 8 * big)), 0.0)
        loss[past] = np.nan
        hard = np.zeros_like(self.z)
        np.add.at(hard, (np.broadcast_to(rows, at.shape), at), np.where(counts[:, None], q, 0.0))
        return loss, off, counts.astype(np.float64), hard

    def grad(self, dloss, soft, hard, takes):
        """(dx, bar), (dweight, bar) of sum dloss loss, with rows outside ``takes`` left out.  dz is rounded to bf16:
        2^-8 of itself; before that it is off by what its exponential's argument and the softmax's factors are."""
        f = np.where(takes, dloss * self.scale / self.t * self.t ** 2, 0.0)[:, None]
        p = np.exp(self.z - self.lse[:, None])
        dz = f * (p * soft[:, None] - hard)
        arg = self.z_off + self.lse_off[:, None] + 8 * U * (np.abs(self.z) + np.abs(self.lse[:, None]) + 4)
        off = np.abs(f) * (p * np.abs(soft[:, None]) * arg + 60 * U * (p + hard))
        off = off * 1.01 + 2.0 ** -8 * (np.abs(dz) + off)
        x = np.where(takes[:, None], self.x, 0.0)

        def product(a, a_off, b):
            v = a @ b
            size = np.abs(a) @ np.abs(b)
            return v, a_off @ np.abs(b) + 2 * (a.shape[1] + 8) * U * size + 2.0 ** -8 * np.abs(v) * 1.01
        return product(dz, off, self.w), product(dz.T, off.T, x)
