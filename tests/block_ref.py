"""Plain 64-bit implementations of the block operators (include/ssmblock.h), used
by their tests (not a test module).  Written from the definitions, one row, one
step and one product at a time; the gradients are the chain rule written out, and
test_block_ref.py checks them against differences of the forwards.
"""
from __future__ import annotations

import numpy as np


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))


def dsilu(z):
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _groups(a, g):
    return a.reshape(*a.shape[:-1], g, a.shape[-1] // g)


def norm(r, w, b, eps, center):
    """Rows of r over the last axis."""
    m = r.mean(-1, keepdims=True) if center else 0.0
    n = (r - m) / np.sqrt(((r - m) ** 2).mean(-1, keepdims=True) + eps)
    n = n if w is None else n * w
    return n if b is None else n + b


def norm_grad(dy, r, w, eps, center):
    """(dr, rows of dweight, rows of dbias) of norm."""
    m = r.mean(-1, keepdims=True) if center else 0.0
    std = np.sqrt(((r - m) ** 2).mean(-1, keepdims=True) + eps)
    n = (r - m) / std
    u = dy if w is None else dy * w
    d = u - n * (u * n).mean(-1, keepdims=True)
    if center:
        d = d - u.mean(-1, keepdims=True)
    return d / std, dy * n, dy + 0 * n


def add_norm(x, residual, w, b, scale, alpha, eps, center):
    r = x if scale is None else x * scale
    if residual is not None:
        r = r + alpha * residual
    return norm(r, w, b, eps, center), r


def add_norm_grad(dout, r, w, dres, x, scale, alpha, eps, center):
    """dx, dresidual, and the rows whose sums are dweight, dbias and dscale."""
    d, dw, db = norm_grad(dout, r, w, eps, center)
    if dres is not None:
        d = d + dres
    return (d if scale is None else d * scale), alpha * d, dw, db, (None if x is None else x * d)


def gated_norm(x, z, w, b, g, gate_first, eps, center):
    x, w, b = _groups(x, g), (None if w is None else _groups(w, g)), (None if b is None else _groups(b, g))
    s = 1.0 if z is None else silu(_groups(z, g))
    y = norm(x * s, w, b, eps, center) if gate_first else norm(x, w, b, eps, center) * s
    return y.reshape(*y.shape[:-2], -1)


def gated_norm_grad(dout, x, z, w, b, g, gate_first, eps, center):
    """dx, dz, and the rows whose sums are dweight and dbias."""
    shape = x.shape
    dout, x = _groups(dout, g), _groups(x, g)
    w, b = (None if w is None else _groups(w, g)), (None if b is None else _groups(b, g))
    s = np.ones_like(x) if z is None else silu(_groups(z, g))
    ds = np.zeros_like(x) if z is None else dsilu(_groups(z, g))
    if gate_first:
        d, dw, db = norm_grad(dout, x * s, w, eps, center)
        dx, dz = d * s, d * x * ds
    else:
        dx, dw, db = norm_grad(dout * s, x, w, eps, center)
        dz = dout * norm(x, w, b, eps, center) * ds
    return [a.reshape(shape) for a in (dx, dz, dw, db)]


def _per_head(a, H):
    """[B, L, G, d] -> [B, L, H, d]: every group serves H / G consecutive heads."""
    return np.repeat(a, H // a.shape[2], axis=2)


def linattn(q, k, v, g, scale, S0=None):
    """S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t.  q, k [B, L, G, dk], v [B, L, H, dv], g [B, L, H] or
    [H].  Returns o and the last state [B, H, dv, dk]."""
    B, L, H, dv = v.shape
    q, k = _per_head(q, H), _per_head(k, H)
    a = np.exp(np.broadcast_to(g, (B, L, H)))
    S = np.zeros((B, H, dv, q.shape[3])) if S0 is None else S0.astype(np.float64).copy()
    o = np.zeros(v.shape)
    for t in range(L):
        S = S * a[:, t, :, None, None] + v[:, t, :, :, None] * k[:, t, :, None, :]
        o[:, t] = scale * (S @ q[:, t, :, :, None])[..., 0]
    return o, S


def linattn_grad(q, k, v, g, scale, dout, S0=None, dlast=None):
    """Gradients of sum(dout o) + sum(dlast S_L): dict of dq, dk, dv, dlog_decay (g's shape), dinitial_state."""
    B, L, H, dv = v.shape
    G, dk = q.shape[2], q.shape[3]
    qh, kh = _per_head(q, H), _per_head(k, H)
    a = np.exp(np.broadcast_to(g, (B, L, H)))
    S = np.zeros((B, H, dv, dk)) if S0 is None else S0.astype(np.float64).copy()
    states = np.zeros((L + 1,) + S.shape)
    states[0] = S
    for t in range(L):
        states[t + 1] = states[t] * a[:, t, :, None, None] + v[:, t, :, :, None] * kh[:, t, :, None, :]
    dS = np.zeros_like(S) if dlast is None else dlast.astype(np.float64).copy()
    dq, dkh, dvh, dg = np.zeros(qh.shape), np.zeros(qh.shape), np.zeros(v.shape), np.zeros((B, L, H))
    for t in range(L - 1, -1, -1):
        do = dout[:, t]
        dq[:, t] = scale * (do[:, :, None, :] @ states[t + 1])[:, :, 0]
        dS = dS + scale * do[..., None] * qh[:, t, :, None, :]
        dvh[:, t] = (dS @ kh[:, t, :, :, None])[..., 0]
        dkh[:, t] = (v[:, t, :, None, :] @ dS)[:, :, 0]
        dg[:, t] = (dS * states[t]).sum((-1, -2)) * a[:, t]
        dS = dS * a[:, t, :, None, None]
    fold = lambda x: x.reshape(B, L, G, H // G, dk).sum(3)  # noqa: E731
    return {"dq": fold(dq), "dk": fold(dkh), "dv": dvh, "dlog_decay": dg if np.ndim(g) == 3 else dg.sum((0, 1)),
            "dinitial_state": dS}


def q4_weights(codes, scales, zeros, group):
    """[n, k] weights of packed codes [n, k / 2] (the low four bits first), scales and zeros [n, k / group]."""
    n = codes.shape[0]
    c = np.stack([codes & 15, codes >> 4], -1).reshape(n, -1, group).astype(np.float64)
    z = 8.0 if zeros is None else zeros.astype(np.float64)[..., None]
    return ((c - z) * scales.astype(np.float64)[..., None]).reshape(n, -1)
