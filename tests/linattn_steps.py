"""Linear attention and its gradients step by step in 64 bits on the GPU, in elementary torch
operations (not a test module): for sequences longer than block_ref.py's numpy loops and their
stored states allow.  The decay's gradient is formed another way than there,
dg_t = <S_L, dS_L> + sum over u >= t of (q_u . dq_u - k_u . dk_u)."""
from __future__ import annotations

import torch


def forward(q, k, v, g, scale, S0=None):
    """o and the last state; q, k [B, L, G, dk], v [B, L, H, dv], g [B, L, H] or [H], any dtype."""
    B, L, H, dv = v.shape
    q, k = (x.double().repeat_interleave(H // x.shape[2], 2) for x in (q, k))
    v, a = v.double(), torch.exp(g.double()).expand(B, L, H)
    S = torch.zeros(B, H, dv, q.shape[3], device=v.device, dtype=torch.float64) if S0 is None else S0.double().clone()
    o = torch.empty_like(v)
    for t in range(L):
        S.mul_(a[:, t, :, None, None]).add_(v[:, t].unsqueeze(-1) * k[:, t].unsqueeze(-2))
        o[:, t] = (S * q[:, t].unsqueeze(-2)).sum(-1) * scale
    return o, S


def gradients(q, k, v, g, scale, dout, S0=None, dlast=None):
    """dq, dk, dv, dlog_decay (of every step, [B, L, H]) and dinitial_state."""
    B, L, H, dv = v.shape
    G, dk = q.shape[2:]
    q, k = (x.double().repeat_interleave(H // G, 2) for x in (q, k))
    v, dout, a = v.double(), dout.double(), torch.exp(g.double()).expand(B, L, H)
    S = torch.zeros(B, H, dv, dk, device=v.device, dtype=torch.float64) if S0 is None else S0.double().clone()
    dq, dkk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(L):
        S.mul_(a[:, t, :, None, None]).add_(v[:, t].unsqueeze(-1) * k[:, t].unsqueeze(-2))
        dq[:, t] = (dout[:, t].unsqueeze(-1) * S).sum(-2) * scale
    R = torch.zeros_like(S) if dlast is None else dlast.double().clone()
    end = (S * R).sum((-1, -2))
    for t in range(L - 1, -1, -1):
        R.add_(dout[:, t].unsqueeze(-1) * (q[:, t] * scale).unsqueeze(-2))
        dkk[:, t] = (v[:, t].unsqueeze(-1) * R).sum(-2)
        dvv[:, t] = (R * k[:, t].unsqueeze(-2)).sum(-1)
        R.mul_(a[:, t, :, None, None])
    dg = ((q * dq).sum(-1) - (k * dkk).sum(-1)).flip(1).cumsum(1).flip(1) + end.unsqueeze(1)
    fold = lambda x: x.unflatten(2, (G, H // G)).sum(3)  # noqa: E731
    return {"dq": fold(dq), "dk": fold(dkk), "dv": dvv, "dlog_decay": dg, "dinitial_state": R}
