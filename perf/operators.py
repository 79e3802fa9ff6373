"""Cases of the operators around the scan: what is timed, in a plain form and as the library computes it.

The operators are those a block of a recurrent language model needs next to its scan:

  add_norm    residual add, residual scale and norm before a block, and its gradients
  gated_norm  the norm after a block, over groups of channels, with the SiLU gate, and its gradients
  linattn     linear attention with a decay for each head: chunked for prompts, its gradients, and one token's step
  q4          products of few rows with 4-bit weights and group scales

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits, rounded once at the end;
with ``own`` true, it calls the library.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the norm in front of a block while one sequence is decoded: latency only
        {"name": "add_norm one token", "op": "add_norm", "rows": 1, "width": 2560, "x": "bf16", "res": "f32",
         "scale": False, "center": False},
        # the same norm over a training batch: 8 sequences of 2048 tokens, fp32 residual stream
        {"name": "add_norm batch", "op": "add_norm", "rows": 16384, "width": 2560, "x": "bf16", "res": "f32",
         "scale": False, "center": False},
        # its backward, with a learned residual scale for each channel
        {"name": "add_norm batch backward", "op": "add_norm_bwd", "rows": 16384, "width": 2560, "x": "bf16",
         "res": "f32", "scale": True, "center": False},
        # the gated norm after a 5120-channel mixer, over all channels at once, gate first
        {"name": "gated_norm batch", "op": "gated_norm", "rows": 16384, "width": 5120, "groups": 1, "x": "bf16",
         "gate_first": True, "center": False},
        # per-head norm (80 heads of 64) with the gate after it, a ragged number of rows, backward
        {"name": "gated_norm heads backward", "op": "gated_norm_bwd", "rows": 16379, "width": 5120, "groups": 80,
         "x": "bf16", "gate_first": False, "center": False},
        # a prompt batch through a 5120-channel layer with a decay for each token and head
        {"name": "linattn prompts", "op": "linattn", "batch": 8, "seqlen": 2048, "heads": 40, "groups": 40, "dk": 128,
         "dv": 128, "decay": "token", "state": False},
        # one long document, continued from a state, keys shared by four heads, a fixed decay for each head
        {"name": "linattn long", "op": "linattn", "batch": 1, "seqlen": 65537, "heads": 16, "groups": 4, "dk": 64,
         "dv": 128, "decay": "head", "state": True},
        # a training step's gradients on the 5120-channel layer
        {"name": "linattn backward", "op": "linattn_bwd", "batch": 4, "seqlen": 2048, "heads": 40, "groups": 40,
         "dk": 128, "dv": 128, "decay": "token", "state": False},
        # decoding one sequence: 80 heads, latency
        {"name": "linattn step one", "op": "linattn_step", "batch": 1, "heads": 80, "groups": 1, "dk": 128, "dv": 64,
         "decay": "token"},
        # decoding a batch of 64 sequences: the state streams through memory
        {"name": "linattn step batch", "op": "linattn_step", "batch": 64, "heads": 80, "groups": 1, "dk": 128,
         "dv": 64, "decay": "token"},
        # the input projection of one token: 2 * 5120 + 2 * 128 + 80 outputs of 2560 inputs
        {"name": "q4 one row", "op": "q4", "m": 1, "n": 10576, "k": 2560, "group": 128, "x": "bf16", "zeros": False},
        # a projection of 8192 channels to 16384 for a decode batch of 48
        {"name": "q4 batch", "op": "q4", "m": 48, "n": 16384, "k": 8192, "group": 64, "x": "bf16", "zeros": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["add_norm", "add_norm_bwd", "gated_norm", "gated_norm_bwd", "linattn", "linattn_bwd",
                     "linattn_step", "q4"])
    if op in ("add_norm", "add_norm_bwd"):
        width = _log_int(rng, 64, 8192)
        return {"op": op, "rows": _log_int(rng, 1, min(16384, 40_000_000 // width)), "width": width,
                "x": rng.choice(["bf16", "f32"]), "res": rng.choice(["bf16", "f32"]),
                "scale": rng.random() < 0.5, "center": rng.random() < 0.3}
    if op in ("gated_norm", "gated_norm_bwd"):
        groups = rng.choice([1, 1, 2, 8, 40, 80])
        each = _log_int(rng, 32, 256) if groups >= 8 else _log_int(rng, 64, 5120 // groups)
        width = groups * each
        return {"op": op, "rows": _log_int(rng, 1, min(16384, 80_000_000 // width)), "width": width,
                "groups": groups, "x": rng.choice(["bf16", "f32"]), "gate_first": rng.random() < 0.5,
                "center": rng.random() < 0.3}
    if op in ("linattn", "linattn_bwd"):
        dk, dv = rng.choice([(64, 64), (128, 128), (64, 128), (96, 96), (80, 64), (128, 64), (32, 48)])
        seqlen = _log_int(rng, 64, 8192)
        most = (8 * 2048 * 40 if op == "linattn" else 4 * 2048 * 40) // seqlen
        groups = _log_int(rng, 1, min(40, most))
        per = rng.choice([1, 1, 2, 4])
        per = per if groups * per <= min(80, most) else 1
        return {"op": op, "batch": _log_int(rng, 1, max(1, min(16, most // (groups * per)))), "seqlen": seqlen,
                "heads": groups * per, "groups": groups, "dk": dk, "dv": dv, "decay": rng.choice(["token", "head"]),
                "state": rng.random() < 0.5}
    if op == "linattn_step":
        dk, dv = rng.choice([(64, 64), (128, 128), (64, 128), (96, 96), (128, 64), (32, 48)])
        groups = _log_int(rng, 1, 40)
        return {"op": op, "batch": _log_int(rng, 1, 64), "heads": groups * rng.choice([1, 2]), "groups": groups,
                "dk": dk, "dv": dv, "decay": rng.choice(["token", "head"])}
    group = rng.choice([32, 64, 128])
    return {"op": "q4", "m": _log_int(rng, 1, 48), "n": _log_int(rng, 64, 16384), "group": group,
            "k": group * (2 * (_log_int(rng, 256, 8192) // (2 * group)) + 1), "x": rng.choice(["bf16", "f32"]),
            "zeros": rng.random() < 0.5}


# ----------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype="f32", std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(_DT[dtype])


def _uniform(g, shape, lo, hi):
    return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo


def _empty(*shape, dtype="f32"):
    return torch.empty(shape, device="cuda", dtype=_DT[dtype])


def _decay(g, case, lead):
    """Log decays: a step in [1e-3, 0.1] (log-uniform) times a rate in [1, 16] for each head, negative."""
    rate = torch.exp(_uniform(g, (case["heads"],), 0.0, math.log(16.0)))
    if case["decay"] == "head":
        return -rate * 0.02
    step = torch.exp(_uniform(g, (*lead, case["heads"]), math.log(1e-3), math.log(0.1)))
    return -rate * step


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op in ("add_norm", "add_norm_bwd"):
        rows, width = case["rows"], case["width"]
        s["x"] = _normal(g, (rows, width), case["x"])
        s["residual"] = _normal(g, (rows, width), case["res"], 3.0)
        s["weight"] = _uniform(g, (width,), 0.5, 1.5)
        s["bias"] = _normal(g, (width,), std=0.1) if case["center"] else None
        s["scale"] = _uniform(g, (width,), 0.1, 1.0) if case["scale"] else None
        if op == "add_norm":
            s["out"] = _empty(rows, width, dtype=case["x"])
            s["residual_out"] = _empty(rows, width, dtype=case["res"])
        else:
            s["dout"] = _normal(g, (rows, width), case["x"])
            s["dresidual_out"] = _normal(g, (rows, width), case["res"])
    elif op in ("gated_norm", "gated_norm_bwd"):
        rows, width = case["rows"], case["width"]
        s["x"] = _normal(g, (rows, width), case["x"], 2.0)
        s["z"] = _normal(g, (rows, width), case["x"])
        s["weight"] = _uniform(g, (width,), 0.5, 1.5)
        s["bias"] = _normal(g, (width,), std=0.1) if case["center"] else None
        if op == "gated_norm_bwd":
            s["dout"] = _normal(g, (rows, width), case["x"])
    elif op in ("linattn", "linattn_bwd"):
        B, L, H, G, dk, dv = (case[n] for n in ("batch", "seqlen", "heads", "groups", "dk", "dv"))
        s["q"], s["k"] = _normal(g, (B, L, G, dk), "bf16"), _normal(g, (B, L, G, dk), "bf16")
        s["v"] = _normal(g, (B, L, H, dv), "bf16")
        s["log_decay"] = _decay(g, case, (B, L))
        s["state"] = _normal(g, (B, H, dv, dk)) if case["state"] else None
        if op == "linattn":
            s["last_state"] = _empty(B, H, dv, dk)
        else:
            s["dout"] = _normal(g, (B, L, H, dv), "bf16")
            s["dlast_state"] = _normal(g, (B, H, dv, dk)) if case["state"] else None
    elif op == "linattn_step":
        B, H, G, dk, dv = (case[n] for n in ("batch", "heads", "groups", "dk", "dv"))
        s["state"] = _normal(g, (B, H, dv, dk))
        s["q"], s["k"] = _normal(g, (B, G, dk), "bf16"), _normal(g, (B, G, dk), "bf16")
        s["v"] = _normal(g, (B, H, dv), "bf16")
        s["log_decay"] = _decay(g, case, (B,))
        s["out"], s["state_out"] = _empty(B, H, dv, dtype="bf16"), _empty(B, H, dv, dk)
    else:
        m, n, k, group = (case[i] for i in ("m", "n", "k", "group"))
        s["x"] = _normal(g, (m, k), case["x"])
        s["codes"] = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = _uniform(g, (n, k // group), 0.5, 1.5).div_(8.0 * math.sqrt(k)).to(torch.bfloat16)
        s["zeros"] = (torch.randint(5, 11, (n, k // group), generator=g, device="cuda", dtype=torch.uint8)
                      if case["zeros"] else None)
        s["out"] = _empty(m, n, dtype=case["x"])
    return s


# -------------------------------------------------------------- the plain form

_EPS = 1e-5


def _norm_plain(r, weight, bias, center):
    r = r - r.mean(-1, keepdim=True) if center else r
    r = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + _EPS)
    r = r * weight
    return r if bias is None else r + bias


def _norm_grad_plain(dy, r, weight, center):
    """Gradients (dr, dweight rows, dbias rows) of the norm of r."""
    if center:
        r = r - r.mean(-1, keepdim=True)
    rstd = torch.rsqrt(r.square().mean(-1, keepdim=True) + _EPS)
    n = r * rstd
    u = dy * weight
    d = u - n * (u * n).mean(-1, keepdim=True)
    if center:
        d = d - u.mean(-1, keepdim=True)
    return d * rstd, dy * n, dy


def _add_norm_plain(s):
    c = s["case"]
    x, r = s["x"].float(), s["residual"].float()
    r = r + (x if s["scale"] is None else x * s["scale"])
    return (_norm_plain(r, s["weight"], s["bias"], c["center"]).to(_DT[c["x"]]), r.to(_DT[c["res"]]))


def _add_norm_bwd_plain(s):
    c = s["case"]
    d, dw, db = _norm_grad_plain(s["dout"].float(), s["residual"].float(), s["weight"], c["center"])
    d = d + s["dresidual_out"].float()
    g = {"dx": (d if s["scale"] is None else d * s["scale"]).to(_DT[c["x"]]), "dresidual": d.to(_DT[c["res"]]),
         "dweight": dw.sum(0)}
    if s["bias"] is not None:
        g["dbias"] = db.sum(0)
    if s["scale"] is not None:
        g["dscale"] = (d * s["x"].float()).sum(0)
    return g


def _heads(t, groups):
    return t.reshape(*t.shape[:-1], groups, t.shape[-1] // groups)


def _gated_norm_plain(s):
    c, G = s["case"], s["case"]["groups"]
    x, z, w = (_heads(s[n].float(), G) for n in ("x", "z", "weight"))
    b = None if s["bias"] is None else _heads(s["bias"], G)
    gate = z / (1 + torch.exp(-z))
    y = _norm_plain(x * gate, w, b, c["center"]) if c["gate_first"] else _norm_plain(x, w, b, c["center"]) * gate
    return y.flatten(-2).to(_DT[c["x"]])


def _gated_norm_bwd_plain(s):
    c, G = s["case"], s["case"]["groups"]
    dy, x, z, w = (_heads(s[n].float(), G) for n in ("dout", "x", "z", "weight"))
    sig = 1 / (1 + torch.exp(-z))
    gate, dgate = z * sig, sig * (1 + z * (1 - sig))
    if c["gate_first"]:
        d, dw, db = _norm_grad_plain(dy, x * gate, w, c["center"])
        dx, dz = d * gate, d * x * dgate
    else:
        b = None if s["bias"] is None else _heads(s["bias"], G)
        dx, dw, db = _norm_grad_plain(dy * gate, x, w, c["center"])
        dz = dy * _norm_plain(x, w, b, c["center"]) * dgate
    g = {"dx": dx.flatten(-2).to(_DT[c["x"]]), "dz": dz.flatten(-2).to(_DT[c["x"]]), "dweight": dw.sum(0).flatten()}
    if s["bias"] is not None:
        g["dbias"] = db.sum(0).flatten()
    return g


_CHUNK = 64


def _segments(a):
    """exp of the sums of a over (j, i] for every i >= j, and 0 for i < j: [..., T, T]."""
    T = a.shape[-1]
    ones = torch.ones(T, T, dtype=torch.bool, device=a.device)
    x = a.unsqueeze(-1).expand(*a.shape, T).masked_fill(~ones.tril(-1), 0.0).cumsum(-2)
    return torch.exp(x.masked_fill(~ones.tril(), -math.inf))


def _chunked(q, k, v, a, S0):
    """o_t = sum_{s<=t} exp(sum a over (s, t]) (q_t . k_s) v_s + exp(sum a over [0, t]) q_t S0 over [B, H, n, C, .]
    chunks (a: [B, H, n, C], S0: [B, H, dk, dv]).  Returns o and the states at the n + 1 chunk borders."""
    B, H, n, C, dk = q.shape
    cum = a.cumsum(-1)
    D = _segments(a)
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * D, v)
    ends = torch.matmul((k * D[..., -1, :].unsqueeze(-1)).transpose(-1, -2), v)           # [B, H, n, dk, dv]
    ends = torch.cat([S0.unsqueeze(2), ends], 2).flatten(3)
    hops = _segments(torch.nn.functional.pad(cum[..., -1], (1, 0)))                        # [B, H, n + 1, n + 1]
    S = torch.matmul(hops, ends).reshape(B, H, n + 1, dk, v.shape[-1])
    return o + torch.matmul(q * torch.exp(cum).unsqueeze(-1), S[:, :, :n]), S


def _cut(t, L):
    """[B, L, H, .] as [B, H, n, C, .], the last chunk filled up with zeros."""
    t = torch.nn.functional.pad(t, (0, 0, 0, 0, 0, -L % _CHUNK)).transpose(1, 2)
    return t.reshape(*t.shape[:2], -1, _CHUNK, t.shape[-1])


def _joined(t, L, dtype):
    return t.flatten(2, 3)[:, :, :L].transpose(1, 2).to(dtype).contiguous()


def _linattn_inputs(s):
    c = s["case"]
    B, L, H, per = c["batch"], c["seqlen"], c["heads"], c["heads"] // c["groups"]
    q = _cut(s["q"].float().repeat_interleave(per, 2) * c["dk"] ** -0.5, L)
    k = _cut(s["k"].float().repeat_interleave(per, 2), L)
    v = _cut(s["v"].float(), L)
    a = s["log_decay"] if s["log_decay"].dim() == 3 else s["log_decay"].expand(B, L, H)
    a = _cut(a.unsqueeze(-1), L).squeeze(-1)
    S0 = s["state"] if s["state"] is not None else torch.zeros(B, H, c["dv"], c["dk"], device="cuda")
    return q, k, v, a, S0.transpose(-1, -2)


def _linattn_plain(s):
    q, k, v, a, S0 = _linattn_inputs(s)
    o, S = _chunked(q, k, v, a, S0)
    return _joined(o, s["case"]["seqlen"], torch.bfloat16), S[:, :, -1].transpose(-1, -2).contiguous()


def _back(t):
    """[B, H, n, C, .] in reverse order of time."""
    return t.flip(2, 3)


def _linattn_bwd_plain(s):
    c = s["case"]
    L, per, dk = c["seqlen"], c["heads"] // c["groups"], c["dk"]
    q, k, v, a, S0 = _linattn_inputs(s)
    do = _cut(s["dout"].float(), L)
    dS = torch.zeros_like(S0) if s["dlast_state"] is None else s["dlast_state"].transpose(-1, -2)
    dq, St = _chunked(do, v, k, a, S0.transpose(-1, -2))                                    # states as [dv, dk]
    # going back, the step from t + 1 to t decays by a of t + 1
    flat = _back(a.unsqueeze(-1)).flatten(2)
    ra = torch.nn.functional.pad(flat[..., :-1], (1, 0)).reshape(a.shape)
    dkk, Rt = _chunked(_back(v), _back(do), _back(q), ra, dS.transpose(-1, -2))             # [dv, dk]
    dvv, R = _chunked(_back(k), _back(q), _back(do), ra, dS)
    dkk, dvv = _back(dkk), _back(dvv)
    # <S, dS> after the last step of each chunk: the gradient that is still to arrive there has not met the
    # decay of the next chunk's first step yet
    decay_in = torch.cat([torch.exp(a[:, :, 1:, 0]), torch.ones_like(a[:, :, :1, 0])], 2)
    border = (St[:, :, 1:] * Rt.flip(2)[:, :, 1:]).sum((-1, -2)) * decay_in
    e = (q * dq).sum(-1) - (k * dkk).sum(-1)
    da = (e.flip(-1).cumsum(-1).flip(-1) + border.unsqueeze(-1)).flatten(2)[:, :, :L].transpose(1, 2)
    dq, dkk = _joined(dq * dk ** -0.5, L, torch.float32), _joined(dkk, L, torch.float32)
    g = {"dq": dq.unflatten(2, (-1, per)).sum(3).to(torch.bfloat16),
         "dk": dkk.unflatten(2, (-1, per)).sum(3).to(torch.bfloat16), "dv": _joined(dvv, L, torch.bfloat16),
         "dlog_decay": da.contiguous() if c["decay"] == "token" else da.sum((0, 1))}
    if s["state"] is not None:
        g["dinitial_state"] = (R[:, :, -1] * torch.exp(a[:, :, 0, 0])[..., None, None]).transpose(-1, -2).contiguous()
    return g


def _linattn_step_plain(s):
    c = s["case"]
    per = c["heads"] // c["groups"]
    q, k = (s[n].float().repeat_interleave(per, 1).unsqueeze(-2) for n in ("q", "k"))
    S = s["state"] * torch.exp(s["log_decay"])[..., None, None] + s["v"].float().unsqueeze(-1) * k
    return ((S * q).sum(-1) * c["dk"] ** -0.5).to(torch.bfloat16), S


def _q4_weights(s, dtype):
    c = s["case"]
    w = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).to(dtype).reshape(c["n"], -1, c["group"])
    z = 8 if s["zeros"] is None else s["zeros"].to(dtype).unsqueeze(-1)
    return ((w - z) * s["scales"].to(dtype).unsqueeze(-1)).reshape(c["n"], c["k"])


def _q4_plain(s):
    return torch.matmul(s["x"].float(), _q4_weights(s, torch.float32).t()).to(_DT[s["case"]["x"]])


_PLAIN = {"add_norm": _add_norm_plain, "add_norm_bwd": _add_norm_bwd_plain, "gated_norm": _gated_norm_plain,
          "gated_norm_bwd": _gated_norm_bwd_plain, "linattn": _linattn_plain, "linattn_bwd": _linattn_bwd_plain,
          "linattn_step": _linattn_step_plain, "q4": _q4_plain}


# ----------------------------------------------------------- the library's form

def _own(s):
    import sequence_scan_amd as ssm
    c, op = s["case"], s["case"]["op"]
    if op == "add_norm":
        return ssm.ssm_add_norm_fwd(s["x"], s["residual"], s["weight"], s["bias"], s["scale"], eps=_EPS,
                                    center=c["center"], out=s["out"], residual_out=s["residual_out"])
    if op == "add_norm_bwd":
        return ssm.ssm_add_norm_bwd(s["dout"], s["residual"], s["weight"], s["dresidual_out"], x=s["x"],
                                    scale=s["scale"], want_bias=s["bias"] is not None, eps=_EPS, center=c["center"])
    if op == "gated_norm":
        return ssm.ssm_gated_norm_fwd(s["x"], s["z"], s["weight"], s["bias"], ngroups=c["groups"],
                                      gate_first=c["gate_first"], eps=_EPS, center=c["center"])
    if op == "gated_norm_bwd":
        return ssm.ssm_gated_norm_bwd(s["dout"], s["x"], s["z"], s["weight"], s["bias"], ngroups=c["groups"],
                                      gate_first=c["gate_first"], eps=_EPS, center=c["center"])
    if op == "linattn":
        out = ssm.ssm_linattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], initial_state=s["state"],
                                  last_state=s["last_state"])
        return out, s["last_state"]
    if op == "linattn_bwd":
        return ssm.ssm_linattn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["dout"], initial_state=s["state"],
                                   dlast_state=s["dlast_state"], want_dinitial_state=s["state"] is not None)
    if op == "linattn_step":
        out = ssm.ssm_linattn_state_update(s["state"], s["q"], s["k"], s["v"], s["log_decay"], out=s["out"],
                                           state_out=s["state_out"])
        return out, s["state_out"]
    return ssm.ssm_q4_matvec(s["x"], s["codes"], s["scales"], s["zeros"], out=s["out"])


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- the work

def work(case):
    op = case["op"]
    if op in ("add_norm", "add_norm_bwd"):
        e, width = case["rows"] * case["width"], case["width"]
        x, r = _SIZE[case["x"]], _SIZE[case["res"]]
        if op == "add_norm":   # x, residual in; out, residual out
            return {"bytes": 2 * e * (x + r) + 4 * width, "flops": 6 * e}
        n = 2 * x + 3 * r if not case["scale"] else 3 * x + 3 * r   # dout, r, its gradient (, x) in; dx, dresidual out
        return {"bytes": n * e + 12 * width, "flops": 12 * e}
    if op in ("gated_norm", "gated_norm_bwd"):
        e, x = case["rows"] * case["width"], _SIZE[case["x"]]
        return {"bytes": (3 if op == "gated_norm" else 5) * e * x + 8 * case["width"],
                "flops": (10 if op == "gated_norm" else 24) * e}
    if op in ("linattn", "linattn_bwd"):
        t = case["batch"] * case["seqlen"]
        qk, v = t * case["groups"] * case["dk"] * 2, t * case["heads"] * case["dv"] * 2
        d = 4 * (t if case["decay"] == "token" else 1) * case["heads"]
        S = 4 * case["batch"] * case["heads"] * case["dk"] * case["dv"]
        f = t * case["heads"] * case["dk"] * case["dv"]
        if op == "linattn":     # q, k, v, decays (, state) in; out and the last state out; update and readout
            return {"bytes": 2 * qk + 2 * v + d + (2 if case["state"] else 1) * S, "flops": 4 * f}
        return {"bytes": 4 * qk + 3 * v + 2 * d + (3 if case["state"] else 0) * S, "flops": 10 * f}
    if op == "linattn_step":
        S = case["batch"] * case["heads"] * case["dk"] * case["dv"]
        io = 2 * case["batch"] * (2 * case["groups"] * case["dk"] + 2 * case["heads"] * case["dv"])
        return {"bytes": 8 * S + io + 4 * case["heads"], "flops": 5 * S}
    m, n, k, x = case["m"], case["n"], case["k"], _SIZE[case["x"]]
    return {"bytes": n * k // 2 + n * (k // case["group"]) * (3 if case["zeros"] else 2) + m * (n + k) * x,
            "flops": 2 * m * n * k}


# ------------------------------------------- the definitions, step by step, in 64 bits

def _exact_norm(r, w, b, center, dy=None):
    """The norm of the rows of r in 64 bits, or with dy its vector-Jacobian product and the parameters' gradients."""
    if center:
        r = r - r.sum(-1, keepdim=True) / r.shape[-1]
    std = torch.sqrt((r * r).sum(-1, keepdim=True) / r.shape[-1] + _EPS)
    if dy is None:
        y = w * r / std
        return y if b is None else y + b
    gr = dy * w / std
    gr = gr - r * (gr * r).sum(-1, keepdim=True) / (r.shape[-1] * std * std)
    if center:
        gr = gr - gr.sum(-1, keepdim=True) / r.shape[-1]
    return gr, (dy * r / std).sum(0), dy.sum(0)


def _exact_add_norm(s, c, d):
    r = d["residual"] + d["x"] * (1.0 if d["scale"] is None else d["scale"])
    return _exact_norm(r, d["weight"], d["bias"], c["center"]), r


def _exact_add_norm_bwd(s, c, d):
    g, dw, db = _exact_norm(d["residual"], d["weight"], None, c["center"], d["dout"])
    g = g + d["dresidual_out"]
    out = {"dx": g if d["scale"] is None else d["scale"] * g, "dresidual": g, "dweight": dw}
    if d["bias"] is not None:
        out["dbias"] = db
    if d["scale"] is not None:
        out["dscale"] = (d["x"] * g).sum(0)
    return out


def _exact_gated(s, c, d):
    backward = "dout" in d
    parts = []
    each = c["width"] // c["groups"]
    for g in range(c["groups"]):
        at = slice(g * each, (g + 1) * each)
        x, z, w = d["x"][:, at], d["z"][:, at], d["weight"][at]
        b = None if d["bias"] is None else d["bias"][at]
        sig = torch.sigmoid(z)
        if not backward:
            y = (_exact_norm(x * z * sig, w, b, c["center"]) if c["gate_first"]
                 else _exact_norm(x, w, b, c["center"]) * z * sig)
            parts.append({"y": y})
            continue
        dy, slope = d["dout"][:, at], sig + z * sig * (1 - sig)
        if c["gate_first"]:
            dr, dw, db = _exact_norm(x * z * sig, w, b, c["center"], dy)
            parts.append({"dx": dr * z * sig, "dz": dr * x * slope, "dweight": dw, "dbias": db})
        else:
            dr, dw, db = _exact_norm(x, w, b, c["center"], dy * z * sig)
            parts.append({"dx": dr, "dz": dy * slope * _exact_norm(x, w, b, c["center"]), "dweight": dw, "dbias": db})
    out = {n: torch.cat([p[n] for p in parts], -1) for n in parts[0]}
    if not backward:
        return out["y"]
    if d["bias"] is None:
        del out["dbias"]
    return out


def _exact_linattn(s, c, d):
    """The recurrence itself, one step at a time, forward and (for gradients) back."""
    B, L, H, dk, dv = (c[n] for n in ("batch", "seqlen", "heads", "dk", "dv"))
    per = H // c["groups"]
    q, k = (d[n].repeat_interleave(per, 2) for n in ("q", "k"))
    v, scale = d["v"], 1.0 / math.sqrt(dk)
    a = torch.exp(d["log_decay"].expand(B, L, H))
    S = torch.zeros(B, H, dv, dk, device="cuda", dtype=torch.float64) if d["state"] is None else d["state"].clone()
    o, dq = torch.empty_like(v), torch.empty_like(q)
    backward = "dout" in d
    for t in range(L):
        S *= a[:, t, :, None, None]
        S += v[:, t].unsqueeze(-1) * k[:, t].unsqueeze(-2)
        if backward:
            dq[:, t] = torch.matmul(d["dout"][:, t].unsqueeze(-2), S).squeeze(-2) * scale
        else:
            o[:, t] = torch.matmul(S, q[:, t].unsqueeze(-1)).squeeze(-1) * scale
    if not backward:
        return o, S
    do = d["dout"]
    R = torch.zeros_like(S) if d["dlast_state"] is None else d["dlast_state"].clone()
    end = (S * R).sum((-1, -2))
    dkk, dvv = torch.empty_like(q), torch.empty_like(v)
    for t in range(L - 1, -1, -1):
        R += do[:, t].unsqueeze(-1) * (q[:, t] * scale).unsqueeze(-2)
        dkk[:, t] = torch.matmul(v[:, t].unsqueeze(-2), R).squeeze(-2)
        dvv[:, t] = torch.matmul(R, k[:, t].unsqueeze(-1)).squeeze(-1)
        R *= a[:, t, :, None, None]
    da = ((q * dq).sum(-1) - (k * dkk).sum(-1)).flip(1).cumsum(1).flip(1) + end.unsqueeze(1)
    out = {"dq": dq.unflatten(2, (-1, per)).sum(3), "dk": dkk.unflatten(2, (-1, per)).sum(3), "dv": dvv,
           "dlog_decay": da if c["decay"] == "token" else da.sum((0, 1))}
    if d["state"] is not None:
        out["dinitial_state"] = R
    return out


def _exact_step(s, c, d):
    per = c["heads"] // c["groups"]
    q, k = (d[n].repeat_interleave(per, 1) for n in ("q", "k"))
    S = torch.exp(d["log_decay"])[..., None, None] * d["state"] + d["v"].unsqueeze(-1) * k.unsqueeze(-2)
    return torch.matmul(S, q.unsqueeze(-1)).squeeze(-1) / math.sqrt(c["dk"]), S


def _exact_q4(s, c, d):
    w = torch.empty(c["n"], c["k"], device="cuda", dtype=torch.float64)
    w[:, 0::2], w[:, 1::2] = s["codes"] % 16, s["codes"] // 16
    each = c["group"]
    zero = torch.full_like(d["scales"], 8.0) if s["zeros"] is None else s["zeros"].double()
    w -= zero.repeat_interleave(each, 1)
    w *= d["scales"].repeat_interleave(each, 1)
    return torch.matmul(d["x"], w.t())


_EXACT = {"add_norm": _exact_add_norm, "add_norm_bwd": _exact_add_norm_bwd, "gated_norm": _exact_gated,
          "gated_norm_bwd": _exact_gated, "linattn": _exact_linattn, "linattn_bwd": _exact_linattn,
          "linattn_step": _exact_step, "q4": _exact_q4}


def exact(case, seed):
    s = prepare(case, seed)
    d = {n: t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t for n, t in s.items()}
    return _EXACT[case["op"]](s, case, d)
