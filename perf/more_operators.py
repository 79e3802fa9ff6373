"""Cases of the operators that train a model of recurrent layers: what is timed, in a plain form and as the library
computes it.

  gscan         a gated linear recurrence for each channel: prompts, a training step (forward and gradients), and
                one token's step
  xent          softmax cross entropy of rows against a large vocabulary, from the rows and the vocabulary's weights,
                forward and (train) with its gradients
  distill       the same for a teacher's top logits: their softmax against the student's over the whole vocabulary

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits, rounded once at the end;
with ``own`` true, it calls the library.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_SEGMENT = 32       # steps between two states that a training forward keeps for the gradients


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # decoding one sequence through a 2560-channel recurrent layer: latency only
        {"name": "gscan step one", "op": "gscan_step", "batch": 1, "width": 2560, "dtype": "bf16", "gate": True,
         "rate": True, "lerp": False},
        # decoding 256 sequences through an 8192-channel layer
        {"name": "gscan step batch", "op": "gscan_step", "batch": 256, "width": 8192, "dtype": "bf16", "gate": True,
         "rate": True, "lerp": False},
        # a prompt batch through a 5120-channel layer
        {"name": "gscan prompts", "op": "gscan", "batch": 8, "seqlen": 2048, "width": 5120, "dtype": "bf16",
         "gate": True, "rate": True, "lerp": False, "state": False},
        # one long document, continued from a state, an odd length, forget gate and its complement
        {"name": "gscan long", "op": "gscan", "batch": 1, "seqlen": 65537, "width": 2560, "dtype": "bf16",
         "gate": False, "rate": False, "lerp": True, "state": True},
        # a training step's forward and gradients on the 5120-channel layer
        {"name": "gscan train", "op": "gscan_train", "batch": 4, "seqlen": 2048, "width": 5120, "dtype": "bf16",
         "gate": True, "rate": True, "lerp": False, "state": False},
        # the same in fp32 for a small model with a ragged length and width
        {"name": "gscan train fp32", "op": "gscan_train", "batch": 3, "seqlen": 1021, "width": 1537, "dtype": "f32",
         "gate": True, "rate": True, "lerp": True, "state": True},
        # how probable one next token was: the vocabulary's weights stream through memory
        {"name": "xent one row", "op": "xent", "rows": 1, "width": 2560, "vocab": 50280},
        # perplexity of a ragged batch of held-out text
        {"name": "xent evaluation", "op": "xent", "rows": 2039, "width": 1536, "vocab": 50280},
        # the loss of a training step and its gradients: 4 sequences of 2048 tokens
        {"name": "xent train", "op": "xent_train", "rows": 8192, "width": 2560, "vocab": 50280},
        # distillation into a smaller model from 64 teacher logits for each token, with gradients
        {"name": "distill train", "op": "distill_train", "rows": 4096, "width": 1536, "vocab": 50280, "top": 64,
         "temperature": 2.0},
        # distillation's loss alone on a small ragged batch with an odd vocabulary
        {"name": "distill evaluation", "op": "distill", "rows": 333, "width": 768, "vocab": 32003, "top": 17,
         "temperature": 1.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["gscan", "gscan", "gscan_train", "gscan_train", "gscan_step", "xent", "xent_train", "distill",
                     "distill_train"])
    if op.startswith("gscan"):
        case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "gate": rng.random() < 0.7,
                "rate": rng.random() < 0.6, "lerp": rng.random() < 0.5}
        if op == "gscan_step":
            return {**case, "batch": _log_int(rng, 1, 256), "width": _log_int(rng, 64, 8192)}
        most = (40_000_000 if op == "gscan" else 20_000_000) // (1 if case["dtype"] == "bf16" else 2)
        width = _log_int(rng, 64, 8192)
        seqlen = _log_int(rng, 2, min(65536, most // width))
        return {**case, "batch": _log_int(rng, 1, min(64, most // (width * seqlen))), "seqlen": seqlen,
                "width": width, "state": rng.random() < 0.5}
    most = 500_000_000_000 if op.endswith("train") else 200_000_000_000
    width = 8 * _log_int(rng, 32, 512)
    vocab = _log_int(rng, 256, 65536)
    case = {"op": op, "rows": _log_int(rng, 1, min(8192, most // (width * vocab))), "width": width, "vocab": vocab}
    if op.startswith("distill"):
        case["top"] = _log_int(rng, 1, 128)
        case["temperature"] = rng.choice([1.0, 2.0, 4.0])
    return case


# ----------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype="f32", std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(_DT[dtype])


def _empty(*shape, dtype="f32"):
    return torch.empty(shape, device="cuda", dtype=_DT[dtype])


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op.startswith("gscan"):
        B, D, dt = case["batch"], case["width"], case["dtype"]
        lead = (B,) if op == "gscan_step" else (B, case["seqlen"])
        s["x"] = _normal(g, (*lead, D), dt)
        # forget gates start open: with a rate its sigmoid scales the decay, without one it is the decay
        s["r"] = _normal(g, (*lead, D), dt, 1.0, 0.0 if case["rate"] else 2.0)
        s["i"] = _normal(g, (*lead, D), dt) if case["gate"] else None
        s["rate"] = torch.exp(torch.rand((D,), generator=g, device="cuda") * math.log(100.0)) * 0.008 \
            if case["rate"] else None
        if op == "gscan_step":
            s["state"], s["state_out"], s["out"] = _normal(g, (B, D)), _empty(B, D), _empty(B, D, dtype=dt)
            return s
        s["state"] = _normal(g, (B, D)) if case["state"] else None
        s["last_state"] = _empty(B, D)
        if op == "gscan_train":
            s["states"] = _empty(B, -(-case["seqlen"] // _SEGMENT), D)
            s["dout"] = _normal(g, (B, case["seqlen"], D), dt)
            s["dlast_state"] = _normal(g, (B, D)) if case["state"] else None
        return s
    T, D, V = case["rows"], case["width"], case["vocab"]
    s["x"] = _normal(g, (T, D), "bf16")
    s["weight"] = _normal(g, (V, D), "bf16", 2.0 / math.sqrt(D))
    if op.startswith("xent"):
        # words by rank: few are frequent; and some rows (a prompt's, padding) have no target
        s["target"] = (torch.rand((T,), generator=g, device="cuda").pow(4) * V).long().clamp_(max=V - 1)
        if T > 8:
            s["target"][torch.rand((T,), generator=g, device="cuda") < 0.05] = -100
    else:
        K = min(case["top"], max(1, V // 2))
        first = torch.randint(0, V, (T, 1), generator=g, device="cuda")
        step = torch.randint(1, max(2, V // K), (T, 1), generator=g, device="cuda")
        s["index"] = (first + step * torch.arange(K, device="cuda")) % V        # distinct in a row
        s["logit"] = _normal(g, (T, K), std=3.0).sort(-1, descending=True).values
    if op.endswith("train"):
        s["dloss"] = torch.full((T,), 1.0 / T, device="cuda")
    return s


# -------------------------------------------------------------- the plain form

def _sigmoid(t):
    return 1 / (1 + torch.exp(-t))


def _coefficients(s):
    """The recurrence's decay a, its logarithm, input coefficient m and gated input u in 32 bits."""
    c = s["case"]
    x, r = s["x"].float(), s["r"].float()
    sr = _sigmoid(r)
    la = -s["rate"] * sr if c["rate"] else -torch.log1p(torch.exp(-r))
    a = torch.exp(la) if c["rate"] else sr
    m = -torch.expm1(la) if c["lerp"] else torch.sqrt(-torch.expm1(2 * la))
    si = _sigmoid(s["i"].float()) if c["gate"] else None
    return a, m, x if si is None else x * si, sr, si


def _scan(a, b, first, dim):
    """h_t = a_t h_{t-1} + b_t along dim by doubling: after each round an entry covers twice as many steps."""
    a, h = a.clone(), b.clone()
    n, k = h.shape[dim], 1
    if first is not None:
        h.select(dim, 0).add_(a.select(dim, 0) * first)
    while k < n:
        late, early = slice(k, n), slice(0, n - k)
        at = (slice(None),) * dim
        h[(*at, late)] += a[(*at, late)] * h[(*at, early)]
        a[(*at, late)] = a[(*at, late)] * a[(*at, early)]
        k *= 2
    return h


def _gscan_plain(s):
    a, m, u, _, _ = _coefficients(s)
    h = _scan(a, m * u, s["state"], 1)
    return h.to(_DT[s["case"]["dtype"]]), h[:, -1].contiguous()


def _gscan_train_plain(s):
    c, dt = s["case"], _DT[s["case"]["dtype"]]
    a, m, u, sr, si = _coefficients(s)
    h = _scan(a, m * u, s["state"], 1)
    before = torch.zeros_like(h[:, :1]) if s["state"] is None else s["state"].unsqueeze(1)
    before = torch.cat([before, h[:, :-1]], 1)
    # back in time: a step's gradient meets the decay of the step behind it
    late = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1).flip(1)
    g = _scan(late, s["dout"].float().flip(1), s["dlast_state"], 1).flip(1)
    slope = -a if c["lerp"] else -a * a / m                        # of m by the decay's logarithm
    dla = g * (a * before + u * slope)
    du = g * m
    out = {"out": h.to(dt), "last_state": h[:, -1].contiguous(),
           "dx": (du if si is None else du * si).to(dt),
           "dr": (dla * (1 - sr) * (-s["rate"] * sr if c["rate"] else 1)).to(dt)}
    if si is not None:
        out["di"] = (du * s["x"].float() * si * (1 - si)).to(dt)
    if c["rate"]:
        out["drate"] = -(dla * sr).sum((0, 1))
    if s["state"] is not None:
        out["dinitial_state"] = a[:, 0] * g[:, 0]
    return out


def _gscan_step_plain(s):
    a, m, u, _, _ = _coefficients(s)
    h = a * s["state"] + m * u
    return h.to(_DT[s["case"]["dtype"]]), h


def _softmax_parts(s, temperature):
    """Logits (over the temperature) and their log sum of exponentials in 32 bits."""
    z = torch.matmul(s["x"].float(), s["weight"].float().t()) / temperature
    top = z.max(-1, keepdim=True).values
    return z, (top + torch.log(torch.exp(z - top).sum(-1, keepdim=True))).squeeze(-1)


def _head_grads(s, dz):
    return {"dx": torch.matmul(dz, s["weight"].float()).to(torch.bfloat16),
            "dweight": torch.matmul(dz.t(), s["x"].float()).to(torch.bfloat16)}


def _xent_plain(s):
    z, lse = _softmax_parts(s, 1.0)
    has = s["target"] >= 0
    at = s["target"].clamp(min=0).unsqueeze(-1)
    loss = torch.where(has, lse - z.gather(-1, at).squeeze(-1), 0.0)
    if s["case"]["op"] == "xent":
        return loss, lse
    p = torch.exp(z - lse.unsqueeze(-1))
    p.scatter_add_(-1, at, -torch.ones_like(at, dtype=torch.float32))
    return {"loss": loss, "lse": lse, **_head_grads(s, p * (has * s["dloss"]).unsqueeze(-1))}


def _distill_plain(s):
    t = s["case"]["temperature"]
    z, lse = _softmax_parts(s, t)
    q = torch.exp(s["logit"] / t - (s["logit"] / t).max(-1, keepdim=True).values)
    q = q / q.sum(-1, keepdim=True)
    logp = z.gather(-1, s["index"]) - lse.unsqueeze(-1)
    loss = t * t * (q * (torch.log(q) - logp)).sum(-1)
    if s["case"]["op"] == "distill":
        return loss, lse
    p = torch.exp(z - lse.unsqueeze(-1))
    p.scatter_add_(-1, s["index"], -q)
    return {"loss": loss, "lse": lse, **_head_grads(s, p * (t * s["dloss"]).unsqueeze(-1))}


_PLAIN = {"gscan": _gscan_plain, "gscan_train": _gscan_train_plain, "gscan_step": _gscan_step_plain,
          "xent": _xent_plain, "xent_train": _xent_plain, "distill": _distill_plain, "distill_train": _distill_plain}


# ----------------------------------------------------------- the library's form

def _own(s):
    import sequence_scan_amd as ssm
    c, op = s["case"], s["case"]["op"]
    if op == "gscan_step":
        out = ssm.ssm_gscan_update(s["state"], s["x"], s["r"], s["i"], s["rate"], lerp=c["lerp"], out=s["out"],
                                   state_out=s["state_out"])
        return out, s["state_out"]
    if op == "gscan":
        out = ssm.ssm_gscan_fwd(s["x"], s["r"], s["i"], s["rate"], lerp=c["lerp"], initial_state=s["state"],
                                last_state=s["last_state"])
        return out, s["last_state"]
    if op == "gscan_train":
        out = ssm.ssm_gscan_fwd(s["x"], s["r"], s["i"], s["rate"], lerp=c["lerp"], initial_state=s["state"],
                                last_state=s["last_state"], states=s["states"])
        g = ssm.ssm_gscan_bwd(s["x"], s["r"], s["i"], s["rate"], s["dout"], s["states"], lerp=c["lerp"],
                              dlast_state=s["dlast_state"], want_dinitial_state=s["state"] is not None)
        return {"out": out, "last_state": s["last_state"], **g}
    if op.startswith("xent"):
        loss, lse = ssm.ssm_xent_fwd(s["x"], s["weight"], s["target"])
        if op == "xent":
            return loss, lse
        return {"loss": loss, "lse": lse, **ssm.ssm_xent_bwd(s["dloss"], s["x"], s["weight"], s["target"], lse)}
    t = c["temperature"]
    loss, lse, logits = ssm.ssm_distill_fwd(s["x"], s["weight"], s["index"], s["logit"], temperature=t)
    if op == "distill":
        return loss, lse
    return {"loss": loss, "lse": lse, **ssm.ssm_distill_bwd(s["dloss"], s["x"], s["weight"], s["index"], s["logit"], lse,
                                                            logits, temperature=t)}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- the work

def work(case):
    op = case["op"]
    if op.startswith("gscan"):
        e = case["batch"] * case["width"] * case.get("seqlen", 1)
        n, size = 3 if case["gate"] else 2, _SIZE[case["dtype"]]
        state, rate = 4 * case["batch"] * case["width"], 4 * case["width"] if case["rate"] else 0
        if op == "gscan_step":          # inputs, state in; out, state out
            return {"bytes": (n + 1) * e * size + 2 * state + rate, "flops": 12 * e}
        if op == "gscan":
            return {"bytes": (n + 1) * e * size + (2 if case["state"] else 1) * state + rate, "flops": 12 * e}
        # inputs and dout in; out and the inputs' gradients out
        return {"bytes": 2 * (n + 1) * e * size + (4 if case["state"] else 1) * state + 2 * rate, "flops": 40 * e}
    T, D, V = case["rows"], case["width"], case["vocab"]
    io = 2 * (T * D + V * D) + 8 * T + (12 * T * case["top"] if op.startswith("distill") else 8 * T)
    if not op.endswith("train"):
        return {"bytes": io, "flops": 2 * T * V * D}
    return {"bytes": io + 2 * (T * D + V * D) + 4 * T, "flops": 6 * T * V * D}


# ------------------------------------------- the definitions, step by step, in 64 bits

def _exact_gscan(s, c, d):
    """The recurrence itself, one step at a time, forward and (for gradients) back."""
    op = c["op"]
    sr = torch.sigmoid(d["r"])
    if c["rate"]:
        a = torch.exp(-d["rate"] * sr)
        rest = -torch.expm1(-d["rate"] * sr)                    # 1 - a
    else:
        a, rest = sr, torch.sigmoid(-d["r"])
    m = rest if c["lerp"] else torch.sqrt(rest * (1 + a))       # 1 - a^2 = (1 - a)(1 + a)
    u = d["x"] * torch.sigmoid(d["i"]) if c["gate"] else d["x"]
    if op == "gscan_step":
        h = a * d["state"] + m * u
        return h, h
    B, L, D = d["x"].shape
    b = m * u
    h = torch.zeros(B, D, device="cuda", dtype=torch.float64) if d["state"] is None else d["state"].clone()
    out = torch.empty_like(b)
    before = torch.empty_like(b) if op == "gscan_train" else None
    for t in range(L):
        if before is not None:
            before[:, t] = h
        h = torch.addcmul(b[:, t], a[:, t], h, out=out[:, t])
    last = out[:, -1].clone()
    if op == "gscan":
        return out, last
    g = torch.empty_like(b)
    arriving = torch.zeros_like(last) if d["dlast_state"] is None else d["dlast_state"]
    for t in range(L - 1, -1, -1):
        torch.add(d["dout"][:, t], arriving, out=g[:, t])
        arriving = a[:, t] * g[:, t]
    by_decay = before * g                                       # of the decay itself, then through m
    by_m = u * g
    dm = -torch.ones_like(a) if c["lerp"] else -a / m
    da = by_decay + by_m * dm
    out_g = {"out": out, "last_state": last}
    if c["gate"]:
        si = torch.sigmoid(d["i"])
        out_g["dx"] = m * g * si
    else:
        out_g["dx"] = m * g
    if c["rate"]:
        out_g["dr"] = -da * a * d["rate"] * sr * torch.sigmoid(-d["r"])
    else:
        out_g["dr"] = da * sr * torch.sigmoid(-d["r"])
    if c["gate"]:
        out_g["di"] = m * g * d["x"] * si * torch.sigmoid(-d["i"])
    if c["rate"]:
        out_g["drate"] = -(da * a * sr).sum((0, 1))
    if d["state"] is not None:
        out_g["dinitial_state"] = arriving
    return out_g


def _exact_head(s, c, d):
    t = c.get("temperature", 1.0)
    logits = (d["x"] @ d["weight"].t()).div_(t)
    lse = torch.logsumexp(logits, -1)
    T = c["rows"]
    row = torch.arange(T, device="cuda")
    if c["op"].startswith("xent"):
        kept = torch.nonzero(s["target"] >= 0).squeeze(-1)
        loss = torch.zeros(T, device="cuda", dtype=torch.float64)
        loss[kept] = lse[kept] - logits[kept, s["target"][kept]]
        if c["op"] == "xent":
            return loss, lse
        dz = torch.zeros_like(logits)
        dz[kept] = torch.softmax(logits[kept], -1)
        dz[kept, s["target"][kept]] -= 1
        dz *= d["dloss"].unsqueeze(-1)
    else:
        logq = torch.log_softmax(d["logit"] / t, -1)
        mine = logits[row.unsqueeze(-1), s["index"]]
        loss = t ** 2 * (torch.exp(logq) * (logq - mine + lse.unsqueeze(-1))).sum(-1)
        if c["op"] == "distill":
            return loss, lse
        dz = torch.softmax(logits, -1)
        dz[row.unsqueeze(-1), s["index"]] -= torch.exp(logq)
        dz *= (t * d["dloss"]).unsqueeze(-1)
    del logits
    return {"loss": loss, "lse": lse, "dx": dz @ d["weight"], "dweight": dz.t() @ d["x"]}


def exact(case, seed):
    s = prepare(case, seed)
    d = {n: t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t for n, t in s.items()}
    return (_exact_gscan if case["op"].startswith("gscan") else _exact_head)(s, case, d)
