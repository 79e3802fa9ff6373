"""Python binding of the block operators (include/ssmblock.h): norms, linear
attention with a decay for each head, and products with 4-bit weights.

As in the package's other calls: argument marshalling only, tensors are passed
to the C ABI as device pointers on the current stream, and there is no
fallback.  Functions carry the C names.
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import SSM_BF16, SSM_F32, _check, _dtype_code, _load, ssm_plan

SSM_NORM_CENTER = 1
SSM_NORM_GATE_LAST = 2
SSM_LINATTN_FIXED_DECAY = 1

_vp, _i64, _int, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_ARGS = {
    "ssm_add_norm_fwd": [_vp, _i64, _vp, _vp, _vp, _vp, _f32, _f32, _int, _vp, _vp, _i64, _i64, _int, _int, _int, _vp],
    "ssm_add_norm_bwd": [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _f32, _f32, _int, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                         _int, _int, _int, _vp],
    "ssm_gated_norm_fwd": [_vp, _i64, _vp, _i64, _vp, _vp, _f32, _int, _vp, _i64, _i64, _i64, _int, _int, _vp],
    "ssm_gated_norm_bwd": [_vp, _vp, _i64, _vp, _i64, _vp, _vp, _f32, _int, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                           _int, _int, _vp],
    "ssm_linattn_plan_query": [_i64] * 5 + [ctypes.POINTER(ssm_plan)],
    "ssm_linattn_fwd": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _int, _f32, _vp, _vp, _vp] + [_i64] * 6 +
                       [_int, _int, _vp, ctypes.POINTER(ssm_plan)],
    "ssm_linattn_bwd": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _int, _f32] + [_vp] * 8 + [_i64] * 6 +
                       [_int, _int, _vp],
    "ssm_q4_matvec": [_vp, _i64] + [_vp] * 5 + [_i64] * 4 + [_int, _int, _int, _vp],
    "ssm_q4_quantize": [_vp] * 4 + [_i64] * 3 + [_int, _int, _vp],
    "ssm_workspace": [_vp, _i64],
    "ssm_workspace_bytes": [],
    "ssm_linattn_state_update": [_vp] * 6 + [_int, _f32, _vp] + [_i64] * 5 + [_int, _int, _vp],
}
_fns: dict = {}
_code: dict = {}            # torch dtype -> the C ABI's code
_F32 = _U8 = _empty = _raw_stream = _device = None


def _fn(name: str):
    """The C function, with its argument types set on first use."""
    f = _fns.get(name)
    if f is None:
        _start()
        f = getattr(_load(), name)
        f.argtypes, f.restype = _ARGS[name], _i64 if name == "ssm_workspace_bytes" else ctypes.c_int
        _fns[name] = f
    return f


def _start():
    """What the wrappers use of PyTorch, looked up once: a decode step makes dozens of
    these calls, and each microsecond of a wrapper counts."""
    global _F32, _U8, _empty, _raw_stream, _device
    import torch
    _F32, _U8, _empty = torch.float32, torch.uint8, torch.empty
    _code.update({torch.float32: SSM_F32, torch.bfloat16: SSM_BF16})
    # the public form builds a Stream object first, 2.7 us against 0.1 us
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda i: torch.cuda.current_stream(i).cuda_stream)
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(stream, dev: int):
    """The HIP stream to run on: the given one, or the current one, of the tensors' device
    (its index), which has to be the current device."""
    if dev < 0:
        raise ValueError("tensors must be on the GPU")
    if dev != _device():
        raise ValueError(f"tensors are on cuda:{dev}, but the current device is cuda:{_device()}")
    if stream is None:
        return _raw_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"tensors are on cuda:{dev}, but the stream is on cuda:{stream.device_index}")
    return stream.cuda_stream


def _bad(t, name: str, shape, dtype, dev: int):
    """Raise for the first thing that is not as wanted."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is None:
        _dtype_code(t)
    elif t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected {'cuda:%d' % dev if dev >= 0 else 'the CPU'}")
    raise ValueError(f"{name} must be contiguous")


def _want(t, name: str, shape, dtype, dev: int):
    """The pointer of a contiguous tensor of this shape, dtype (None: float32 or
    bfloat16) and device index, or of no tensor.  The C ABI trusts the sizes it is given,
    so every tensor is checked before its pointer is passed (that the device is a GPU:
    ``_on``)."""
    if t is None:
        return None
    if (t.shape != shape or (t.dtype not in _code if dtype is None else t.dtype is not dtype) or t.get_device() != dev
            or not t.is_contiguous()):
        _bad(t, name, shape, dtype, dev)
    return t.data_ptr()


def _rows(t, name: str, shape, dtype, dev: int, inner: int = 1):
    """(pointer, row stride) of a tensor whose last ``inner`` dimensions are
    contiguous and whose leading ones are evenly spaced rows, such as a slice of a
    packed projection's last dimension."""
    if t is None:
        return None, 0
    if t.shape != shape or (t.dtype not in _code if dtype is None else t.dtype is not dtype) or t.get_device() != dev:
        _bad(t, name, shape, dtype, dev)
    if t.is_contiguous():
        return t.data_ptr(), shape[-1] if inner == 1 else shape[-1] * shape[-2]
    lead, step = t.dim() - inner, 1
    for d in range(t.dim() - 1, lead - 1, -1):
        if t.shape[d] != 1 and t.stride(d) != step:
            raise ValueError(f"{name} must be contiguous in its last {inner} dimension(s)")
        step *= t.shape[d]
    row, expect = None, None
    for d in range(lead - 1, -1, -1):
        if t.shape[d] == 1:
            continue
        if row is None:
            row = t.stride(d)
        elif t.stride(d) != expect:
            raise ValueError(f"{name} must have evenly spaced rows")
        expect = t.stride(d) * t.shape[d]
    return t.data_ptr(), step if row is None else row


def _kind(dtype) -> int:
    """The C ABI's code of an output's dtype."""
    if dtype not in _code:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    return _code[dtype]


def _new(shape, dtype, like):
    return _empty(shape, dtype=dtype, device=like.device)


def ssm_add_norm_fwd(x, residual=None, weight=None, bias=None, scale=None, alpha: float = 1.0, eps: float = 1e-5,
                     center: bool = False, out=None, residual_out=None, out_dtype=None, stream=None):
    """Residual add and norm before a block: r = alpha * residual + scale * x and
    out = norm(r) * weight + bias over the last dimension (root mean square, or with
    ``center`` mean and variance).  x, residual: [..., width] (float32 or bfloat16
    each; x may be a slice of a packed tensor); weight, bias, scale: [width] float32.
    ``residual_out`` (residual's dtype, or float32 without one) may be ``residual``.
    Returns (out, residual_out)."""
    call = _fn("ssm_add_norm_fwd")
    dev, shape = x.get_device(), x.shape
    width = shape[-1]
    rows = x.numel() // width if width else 0
    xp, xs = _rows(x, "x", shape, None, dev)
    rp = _want(residual, "residual", shape, None, dev)
    if out is None:
        out = _new(shape, out_dtype or x.dtype, x)
    if residual_out is None:
        residual_out = _new(shape, _F32 if residual is None else residual.dtype, x)
    cols = (width,)
    _check(call(
        xp, xs, rp, _want(weight, "weight", cols, _F32, dev), _want(bias, "bias", cols, _F32, dev),
        _want(scale, "scale", cols, _F32, dev), alpha, eps, SSM_NORM_CENTER if center else 0,
        _want(out, "out", shape, None, dev),
        _want(residual_out, "residual_out", shape, None if residual is None else residual.dtype, dev), rows, width,
        _code[x.dtype], _code[residual_out.dtype], _code[out.dtype], _on(stream, dev)))
    return out, residual_out


def ssm_add_norm_bwd(dout, r, weight=None, dresidual_out=None, x=None, scale=None, alpha: float = 1.0,
                     eps: float = 1e-5, center: bool = False, want_weight: bool = True, want_bias: bool = False,
                     want_scale: Optional[bool] = None, dx_dtype=None, stream=None):
    """Gradients of ``ssm_add_norm_fwd`` from r (its ``residual_out``), dout [..., width]
    and, optionally, the gradient that arrives at the residual stream.  Returns a dict
    with dx (``dx_dtype``, or x's or dout's dtype), dresidual (r's dtype) and, as asked,
    dweight, dbias and dscale (wanted by default where ``scale`` and ``x`` are given)."""
    call = _fn("ssm_add_norm_bwd")
    dev, shape = dout.get_device(), dout.shape
    width = shape[-1]
    rows = dout.numel() // width if width else 0
    if want_scale is None:
        want_scale = scale is not None and x is not None
    if want_scale and x is None:
        raise ValueError("dscale needs x")
    xdt = x.dtype if x is not None else (dx_dtype or dout.dtype)
    if dx_dtype is not None and dx_dtype != xdt:
        raise TypeError("dx has x's dtype")
    _kind(xdt)
    xp, xs = _rows(x, "x", shape, None, dev) if want_scale else (None, width)
    cols = (width,)
    g = {"dx": _new(shape, xdt, dout), "dresidual": _new(shape, r.dtype, dout)}
    if want_weight:
        g["dweight"] = _new(cols, _F32, dout)
    if want_bias:
        g["dbias"] = _new(cols, _F32, dout)
    if want_scale:
        g["dscale"] = _new(cols, _F32, dout)
    ptr = {k: v.data_ptr() for k, v in g.items()}
    key = ("add", rows, width, r.dtype, dout.dtype, want_weight, want_bias, want_scale, dev)
    _with_workspace(call, key, dout, stream, (
        _want(dout, "dout", shape, None, dev), _want(r, "r", shape, None, dev), _want(weight, "weight", cols, _F32, dev),
        _want(dresidual_out, "dresidual_out", shape, r.dtype, dev), xp, xs, _want(scale, "scale", cols, _F32, dev),
        alpha, eps, SSM_NORM_CENTER if center else 0, ptr["dx"], ptr["dresidual"], ptr.get("dweight"),
        ptr.get("dbias"), ptr.get("dscale"), rows, width, _code[g["dx"].dtype], _code[r.dtype], _code[dout.dtype],
        _on(stream, dev)))
    return g


_wanted: dict = {}          # sizes and kind of a call -> bytes of workspace that it wants


def ssm_workspace(memory, nbytes: int):
    """Offer device memory (a pointer, or None) for this thread's next call that needs a
    workspace (include/ssmblock.h).  The calls of this module do so themselves, except on a
    stream of the caller's.  An offer is the caller's to withdraw where the call that it was for
    raises before the library is entered (a tensor of the wrong shape or type)."""
    _check(_fn("ssm_workspace")(memory, nbytes))


def ssm_workspace_bytes() -> int:
    """Bytes of workspace that this thread's last call wanted."""
    return _fn("ssm_workspace_bytes")()


def _with_workspace(call, key, like, stream, args):
    """The call, with memory of PyTorch's for its workspace: 2 us in place of the 28 us that
    the library's own allocation takes.  What a call of these sizes wants is known
    after the first one.  A caller's own stream is not PyTorch's current one: there
    the library allocates."""
    n = _wanted.get(key)
    if n and stream is None:
        t = _empty((n,), dtype=_U8, device=like.device)
        try:
            _fn("ssm_workspace")(t.data_ptr(), n)
            status = call(*args)
        except BaseException:
            # the library may not have been entered (an argument that ctypes cannot
            # convert): the offer must not outlive t, for a later call to write into
            _fn("ssm_workspace")(None, 0)
            raise
    else:
        status = call(*args)
    if n is None and status == 0:
        if len(_wanted) >= 4096:
            _wanted.clear()
        _wanted[key] = _fn("ssm_workspace_bytes")()
    _check(status)


def _norm_flags(center, gate_first):
    return (SSM_NORM_CENTER if center else 0) | (0 if gate_first else SSM_NORM_GATE_LAST)


def ssm_gated_norm_fwd(x, z=None, weight=None, bias=None, ngroups: int = 1, gate_first: bool = True,
                       eps: float = 1e-5, center: bool = False, out=None, out_dtype=None, stream=None):
    """The norm after a block's mixer over ``ngroups`` groups of the last dimension's
    channels, gated by SiLU(z): norm(x * silu(z)) * weight + bias with ``gate_first``,
    (norm(x) * weight + bias) * silu(z) without.  x, z: [..., width] of one dtype (each
    may be a slice of a packed tensor); weight, bias: [width] float32.  Returns out."""
    call = _fn("ssm_gated_norm_fwd")
    dev, shape = x.get_device(), x.shape
    width = shape[-1]
    rows = x.numel() // width if width else 0
    xp, xs = _rows(x, "x", shape, None, dev)
    zp, zs = _rows(z, "z", shape, x.dtype, dev)
    if out is None:
        out = _new(shape, out_dtype or x.dtype, x)
    cols = (width,)
    _check(call(
        xp, xs, zp, zs, _want(weight, "weight", cols, _F32, dev), _want(bias, "bias", cols, _F32, dev), eps,
        _norm_flags(center, gate_first), _want(out, "out", shape, None, dev), rows, width, ngroups, _code[x.dtype],
        _code[out.dtype], _on(stream, dev)))
    return out


def ssm_gated_norm_bwd(dout, x, z=None, weight=None, bias=None, ngroups: int = 1, gate_first: bool = True,
                       eps: float = 1e-5, center: bool = False, want_weight: bool = True,
                       want_bias: Optional[bool] = None, stream=None):
    """Gradients of ``ssm_gated_norm_fwd`` from its inputs and dout.  Returns a dict with
    dx, dz (where z is given), and dweight and dbias as asked (dbias by default where
    ``bias`` is given)."""
    call = _fn("ssm_gated_norm_bwd")
    dev, shape = x.get_device(), x.shape
    width = shape[-1]
    rows = x.numel() // width if width else 0
    if want_bias is None:
        want_bias = bias is not None
    xp, xs = _rows(x, "x", shape, None, dev)
    zp, zs = _rows(z, "z", shape, x.dtype, dev)
    cols = (width,)
    g = {"dx": _new(shape, x.dtype, dout)}
    if z is not None:
        g["dz"] = _new(shape, x.dtype, dout)
    if want_weight:
        g["dweight"] = _new(cols, _F32, dout)
    if want_bias:
        g["dbias"] = _new(cols, _F32, dout)
    ptr = {k: v.data_ptr() for k, v in g.items()}
    key = ("gate", rows, width, ngroups, x.dtype, dout.dtype, want_weight, want_bias, dev)
    _with_workspace(call, key, dout, stream, (
        _want(dout, "dout", shape, None, dev), xp, xs, zp, zs, _want(weight, "weight", cols, _F32, dev),
        _want(bias, "bias", cols, _F32, dev), eps, _norm_flags(center, gate_first), ptr["dx"], ptr.get("dz"),
        ptr.get("dweight"), ptr.get("dbias"), rows, width, ngroups, _code[x.dtype], _code[dout.dtype],
        _on(stream, dev)))
    return g


def ssm_linattn_plan_query(batch: int, seqlen: int, nheads: int, dk: int = 128, dv: int = 128) -> dict:
    """The time chunks ``ssm_linattn_fwd`` picks for these sizes."""
    call = _fn("ssm_linattn_plan_query")
    p = ssm_plan()
    _check(call(batch, seqlen, nheads, dk, dv, ctypes.byref(p)))
    return {"chunk_len": p.chunk_len, "n_chunks": p.n_chunks}


def _la_shapes(q, v, tokens: int):
    if q.dim() != tokens + 2 or v.dim() != tokens + 2:
        lead = "batch, seqlen" if tokens == 2 else "batch"
        raise ValueError(f"q must be [{lead}, ngroups, dk] and v [{lead}, nheads, dv]")
    return q.shape[-2], q.shape[-1], v.shape[-2], v.shape[-1]


def _la_decay(g, lead, nheads, dev):
    """(pointer, flags) of the log decay: [*lead, nheads], or [nheads] for a fixed one."""
    fixed = g.dim() == 1
    return (_want(g, "log_decay", (nheads,) if fixed else (*lead, nheads), _F32, dev),
            SSM_LINATTN_FIXED_DECAY if fixed else 0)


def ssm_linattn_fwd(q, k, v, log_decay, scale: Optional[float] = None, initial_state=None, out=None, last_state=None,
                    out_dtype=None, stream=None, plan: Optional[dict] = None):
    """Linear attention with a decay for each head (see include/ssmblock.h): q, k
    [batch, seqlen, ngroups, dk] and v [batch, seqlen, nheads, dv] bfloat16 (each may be a
    slice of a packed tensor); log_decay [batch, seqlen, nheads] or [nheads] float32; scale
    1 / sqrt(dk) by default; states [batch, nheads, dv, dk] float32 (last_state is written
    where given, and may be initial_state).  Returns out [batch, seqlen, nheads, dv].
    ``plan`` = {"chunk_len": ..} forces the time chunks."""
    call = _fn("ssm_linattn_fwd")
    G, dk, H, dv = _la_shapes(q, v, 2)
    B, L, dev = q.shape[0], q.shape[1], q.get_device()
    qs, vs, st = (B, L, G, dk), (B, L, H, dv), (B, H, dv, dk)
    qp, qr = _rows(q, "q", qs, None, dev, 2)
    kp, kr = _rows(k, "k", qs, q.dtype, dev, 2)
    vp, vr = _rows(v, "v", vs, q.dtype, dev, 2)
    gp, flags = _la_decay(log_decay, (B, L), H, dev)
    if out is None:
        out = _new(vs, out_dtype or v.dtype, q)
    p = None
    if plan is not None:
        p = ssm_plan()
        p.chunk_len = int(plan["chunk_len"])
        p = ctypes.byref(p)
    in_place = initial_state is not None and initial_state is last_state
    key = ("la", B, L, H, dk, dv, 0 if plan is None else plan["chunk_len"], in_place, dev)
    _with_workspace(call, key, q, stream, (
        qp, qr, kp, kr, vp, vr, gp, flags, dk ** -0.5 if scale is None else scale,
        _want(initial_state, "initial_state", st, _F32, dev), _want(out, "out", vs, None, dev),
        _want(last_state, "last_state", st, _F32, dev), B, L, H, G, dk, dv, _code[q.dtype], _code[out.dtype],
        _on(stream, dev), p))
    return out


def ssm_linattn_bwd(q, k, v, log_decay, dout, scale: Optional[float] = None, initial_state=None, dlast_state=None,
                    want_dinitial_state: bool = False, grad_dtype=None, stream=None):
    """Gradients of ``ssm_linattn_fwd`` from its inputs, dout [batch, seqlen, nheads, dv]
    (bfloat16) and, optionally, the gradient of the last state.  Returns a dict with dq, dk,
    dv (``grad_dtype``, or q's dtype), dlog_decay (float32, of log_decay's shape) and, as
    asked, dinitial_state."""
    call = _fn("ssm_linattn_bwd")
    G, dk, H, dv = _la_shapes(q, v, 2)
    B, L, dev = q.shape[0], q.shape[1], q.get_device()
    qs, vs, st = (B, L, G, dk), (B, L, H, dv), (B, H, dv, dk)
    gdt = grad_dtype or q.dtype
    _kind(gdt)
    qp, qr = _rows(q, "q", qs, None, dev, 2)
    kp, kr = _rows(k, "k", qs, q.dtype, dev, 2)
    vp, vr = _rows(v, "v", vs, q.dtype, dev, 2)
    gp, flags = _la_decay(log_decay, (B, L), H, dev)
    g = {"dq": _new(qs, gdt, q), "dk": _new(qs, gdt, q), "dv": _new(vs, gdt, q),
         "dlog_decay": _new(log_decay.shape, _F32, q)}
    if want_dinitial_state:
        g["dinitial_state"] = _new(st, _F32, q)
    key = ("la_bwd", B, L, H, G, dk, dv, flags, initial_state is None, dlast_state is None, dev)
    _with_workspace(call, key, q, stream, (
        qp, qr, kp, kr, vp, vr, gp, flags, dk ** -0.5 if scale is None else scale,
        _want(initial_state, "initial_state", st, _F32, dev), _want(dout, "dout", vs, q.dtype, dev),
        _want(dlast_state, "dlast_state", st, _F32, dev), g["dq"].data_ptr(), g["dk"].data_ptr(), g["dv"].data_ptr(),
        g["dlog_decay"].data_ptr(), g["dinitial_state"].data_ptr() if want_dinitial_state else None, B, L, H, G, dk,
        dv, _code[q.dtype], _code[g["dq"].dtype], _on(stream, dev)))
    return g


def ssm_linattn_state_update(state, q, k, v, log_decay, scale: Optional[float] = None, out=None, state_out=None,
                             out_dtype=None, stream=None):
    """One token of linear attention: state [batch, nheads, dv, dk] float32 moves on (in
    place, or into ``state_out``, which keeps ``state``).  q, k: [batch, ngroups, dk]; v:
    [batch, nheads, dv] (float32 or bfloat16); log_decay: [batch, nheads] or [nheads]
    float32.  Returns out [batch, nheads, dv]."""
    call = _fn("ssm_linattn_state_update")
    G, dk, H, dv = _la_shapes(q, v, 1)
    B, dev = q.shape[0], q.get_device()
    qs, vs, st = (B, G, dk), (B, H, dv), (B, H, dv, dk)
    gp, flags = _la_decay(log_decay, (B,), H, dev)
    if out is None:
        out = _new(vs, out_dtype or v.dtype, q)
    sp = _want(state, "state", st, _F32, dev)
    _check(call(
        sp, sp if state_out is None else _want(state_out, "state_out", st, _F32, dev), _want(q, "q", qs, None, dev),
        _want(k, "k", qs, q.dtype, dev), _want(v, "v", vs, q.dtype, dev), gp, flags,
        dk ** -0.5 if scale is None else scale, _want(out, "out", vs, None, dev), B, H, G, dk, dv, _code[q.dtype],
        _code[out.dtype], _on(stream, dev)))
    return out


def ssm_q4_quantize(w, group: int = 128, scale_dtype=None, stream=None):
    """4-bit form of a weight matrix w [n, k] (float32 or bfloat16), k a multiple of
    ``group`` (32, 64 or 128): codes [n, k // 2] uint8 (two per byte, the lower k in the low
    bits), scales [n, k // group] (``scale_dtype``, float32 by default) and zeros
    [n, k // group] uint8, with w close to (code - zero) * scale (see include/ssmblock.h)."""
    call = _fn("ssm_q4_quantize")
    if w.dim() != 2:
        raise ValueError("w must be [n, k]")
    n, k = w.shape
    if group not in (32, 64, 128) or k % group:
        raise ValueError(f"group must be 32, 64 or 128 and divide k={k}, got {group}")
    dev, ng = w.get_device(), k // group
    codes, zeros = _new((n, k // 2), _U8, w), _new((n, ng), _U8, w)
    scales = _new((n, ng), scale_dtype or _F32, w)
    _kind(scales.dtype)
    _check(call(_want(w, "w", w.shape, None, dev), codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(), n, k,
                                  group, _code[w.dtype], _code[scales.dtype], _on(stream, dev)))
    return codes, scales, zeros


def ssm_q4_matvec(x, codes, scales, zeros=None, bias=None, out=None, out_dtype=None, stream=None):
    """x W^T + bias for x [..., k] (float32 or bfloat16; rows may be slices of a packed
    tensor) and 4-bit weights: codes [n, k // 2] uint8, scales [n, k // group] (float32 or
    bfloat16), zeros [n, k // group] uint8 (None: 8), bias [n] float32.  Returns out
    [..., n] (allocated if None, dtype ``out_dtype`` or x's)."""
    call = _fn("ssm_q4_matvec")
    dev = x.get_device()
    if codes.dim() != 2 or scales.dim() != 2 or x.dim() < 1:
        raise ValueError("x must be [..., k], codes [n, k // 2] and scales [n, k // group]")
    n, k = codes.shape[0], 2 * codes.shape[1]
    ng = scales.shape[1]
    group = k // ng if ng else 128
    if x.shape[-1] != k or group * ng != k:
        raise ValueError(f"x has {x.shape[-1]} columns, codes {k} and scales {ng} groups")
    shape = (*x.shape[:-1], n)
    if out is None:
        out = _new(shape, out_dtype or x.dtype, x)
    xp, xr = _rows(x, "x", x.shape, None, dev)
    m = x.numel() // k if k else out.numel() // n if n else 0
    _with_workspace(call, ("q4", m, n, k, group, x.dtype, dev), x, stream, (
        xp, xr, _want(codes, "codes", (n, k // 2), _U8, dev), _want(scales, "scales", (n, ng), None, dev),
        _want(zeros, "zeros", (n, ng), _U8, dev), _want(bias, "bias", (n,), _F32, dev),
        _want(out, "out", shape, None, dev), m, n, k, group, _code[x.dtype], _code[scales.dtype], _code[out.dtype],
        _on(stream, dev)))
    return out
