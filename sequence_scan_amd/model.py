"""Python binding of the model operators (include/ssmmodel.h): a gated linear recurrence,
and cross entropy and distillation against a large vocabulary.

As in ``block``: argument marshalling only, tensors are passed to the C ABI as device
pointers on the current stream, and there is no fallback.  Functions carry the C names.
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import _check, block
from .block import _fn, _kind, _new, _on, _rows, _want, _with_workspace

SSM_GSCAN_LERP = 1
SSM_GSCAN_SEGMENT = 32

_vp, _i64, _int, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
block._ARGS.update({
    "ssm_gscan_fwd": [_vp, _i64] * 3 + [_vp, _int] + [_vp] * 4 + [_i64] * 3 + [_int, _int, _vp],
    "ssm_gscan_bwd": [_vp, _i64] * 3 + [_vp, _int] + [_vp] * 8 + [_i64] * 3 + [_int, _int, _vp],
    "ssm_gscan_update": [_vp, _vp] + [_vp, _i64] * 3 + [_vp, _int, _vp] + [_i64] * 2 + [_int, _int, _vp],
    "ssm_xent_fwd": [_vp, _i64] * 2 + [_vp, _f32, _f32, _vp, _vp] + [_i64] * 3 + [_int, _vp],
    "ssm_xent_bwd": [_vp] + [_vp, _i64] * 2 + [_vp, _f32, _f32, _vp, _vp, _vp] + [_i64] * 3 + [_int, _vp],
    "ssm_distill_fwd": [_vp, _i64] * 2 + [_vp, _vp, _f32, _f32, _vp, _vp, _vp] + [_i64] * 4 + [_int, _vp],
    "ssm_distill_bwd": [_vp] + [_vp, _i64] * 2 + [_vp, _vp, _f32, _f32, _vp, _vp, _vp, _vp] + [_i64] * 4 + [_int, _vp],
})


def _missing(name: str):
    # (of the tensors that sizes and types are taken from; the C ABI names the others)
    return ValueError(f"{name} is required")


def _gates(x, r, i, rate, dims: int):
    """What the recurrence's calls share: sizes, and the arguments up to rate."""
    if x is None:
        raise _missing("x")
    if x.dim() != dims:
        raise ValueError("x must be [batch, seqlen, width]" if dims == 3 else "x must be [batch, width]")
    dev, shape = x.get_device(), x.shape
    xp, xr = _rows(x, "x", shape, None, dev)
    rp, rr = _rows(r, "r", shape, x.dtype, dev)
    ip, ir = _rows(i, "i", shape, x.dtype, dev)
    return dev, shape, (xp, xr, rp, rr, ip, ir, _want(rate, "rate", shape[-1:], block._F32, dev))


def _out(out, out_dtype, x, shape, dev):
    """The output, a new one if none is given, its pointer and the C ABI's code of its dtype."""
    if out is None:
        dtype = out_dtype or x.dtype
        code = _kind(dtype)
        out = _new(shape, dtype, x)
        return out, out.data_ptr(), code
    return out, _want(out, "out", shape, None, dev), block._code[out.dtype]


def ssm_gscan_fwd(x, r, i=None, rate=None, lerp: bool = False, initial_state=None, out=None, last_state=None,
                  states=None, out_dtype=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t for each channel, with
    a = exp(-rate sigmoid(r)), or sigmoid(r) without a rate, and m = sqrt(1 - a^2), or 1 - a
    with ``lerp`` (see include/ssmmodel.h).  x, r, i (optional): [batch, seqlen, width] of
    one dtype, float32 or bfloat16 (each may be a slice of a packed tensor); rate: [width]
    float32; states [batch, width] float32 (``last_state`` is written where given, and may
    be ``initial_state``).  ``states`` [batch, ceil(seqlen / SSM_GSCAN_SEGMENT), width]
    float32, where given, receives the states that ``ssm_gscan_bwd`` needs.  Returns out
    [batch, seqlen, width]."""
    call = _fn("ssm_gscan_fwd")
    dev, shape, args = _gates(x, r, i, rate, 3)
    B, L, D = shape
    out, op, code = _out(out, out_dtype, x, shape, dev)
    st, f32 = (B, D), block._F32
    _with_workspace(call, ("gscan", B, L, D, dev), x, stream, (
        *args, SSM_GSCAN_LERP if lerp else 0, _want(initial_state, "initial_state", st, f32, dev), op,
        _want(last_state, "last_state", st, f32, dev),
        _want(states, "states", (B, -(-L // SSM_GSCAN_SEGMENT), D), f32, dev), B, L, D, block._code[x.dtype], code,
        _on(stream, dev)))
    return out


def ssm_gscan_bwd(x, r, i, rate, dout, states, lerp: bool = False, dlast_state=None, want_rate: Optional[bool] = None,
                  want_dinitial_state: bool = False, stream=None):
    """Gradients of ``ssm_gscan_fwd`` from its inputs, the ``states`` that it stored, dout
    [batch, seqlen, width] and, optionally, the gradient of the last state.  Returns a dict
    with dx, dr, di (where i is given), drate (where rate is, unless ``want_rate`` is
    false) and, as asked, dinitial_state."""
    call = _fn("ssm_gscan_bwd")
    dev, shape, args = _gates(x, r, i, rate, 3)
    if dout is None:
        raise _missing("dout")
    B, L, D = shape
    f32 = block._F32
    if want_rate is None:
        want_rate = rate is not None
    g = {"dx": _new(shape, x.dtype, x), "dr": _new(shape, x.dtype, x)}
    if i is not None:
        g["di"] = _new(shape, x.dtype, x)
    if want_rate:
        g["drate"] = _new((D,), f32, x)
    if want_dinitial_state:
        g["dinitial_state"] = _new((B, D), f32, x)
    ptr = {k: v.data_ptr() for k, v in g.items()}
    _with_workspace(call, ("gscan_bwd", B, L, D, want_rate, dev), x, stream, (
        *args, SSM_GSCAN_LERP if lerp else 0,
        _want(states, "states", (B, -(-L // SSM_GSCAN_SEGMENT), D), f32, dev), _want(dout, "dout", shape, None, dev),
        _want(dlast_state, "dlast_state", (B, D), f32, dev), ptr["dx"], ptr["dr"], ptr.get("di"), ptr.get("drate"),
        ptr.get("dinitial_state"), B, L, D, block._code[x.dtype], block._code[dout.dtype], _on(stream, dev)))
    return g


def ssm_gscan_update(state, x, r, i=None, rate=None, lerp: bool = False, out=None, state_out=None, out_dtype=None,
                     stream=None):
    """One token of the recurrence: state [batch, width] float32 moves on (in place, or into
    ``state_out``, which keeps ``state``).  x, r, i: [batch, width].  Returns out [batch, width]."""
    call = _fn("ssm_gscan_update")
    dev, shape, args = _gates(x, r, i, rate, 2)
    B, D = shape
    out, op, code = _out(out, out_dtype, x, shape, dev)
    sp = _want(state, "state", shape, block._F32, dev)
    _check(call(sp, sp if state_out is None else _want(state_out, "state_out", shape, block._F32, dev), *args,
                SSM_GSCAN_LERP if lerp else 0, op, B, D, block._code[x.dtype], code, _on(stream, dev)))
    return out


def _int64():
    import torch
    return torch.int64


def _head(x, weight):
    """Sizes, and the arguments x to w_row, of a loss over a vocabulary: x [..., width]."""
    if x is None or weight is None:
        raise _missing("x" if x is None else "weight")
    if x.dim() < 1 or weight.dim() != 2:
        raise ValueError("x must be [..., width] and weight [vocab, width]")
    V, D = weight.shape
    if x.shape[-1] != D:
        raise ValueError(f"x has {x.shape[-1]} columns, weight {D}")
    dev, lead = x.get_device(), x.shape[:-1]
    xp, xr = _rows(x, "x", x.shape, None, dev)
    wp, wr = _rows(weight, "weight", weight.shape, x.dtype, dev)
    T = 1
    for n in lead:
        T *= n
    return dev, lead, T, D, V, (xp, xr, wp, wr)


def _head_grads(x, weight, want_x, want_weight):
    g = {}
    if want_x:
        g["dx"] = _new(x.shape, x.dtype, x)
    if want_weight:
        g["dweight"] = _new(weight.shape, x.dtype, x)
    return g, [g[n].data_ptr() if n in g else None for n in ("dx", "dweight")]


def ssm_xent_fwd(x, weight, target, scale: float = 1.0, z_loss: float = 0.0, stream=None):
    """Softmax cross entropy of rows x [..., width] (bfloat16; rows may be slices of a packed
    tensor) against a vocabulary's weights [vocab, width] (bfloat16), without storing the
    logits scale * x weight^T: target [...] int64, negative for none (loss 0).  ``z_loss``
    adds z_loss * lse^2.  Returns (loss, lse), [...] float32 each, for each row: a mean
    over the rows with a target is the caller's."""
    call = _fn("ssm_xent_fwd")
    dev, lead, T, D, V, args = _head(x, weight)
    f32 = block._F32
    loss = _new(lead, f32, x)
    lse = _new(lead, f32, loss)
    _with_workspace(call, ("xent", T, D, V, dev), x, stream, (
        *args, _want(target, "target", lead, _int64(), dev), scale, z_loss, loss.data_ptr(), lse.data_ptr(), T, D, V,
        block._code[x.dtype], _on(stream, dev)))
    return loss, lse


def ssm_xent_bwd(dloss, x, weight, target, lse, scale: float = 1.0, z_loss: float = 0.0, want_x: bool = True,
                 want_weight: bool = True, stream=None):
    """Gradients of ``ssm_xent_fwd`` for dloss [...] float32, what arrives at each row's loss
    (1 / rows for a mean), and the forward's lse.  Returns a dict with dx and dweight
    (bfloat16), as asked."""
    call = _fn("ssm_xent_bwd")
    dev, lead, T, D, V, args = _head(x, weight)
    f32 = block._F32
    g, ptrs = _head_grads(x, weight, want_x, want_weight)
    _with_workspace(call, ("xent_bwd", T, D, V, want_x, want_weight, dev), x, stream, (
        _want(dloss, "dloss", lead, f32, dev), *args, _want(target, "target", lead, _int64(), dev), scale, z_loss,
        _want(lse, "lse", lead, f32, dev), *ptrs, T, D, V, block._code[x.dtype], _on(stream, dev)))
    return g


def _tops(index, lead):
    if index is None:
        raise _missing("index")
    if index.dim() != len(lead) + 1:
        raise ValueError("index must be [..., top], with x's leading dimensions")
    return index.shape[-1], (*lead, index.shape[-1])


def ssm_distill_fwd(x, weight, index, teacher, temperature: float = 1.0, scale: float = 1.0, stream=None):
    """Distillation from a teacher's top logits: temperature^2 times the divergence of the
    softmax of scale * x weight^T / temperature over the whole vocabulary from that of the
    teacher's logits / temperature over their own [..., top] (float32) at the places
    ``index`` [..., top] (int64; negative for none).  x and weight as for ``ssm_xent_fwd``.
    Returns (loss [...], lse [...], logits [..., top]) float32: the last two are for
    ``ssm_distill_bwd``."""
    call = _fn("ssm_distill_fwd")
    dev, lead, T, D, V, args = _head(x, weight)
    K, tops = _tops(index, lead)
    f32 = block._F32
    loss, logits = _new(lead, f32, x), _new(tops, f32, x)
    lse = _new(lead, f32, loss)
    _with_workspace(call, ("distill", T, D, V, K, dev), x, stream, (
        *args, _want(index, "index", tops, _int64(), dev), _want(teacher, "teacher", tops, f32, dev), scale, temperature,
        loss.data_ptr(), lse.data_ptr(), logits.data_ptr(), T, D, V, K, block._code[x.dtype], _on(stream, dev)))
    return loss, lse, logits


def ssm_distill_bwd(dloss, x, weight, index, teacher, lse, logits, temperature: float = 1.0, scale: float = 1.0,
                    want_x: bool = True, want_weight: bool = True, stream=None):
    """Gradients of ``ssm_distill_fwd`` for dloss [...] float32, from the forward's lse and
    logits.  Returns a dict with dx and dweight (bfloat16), as asked."""
    call = _fn("ssm_distill_bwd")
    dev, lead, T, D, V, args = _head(x, weight)
    K, tops = _tops(index, lead)
    f32 = block._F32
    g, ptrs = _head_grads(x, weight, want_x, want_weight)
    _with_workspace(call, ("distill_bwd", T, D, V, K, want_x, want_weight, dev), x, stream, (
        _want(dloss, "dloss", lead, f32, dev), *args, _want(index, "index", tops, _int64(), dev),
        _want(teacher, "teacher", tops, f32, dev), scale, temperature, _want(lse, "lse", lead, f32, dev),
        _want(logits, "logits", tops, f32, dev), *ptrs, T, D, V, K, block._code[x.dtype], _on(stream, dev)))
    return g
