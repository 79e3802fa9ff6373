"""The model operators' C ABI (include/ssmmodel.h) and binding without a GPU: exports, and
every refusal of the host layer (each returns before any HIP call is made)."""
import os
import re

import pytest

import sequence_scan_amd as ssm
from sequence_scan_amd import block
from test_block_abi import BF16, F32, NULL, SHAPE, UNSUPPORTED, Call, ptr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssmmodel.h")


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(ssm_\w+)\s*\(", text, flags=re.M)))


def test_every_declared_function_is_exported_and_bound():
    lib = ssm.library()
    names = declared()
    assert len(names) == 7
    for n in names:
        assert hasattr(lib, n), f"{n} is declared in ssmmodel.h but not exported"
        assert n in block._ARGS
        assert callable(getattr(ssm, n))


def test_constants_agree_with_the_header():
    text = open(HEADER).read()
    for name in ("SSM_GSCAN_LERP", "SSM_GSCAN_SEGMENT"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(ssm, name)


gates = dict(x=ptr(0), x_row=64, r=ptr(1), r_row=64, i=ptr(2), i_row=64, rate=ptr(3), flags=0)
fwd = Call("ssm_gscan_fwd", **gates, initial_state=ptr(4), out=ptr(5), last_state=ptr(6), states=ptr(7), batch=2, seqlen=300, width=64,
           in_dtype=BF16, out_dtype=BF16, stream=None)
bwd = Call("ssm_gscan_bwd", **gates, states=ptr(4), dout=ptr(5), dlast_state=ptr(6), dx=ptr(7), dr=ptr(8), di=ptr(9), drate=ptr(10),
           dinitial_state=ptr(11), batch=2, seqlen=300, width=64, in_dtype=BF16, out_dtype=BF16, stream=None)
step = Call("ssm_gscan_update", state=ptr(8), state_out=ptr(9), **gates, out=ptr(10), batch=2, width=64, in_dtype=BF16, out_dtype=F32,
            stream=None)
xent = Call("ssm_xent_fwd", x=ptr(0), x_row=64, weight=ptr(1), w_row=64, target=ptr(2), scale=1.0, z_loss=0.0, loss=ptr(3), lse=ptr(4),
            rows=5, width=64, vocab=300, in_dtype=BF16, stream=None)
xent_bwd = Call("ssm_xent_bwd", dloss=ptr(0), x=ptr(1), x_row=64, weight=ptr(2), w_row=64, target=ptr(3), scale=1.0, z_loss=0.0,
                lse=ptr(4), dx=ptr(5), dweight=ptr(6), rows=5, width=64, vocab=300, in_dtype=BF16, stream=None)
distill = Call("ssm_distill_fwd", x=ptr(0), x_row=64, weight=ptr(1), w_row=64, index=ptr(2), teacher=ptr(3), scale=1.0, temperature=2.0,
               loss=ptr(4), lse=ptr(5), logits=ptr(6), rows=5, width=64, vocab=300, top=8, in_dtype=BF16, stream=None)
distill_bwd = Call("ssm_distill_bwd", dloss=ptr(0), x=ptr(1), x_row=64, weight=ptr(2), w_row=64, index=ptr(3), teacher=ptr(4), scale=1.0,
                   temperature=2.0, lse=ptr(5), logits=ptr(6), dx=ptr(7), dweight=ptr(8), rows=5, width=64, vocab=300, top=8,
                   in_dtype=BF16, stream=None)

REQUIRED = {
    fwd: "x r out", bwd: "x r states dout dx dr di", step: "state state_out x r out", xent: "x weight target loss lse",
    xent_bwd: "dloss x weight target lse", distill: "x weight index teacher loss lse logits",
    distill_bwd: "dloss x weight index teacher lse logits",
}


@pytest.mark.parametrize("call,arg", [(c, a) for c, args in REQUIRED.items() for a in args.split()],
                         ids=lambda v: v.name if isinstance(v, Call) else v)
def test_missing_tensor(call, arg):
    assert call(**{arg: None}) == NULL
    assert arg in ssm.ssm_last_error()


BAD = [
    (fwd, dict(batch=-1), SHAPE, "batch"), (fwd, dict(seqlen=-1), SHAPE, "seqlen"), (fwd, dict(width=-2), SHAPE, "width"),
    (fwd, dict(flags=2), UNSUPPORTED, "flags"), (fwd, dict(in_dtype=4), UNSUPPORTED, "dtype"), (fwd, dict(out_dtype=-1), UNSUPPORTED, "dtype"),
    (fwd, dict(x_row=63), UNSUPPORTED, "x rows"), (fwd, dict(r_row=0), UNSUPPORTED, "r rows"), (fwd, dict(i_row=(1 << 24) + 1), UNSUPPORTED, "i rows"),
    (fwd, dict(x=ptr(0) + 1), UNSUPPORTED, "x"), (fwd, dict(rate=ptr(3) + 2), UNSUPPORTED, "rate"),
    (fwd, dict(out=ptr(0)), UNSUPPORTED, "overlaps"), (fwd, dict(last_state=ptr(4) + 4), UNSUPPORTED, "overlaps"),
    (fwd, dict(states=ptr(5) + 64), UNSUPPORTED, "overlaps"), (fwd, dict(states=ptr(4)), UNSUPPORTED, "overlaps"),
    (fwd, dict(batch=1 << 40, seqlen=1 << 40), SHAPE, "overflow"), (fwd, dict(batch=1 << 26), UNSUPPORTED, "2^31"),
    (fwd, dict(batch=1, width=1 << 25, x_row=1 << 25, r_row=1 << 25, i_row=1 << 25), UNSUPPORTED, "2^24"),
    (fwd, dict(batch=1, seqlen=1 << 32), UNSUPPORTED, "grid"),
    (fwd, dict(batch=1 << 23, seqlen=1, width=1), UNSUPPORTED, "grid"), (fwd, dict(batch=1 << 22, seqlen=65, width=1), UNSUPPORTED, "grid"),
    (bwd, dict(dx=ptr(0)), UNSUPPORTED, "overlaps"), (bwd, dict(di=ptr(8)), UNSUPPORTED, "overlaps"),
    (bwd, dict(dinitial_state=ptr(6)), UNSUPPORTED, "overlaps"), (bwd, dict(rate=None), UNSUPPORTED, "drate"),
    (bwd, dict(i=None), UNSUPPORTED, "di"), (bwd, dict(seqlen=-1), SHAPE, "seqlen"), (bwd, dict(dr=ptr(8) + 1), UNSUPPORTED, "dr"),
    (bwd, dict(r_row=5), UNSUPPORTED, "r rows"), (bwd, dict(flags=1 << 30), UNSUPPORTED, "flags"),
    (step, dict(state_out=ptr(8) + 4), UNSUPPORTED, "overlaps"), (step, dict(out=ptr(0)), UNSUPPORTED, "overlaps"),
    (step, dict(batch=-1), SHAPE, "batch"), (step, dict(x_row=1), UNSUPPORTED, "x rows"), (step, dict(in_dtype=7), UNSUPPORTED, "dtype"),
    (xent, dict(rows=-1), SHAPE, "rows"), (xent, dict(width=60, x_row=64), UNSUPPORTED, "multiple of 8"), (xent, dict(width=0), UNSUPPORTED, "width"),
    (xent, dict(width=65544, x_row=65544, w_row=65544), UNSUPPORTED, "65536"), (xent, dict(vocab=0), UNSUPPORTED, "vocab"),
    (xent, dict(vocab=(1 << 30) + 1), UNSUPPORTED, "vocab"), (xent, dict(rows=(1 << 22) + 1), UNSUPPORTED, "rows"),
    (xent, dict(rows=1 << 22, vocab=1 << 20), UNSUPPORTED, "tiles"), (xent, dict(in_dtype=F32), UNSUPPORTED, "bf16"),
    (xent, dict(rows=1 << 22, vocab=65537), UNSUPPORTED, "tiles"),
    (xent, dict(vocab=1 << 24, width=65536, x_row=65536, w_row=65536), UNSUPPORTED, "2^37"),
    (xent, dict(x_row=56), UNSUPPORTED, "x rows"), (xent, dict(x_row=68), UNSUPPORTED, "x rows"), (xent, dict(w_row=(1 << 22) + 8), UNSUPPORTED, "weight rows"),
    (xent, dict(x=ptr(0) + 8), UNSUPPORTED, "x"), (xent, dict(weight=ptr(1) + 2), UNSUPPORTED, "weight"), (xent, dict(target=ptr(2) + 4), UNSUPPORTED, "target"),
    (xent, dict(scale=float("inf")), UNSUPPORTED, "scale"), (xent, dict(z_loss=float("nan")), UNSUPPORTED, "z_loss"),
    (xent, dict(lse=ptr(3)), UNSUPPORTED, "overlaps"), (xent, dict(loss=ptr(1)), UNSUPPORTED, "overlaps"),
    (xent_bwd, dict(dx=ptr(1)), UNSUPPORTED, "overlaps"), (xent_bwd, dict(dweight=ptr(2)), UNSUPPORTED, "overlaps"),
    (xent_bwd, dict(dweight=ptr(5)), UNSUPPORTED, "overlaps"), (xent_bwd, dict(dx=ptr(5) + 8), UNSUPPORTED, "dx"),
    (xent_bwd, dict(z_loss=float("inf")), UNSUPPORTED, "z_loss"), (xent_bwd, dict(in_dtype=F32), UNSUPPORTED, "bf16"), (xent_bwd, dict(vocab=-1), SHAPE, "vocab"),
    (distill, dict(top=0), UNSUPPORTED, "top"), (distill, dict(top=1025), UNSUPPORTED, "1024"), (distill, dict(top=-1), SHAPE, "top"),
    (distill, dict(temperature=0.0), UNSUPPORTED, "temperature"), (distill, dict(temperature=float("nan")), UNSUPPORTED, "temperature"),
    (distill, dict(temperature=1e-39), UNSUPPORTED, "temperature"), (distill, dict(temperature=1e30), UNSUPPORTED, "temperature"),
    (distill, dict(temperature=1e-20), UNSUPPORTED, "temperature"),
    (distill, dict(logits=ptr(3)), UNSUPPORTED, "overlaps"), (distill, dict(index=ptr(2) + 4), UNSUPPORTED, "index"),
    (distill_bwd, dict(dx=ptr(6)), UNSUPPORTED, "overlaps"), (distill_bwd, dict(dweight=ptr(2) + 16), UNSUPPORTED, "overlaps"),
    (distill_bwd, dict(temperature=-1.0), UNSUPPORTED, "temperature"), (distill_bwd, dict(w_row=8), UNSUPPORTED, "weight rows"),
]


@pytest.mark.parametrize("call,kw,status,says", BAD, ids=[f"{c.name}-{'-'.join(k)}-{i}" for i, (c, k, _, _) in enumerate(BAD)])
def test_refusal(call, kw, status, says):
    assert call(**kw) == status, ssm.ssm_last_error()
    assert says in ssm.ssm_last_error()


def test_a_refused_call_ends_an_offer():
    offer = block._fn("ssm_workspace")
    for call, kw in ((fwd, dict(flags=2)), (bwd, dict(flags=2)), (xent, dict(rows=-1)), (xent_bwd, dict(rows=-1)),
                     (distill, dict(top=0)), (distill_bwd, dict(top=0))):
        assert offer(ptr(20), 4096) == ssm.SSM_OK
        assert call(**kw) != ssm.SSM_OK and ssm.ssm_workspace_bytes() == 0


def test_empty_calls_need_no_tensors():
    none = dict(x=None, r=None, i=None, out=None, states=None)
    assert fwd(**none, batch=0, initial_state=None, last_state=None) == ssm.SSM_OK
    assert step(state=None, state_out=None, x=None, r=None, out=None, batch=0) == ssm.SSM_OK
    assert xent(x=None, weight=None, target=None, loss=None, lse=None, rows=0) == ssm.SSM_OK
    assert distill(x=None, weight=None, index=None, teacher=None, loss=None, lse=None, logits=None, rows=0) == ssm.SSM_OK
    assert xent_bwd(dloss=None, x=None, weight=None, target=None, lse=None, dx=None, dweight=None, rows=0) == ssm.SSM_OK


def test_binding_refuses_before_the_library_is_called():
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    x = torch.zeros(2, 40, 64, dtype=bf)
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_gscan_fwd(x, x)
    with pytest.raises(ValueError, match=r"\[batch, seqlen, width\]"):
        ssm.ssm_gscan_fwd(x[0], x[0])
    with pytest.raises(ValueError, match="shape"):
        ssm.ssm_gscan_fwd(x, x[:, :39])
    with pytest.raises(TypeError):
        ssm.ssm_gscan_fwd(x, x.float())
    with pytest.raises(TypeError):
        ssm.ssm_gscan_fwd(x.half(), x.half())
    with pytest.raises(TypeError):
        ssm.ssm_gscan_fwd(x, x, rate=torch.zeros(64, dtype=bf))
    with pytest.raises(ValueError, match="states"):
        ssm.ssm_gscan_fwd(x, x, states=torch.zeros(2, 1, 64))
    with pytest.raises(ValueError, match="states"):
        ssm.ssm_gscan_bwd(x, x, None, None, x, torch.zeros(2, 3, 64))
    with pytest.raises(ValueError, match=r"\[batch, width\]"):
        ssm.ssm_gscan_update(torch.zeros(2, 64), x, x)
    with pytest.raises(ValueError, match="evenly spaced"):
        ssm.ssm_gscan_fwd(torch.zeros(4, 40, 64, dtype=bf)[::2][:, ::3], torch.zeros(2, 14, 64, dtype=bf))
    h, w = torch.zeros(6, 64, dtype=bf), torch.zeros(100, 64, dtype=bf)
    t = torch.zeros(6, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_xent_fwd(h, w, t)
    with pytest.raises(ValueError, match="columns"):
        ssm.ssm_xent_fwd(h, w[:, :32], t)
    with pytest.raises(TypeError):
        ssm.ssm_xent_fwd(h, w, t.int())
    with pytest.raises(ValueError, match="target"):
        ssm.ssm_xent_fwd(h, w, t[:5])
    with pytest.raises(TypeError):
        ssm.ssm_xent_fwd(h, w.float(), t)
    with pytest.raises(ValueError, match="lse"):
        ssm.ssm_xent_bwd(torch.zeros(6), h, w, t, torch.zeros(5))
    with pytest.raises(ValueError, match="top"):
        ssm.ssm_distill_fwd(h, w, t, torch.zeros(6))
    with pytest.raises(ValueError, match="teacher"):
        ssm.ssm_distill_fwd(h, w, t[:, None], torch.zeros(6, 2))
    with pytest.raises(TypeError):
        ssm.ssm_distill_fwd(h, w, t[:, None], torch.zeros(6, 1, dtype=bf))
