"""The block operators' C ABI (include/ssmblock.h) and binding without a GPU: exports,
and every refusal of the host layer (each returns before any HIP call is made)."""
import os
import re

import pytest

import sequence_scan_amd as ssm
from sequence_scan_amd import block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssmblock.h")
F32, BF16 = ssm.SSM_F32, ssm.SSM_BF16
NULL, SHAPE, UNSUPPORTED = ssm.SSM_ERR_NULL_ARG, ssm.SSM_ERR_BAD_SHAPE, ssm.SSM_ERR_UNSUPPORTED
P = 0x10000000      # aligned addresses far apart: never read on these paths
STEP = 1 << 40


def ptr(i):
    return P + i * STEP


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(ssm_\w+)\s*\(", text, flags=re.M)))


def test_every_declared_function_is_exported_and_bound():
    lib = ssm.library()
    names = declared()
    assert len(names) == 12
    for n in names:
        assert hasattr(lib, n), f"{n} is declared in ssmblock.h but not exported"
        assert n in block._ARGS
        assert callable(getattr(ssm, n))


def test_constants_agree_with_the_header():
    text = open(HEADER).read()
    for name in ("SSM_NORM_CENTER", "SSM_NORM_GATE_LAST", "SSM_LINATTN_FIXED_DECAY"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(ssm, name)


class Call:
    """A C call by named arguments, in the order of the declaration."""

    def __init__(self, name, **args):
        self.name, self.args = name, args

    def __call__(self, **kw):
        assert set(kw) <= set(self.args), kw
        return block._fn(self.name)(*{**self.args, **kw}.values())


add_fwd = Call("ssm_add_norm_fwd", x=ptr(0), x_stride=64, residual=ptr(1), weight=ptr(2), bias=ptr(3), scale=ptr(4), alpha=1.0,
               eps=1e-5, flags=0, out=ptr(5), residual_out=ptr(6), rows=8, width=64, x_dtype=BF16, res_dtype=F32, out_dtype=BF16,
               stream=None)
add_bwd = Call("ssm_add_norm_bwd", dout=ptr(0), r=ptr(1), weight=ptr(2), dresidual_out=ptr(3), x=ptr(4), x_stride=64,
               scale=ptr(5), alpha=1.0, eps=1e-5, flags=0, dx=ptr(6), dresidual=ptr(7), dweight=ptr(8), dbias=ptr(9),
               dscale=ptr(10), rows=8, width=64, x_dtype=BF16, res_dtype=F32, out_dtype=BF16, stream=None)
gate_fwd = Call("ssm_gated_norm_fwd", x=ptr(0), x_stride=64, z=ptr(1), z_stride=64, weight=ptr(2), bias=ptr(3), eps=1e-5, flags=0,
                out=ptr(4), rows=8, width=64, ngroups=4, in_dtype=BF16, out_dtype=BF16, stream=None)
gate_bwd = Call("ssm_gated_norm_bwd", dout=ptr(0), x=ptr(1), x_stride=64, z=ptr(2), z_stride=64, weight=ptr(3), bias=ptr(4),
                eps=1e-5, flags=0, dx=ptr(5), dz=ptr(6), dweight=ptr(7), dbias=ptr(8), rows=8, width=64, ngroups=4, in_dtype=BF16,
                out_dtype=BF16, stream=None)
la_fwd = Call("ssm_linattn_fwd", q=ptr(0), q_row=128, k=ptr(1), k_row=128, v=ptr(2), v_row=256, log_decay=ptr(3), flags=0, scale=1.0,
              initial_state=ptr(4), out=ptr(5), last_state=ptr(6), batch=2, seqlen=40, nheads=4, ngroups=2, dk=64, dv=64,
              in_dtype=BF16, out_dtype=BF16, stream=None, plan=None)
la_bwd = Call("ssm_linattn_bwd", q=ptr(0), q_row=128, k=ptr(1), k_row=128, v=ptr(2), v_row=256, log_decay=ptr(3), flags=0, scale=1.0,
              initial_state=ptr(4), dout=ptr(5), dlast_state=ptr(6), dq=ptr(7), dk=ptr(8), dv=ptr(9), dlog_decay=ptr(10),
              dinitial_state=ptr(11), batch=2, seqlen=40, nheads=4, ngroups=2, dk_=64, dv_=64, in_dtype=BF16, grad_dtype=BF16,
              stream=None)
la_step = Call("ssm_linattn_state_update", state=ptr(0), state_out=ptr(1), q=ptr(2), k=ptr(3), v=ptr(4), log_decay=ptr(5), flags=0,
               scale=1.0, out=ptr(6), batch=2, nheads=4, ngroups=2, dk=64, dv=64, in_dtype=BF16, out_dtype=BF16, stream=None)
q4 = Call("ssm_q4_matvec", x=ptr(0), x_row=256, codes=ptr(1), scales=ptr(2), zeros=ptr(3), bias=ptr(4), out=ptr(5), m=3, n=48, k=256,
          group=64, in_dtype=BF16, scale_dtype=F32, out_dtype=BF16, stream=None)
quantize = Call("ssm_q4_quantize", w=ptr(0), codes=ptr(1), scales=ptr(2), zeros=ptr(3), n=48, k=256, group=64, w_dtype=BF16,
                scale_dtype=F32, stream=None)

REQUIRED = {
    add_fwd: "x out", add_bwd: "dout r x", gate_fwd: "x out", gate_bwd: "dout x dx dz",
    la_fwd: "q k v log_decay out", la_bwd: "q k v log_decay dout dq dk dv dlog_decay",
    la_step: "state state_out q k v log_decay out", q4: "x codes scales out", quantize: "w codes scales zeros",
}


@pytest.mark.parametrize("call,arg", [(c, a) for c, args in REQUIRED.items() for a in args.split()],
                         ids=lambda v: v.name if isinstance(v, Call) else v)
def test_missing_tensor(call, arg):
    assert call(**{arg: None}) == NULL
    assert arg in ssm.ssm_last_error()


BAD = [
    (add_fwd, dict(rows=-1), SHAPE, "rows"), (add_fwd, dict(width=-4), SHAPE, "width"),
    (add_fwd, dict(rows=8, width=1 << 23, x_stride=1 << 23), UNSUPPORTED, "channels"),
    (add_fwd, dict(rows=1 << 60), SHAPE, "overflow"),
    (add_fwd, dict(width=8193, x_stride=8193), UNSUPPORTED, "8193"), (add_fwd, dict(x_stride=63), UNSUPPORTED, "x rows"),
    (add_fwd, dict(eps=-1.0), UNSUPPORTED, "eps"), (add_fwd, dict(eps=float("nan")), UNSUPPORTED, "eps"),
    (add_fwd, dict(eps=float("inf")), UNSUPPORTED, "eps"), (add_fwd, dict(flags=2), UNSUPPORTED, "flags"),
    (add_fwd, dict(flags=4), UNSUPPORTED, "flags"), (add_fwd, dict(x_dtype=2), UNSUPPORTED, "dtype"),
    (add_fwd, dict(res_dtype=-1), UNSUPPORTED, "dtype"), (add_fwd, dict(out_dtype=9), UNSUPPORTED, "dtype"),
    (add_fwd, dict(x=ptr(0) + 1), UNSUPPORTED, "x"), (add_fwd, dict(weight=ptr(2) + 2), UNSUPPORTED, "weight"),
    (add_fwd, dict(out=ptr(0)), UNSUPPORTED, "overlaps"), (add_fwd, dict(out=ptr(1) + 64), UNSUPPORTED, "overlaps"),
    (add_fwd, dict(residual_out=ptr(1) + 4), UNSUPPORTED, "overlaps"),
    (add_fwd, dict(residual_out=ptr(5)), UNSUPPORTED, "overlaps"),
    (add_bwd, dict(rows=-1), SHAPE, "rows"), (add_bwd, dict(x_stride=1), UNSUPPORTED, "x rows"),
    (add_bwd, dict(flags=2), UNSUPPORTED, "flags"), (add_bwd, dict(dx=ptr(0)), UNSUPPORTED, "overlaps"),
    (add_bwd, dict(dresidual=ptr(1)), UNSUPPORTED, "overlaps"), (add_bwd, dict(dbias=ptr(8)), UNSUPPORTED, "overlaps"),
    (add_bwd, dict(dresidual=ptr(3) + 4), UNSUPPORTED, "overlaps"),
    (gate_fwd, dict(ngroups=3), UNSUPPORTED, "ngroups"), (gate_fwd, dict(ngroups=0), UNSUPPORTED, "ngroups"),
    (gate_fwd, dict(width=70000, ngroups=70000, x_stride=70000, z_stride=70000), UNSUPPORTED, "65535"),
    (gate_fwd, dict(width=1 << 25, ngroups=1 << 14, x_stride=1 << 25, z_stride=1 << 25), UNSUPPORTED, "exceeds"),
    (gate_fwd, dict(z_stride=60), UNSUPPORTED, "z rows"), (gate_fwd, dict(flags=4), UNSUPPORTED, "flags"),
    (gate_fwd, dict(out=ptr(1)), UNSUPPORTED, "overlaps"), (gate_fwd, dict(in_dtype=5), UNSUPPORTED, "dtype"),
    (gate_bwd, dict(z=None), UNSUPPORTED, "dz"), (gate_bwd, dict(dz=ptr(5)), UNSUPPORTED, "overlaps"),
    (gate_bwd, dict(dx=ptr(1)), UNSUPPORTED, "overlaps"), (gate_bwd, dict(rows=-3), SHAPE, "rows"),
    (la_fwd, dict(seqlen=-1), SHAPE, "seqlen"), (la_fwd, dict(ngroups=3), UNSUPPORTED, "ngroups"),
    (la_fwd, dict(nheads=0, ngroups=1), UNSUPPORTED, "nheads"), (la_fwd, dict(dk=60, q_row=120, k_row=120), UNSUPPORTED, "multiples of 8"),
    (la_fwd, dict(dv=136, v_row=544), UNSUPPORTED, "128"), (la_fwd, dict(in_dtype=F32), UNSUPPORTED, "bf16"),
    (la_fwd, dict(q_row=120), UNSUPPORTED, "q rows"), (la_fwd, dict(k_row=132), UNSUPPORTED, "k rows"),
    (la_fwd, dict(v_row=(1 << 24) + 8), UNSUPPORTED, "v rows"), (la_fwd, dict(flags=2), UNSUPPORTED, "flags"),
    (la_fwd, dict(scale=float("nan")), UNSUPPORTED, "scale"), (la_fwd, dict(q=ptr(0) + 8), UNSUPPORTED, "q"),
    (la_fwd, dict(out=ptr(2)), UNSUPPORTED, "overlaps"), (la_fwd, dict(last_state=ptr(4) + 16), UNSUPPORTED, "overlaps"),
    (la_fwd, dict(last_state=ptr(5)), UNSUPPORTED, "overlaps"), (la_fwd, dict(nheads=65536, v_row=65536 * 64), UNSUPPORTED, "65535"),
    (la_fwd, dict(batch=65535, nheads=200, v_row=12800), UNSUPPORTED, "grid"),
    (la_fwd, dict(batch=1 << 15, seqlen=1 << 60), SHAPE, "overflow"),
    (la_bwd, dict(in_dtype=F32), UNSUPPORTED, "bf16"), (la_bwd, dict(dq=ptr(0)), UNSUPPORTED, "overlaps"),
    (la_bwd, dict(dinitial_state=ptr(6)), UNSUPPORTED, "overlaps"), (la_bwd, dict(dv=ptr(9) + 4), UNSUPPORTED, "dv"),
    (la_bwd, dict(grad_dtype=3), UNSUPPORTED, "dtype"), (la_bwd, dict(batch=-2), SHAPE, "batch"),
    (la_bwd, dict(seqlen=1 << 28), UNSUPPORTED, "time chunks"),
    (la_step, dict(dk=66), UNSUPPORTED, "multiple of 4"), (la_step, dict(dk=260), UNSUPPORTED, "256"),
    (la_step, dict(dv=0), UNSUPPORTED, "positive"), (la_step, dict(state_out=ptr(0) + 16), UNSUPPORTED, "overlaps"),
    (la_step, dict(out=ptr(4)), UNSUPPORTED, "overlaps"), (la_step, dict(q=ptr(2) + 2), UNSUPPORTED, "q"),
    (la_step, dict(batch=65536), UNSUPPORTED, "65535"), (la_step, dict(flags=8), UNSUPPORTED, "flags"),
    (q4, dict(group=16), UNSUPPORTED, "group"), (q4, dict(group=256), UNSUPPORTED, "group"),
    (q4, dict(k=224), UNSUPPORTED, "multiple of group"), (q4, dict(m=-1), SHAPE, "m="),
    (q4, dict(x_row=255), UNSUPPORTED, "x rows"), (q4, dict(x_row=260), UNSUPPORTED, "x rows"),
    (q4, dict(x=ptr(0) + 2), UNSUPPORTED, "x"), (q4, dict(codes=ptr(1) + 8), UNSUPPORTED, "codes"),
    (q4, dict(out=ptr(0)), UNSUPPORTED, "overlaps"), (q4, dict(scale_dtype=4), UNSUPPORTED, "dtype"),
    (q4, dict(n=1 << 28), UNSUPPORTED, "indexes"), (q4, dict(m=400000), UNSUPPORTED, "indexes"),
    (q4, dict(n=1 << 40, k=1 << 40), SHAPE, "overflow"),
    (quantize, dict(codes=ptr(0)), UNSUPPORTED, "overlaps"), (quantize, dict(scales=ptr(1)), UNSUPPORTED, "overlaps"),
    (quantize, dict(n=1 << 27, k=1 << 13, group=32), UNSUPPORTED, "grid"), (quantize, dict(w_dtype=3), UNSUPPORTED, "dtype"),
]


@pytest.mark.parametrize("call,kw,status,says", BAD, ids=[f"{c.name}-{'-'.join(k)}-{i}" for i, (c, k, _, _) in enumerate(BAD)])
def test_refusal(call, kw, status, says):
    assert call(**kw) == status, ssm.ssm_last_error()
    assert says in ssm.ssm_last_error()


def test_workspace_offers():
    offer = block._fn("ssm_workspace")
    assert offer(ptr(0), 4096) == ssm.SSM_OK and ssm.ssm_workspace_bytes() == 0
    assert offer(ptr(0) + 8, 4096) == UNSUPPORTED and offer(ptr(0), -1) == SHAPE
    assert offer(None, 0) == ssm.SSM_OK
    assert offer(ptr(0), 4096) == ssm.SSM_OK
    assert la_bwd(batch=-1) == SHAPE and ssm.ssm_workspace_bytes() == 0     # (a refused call ends the offer)


@pytest.mark.parametrize("chunk_len", [-1, 0, 31, 33])
def test_plan_refusal(chunk_len):
    import ctypes
    p = ssm.ssm_plan()
    p.chunk_len = chunk_len
    assert la_fwd(plan=ctypes.byref(p)) == UNSUPPORTED
    assert "chunk_len" in ssm.ssm_last_error()
    assert block._fn("ssm_linattn_plan_query")(1, 8, 1, 64, 64, None) == NULL


@pytest.mark.parametrize("sizes", [(1, 0, 1, 8, 8), (1, 1, 1, 8, 8), (1, 100000, 1, 128, 128), (64, 2048, 32, 64, 64)])
def test_plan_covers_the_sequence(sizes):
    p = ssm.ssm_linattn_plan_query(*sizes)
    L = sizes[1]
    assert p["chunk_len"] >= 1 and p["n_chunks"] == -(-L // p["chunk_len"])
    assert p["n_chunks"] <= 1 or p["chunk_len"] % 32 == 0


def test_binding_refuses_before_the_library_is_called():
    torch = pytest.importorskip("torch")
    bf, f = torch.bfloat16, torch.float32
    x = torch.zeros(4, 64, dtype=bf)
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_add_norm_fwd(x)
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_gated_norm_fwd(x)
    with pytest.raises(TypeError):
        ssm.ssm_add_norm_fwd(x.half())
    with pytest.raises(ValueError, match="needs x"):
        ssm.ssm_add_norm_bwd(x, x.float(), want_scale=True)
    with pytest.raises(TypeError, match="dx"):
        ssm.ssm_add_norm_bwd(x, x.float(), x=x, dx_dtype=f)
    q, v, g = torch.zeros(1, 8, 2, 64, dtype=bf), torch.zeros(1, 8, 4, 64, dtype=bf), torch.zeros(1, 8, 4)
    with pytest.raises(ValueError, match="batch, seqlen"):
        ssm.ssm_linattn_fwd(q[0], q[0], v[0], g)
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_linattn_fwd(q, q, v, g)
    with pytest.raises(TypeError):
        ssm.ssm_linattn_bwd(q, q, v, g, v, grad_dtype=torch.float16)
    with pytest.raises(ValueError, match="shape"):
        ssm.ssm_linattn_state_update(torch.zeros(1, 4, 64, 64), q[:, 0], q[:, 0], v[:, 0], g[:, 0, :3])
    codes, scales = torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 2)
    with pytest.raises(ValueError, match="columns"):
        ssm.ssm_q4_matvec(torch.zeros(1, 64, dtype=bf), codes, scales)
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_q4_matvec(torch.zeros(1, 128, dtype=bf), codes, scales)
    with pytest.raises(ValueError, match="group"):
        ssm.ssm_q4_quantize(torch.zeros(8, 128), group=48)
    with pytest.raises(ValueError, match=r"\[n, k\]"):
        ssm.ssm_q4_quantize(torch.zeros(8, 4, 128))
