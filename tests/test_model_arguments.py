"""Arguments of the model operators' binding and host layer that the other tests leave out,
without a GPU (each refusal comes before any HIP call is made)."""
import pytest

import sequence_scan_amd as ssm
from test_block_abi import NULL, UNSUPPORTED
from test_model_abi import step

torch = pytest.importorskip("torch")


BF = torch.bfloat16


def calls():
    """(entry point, a tensor that sizes or types are taken from, the other arguments)."""
    x, one, states = torch.zeros(2, 40, 64, dtype=BF), torch.zeros(2, 64, dtype=BF), torch.zeros(2, 2, 64)
    h, w, f = torch.zeros(6, 64, dtype=BF), torch.zeros(100, 64, dtype=BF), torch.zeros(6)
    t, index, top = torch.zeros(6, dtype=torch.int64), torch.zeros(6, 3, dtype=torch.int64), torch.zeros(6, 3)
    sizes = {
        "ssm_gscan_fwd": (dict(x=x, r=x), "x"),
        "ssm_gscan_bwd": (dict(x=x, r=x, i=None, rate=None, dout=x, states=states), "x dout"),
        "ssm_gscan_update": (dict(state=torch.zeros(2, 64), x=one, r=one), "x"),
        "ssm_xent_fwd": (dict(x=h, weight=w, target=t), "x weight"),
        "ssm_xent_bwd": (dict(dloss=f, x=h, weight=w, target=t, lse=f), "x weight"),
        "ssm_distill_fwd": (dict(x=h, weight=w, index=index, teacher=top), "x weight index"),
        "ssm_distill_bwd": (dict(dloss=f, x=h, weight=w, index=index, teacher=top, lse=f, logits=top), "x weight index"),
    }
    return [(name, m, {**kw, m: None}) for name, (kw, missing) in sizes.items() for m in missing.split()]


@pytest.mark.parametrize("name,missing,kw", calls(), ids=lambda v: v if isinstance(v, str) else "")
def test_a_missing_tensor_is_named(name, missing, kw):
    with pytest.raises(ValueError, match=rf"\b{missing} is required"):
        getattr(ssm, name)(**kw)


@pytest.mark.parametrize("batch,width", [((1 << 23) - 1, 1), (1 << 23, 1), ((1 << 31) - 1024, 1), (1 << 24, 64), (1 << 23, 255), (127, 1 << 24)])
def test_a_token_for_as_many_rows_as_the_header_says(batch, width):
    """Only batch * width and width are limited (a tensor is left out, so that nothing runs)."""
    rows = dict(x_row=width, r_row=width, i_row=width)
    assert step(x=None, batch=batch, width=width, **rows) == NULL, ssm.ssm_last_error()
    assert step(x=None, batch=batch + (1 << 31) // width, width=width, **rows) == UNSUPPORTED
    assert "2^31" in ssm.ssm_last_error()
