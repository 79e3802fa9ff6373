"""The gated linear recurrence at the ends of its ranges."""
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ssm = pytest.importorskip("sequence_scan_amd")

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ssm.library()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_token_of_many_narrow_rows(dtype):
    """More rows than the sequences' grids have workgroups: the same bits as of one wide row."""
    say(f"many narrow rows {dtype}")
    B = (1 << 23) + 5
    g = torch.Generator(device="cuda").manual_seed(0)
    x, r, i = (torch.randn(B, 1, device="cuda", generator=g).to(dtype) for _ in range(3))
    S, wide = (torch.randn(B, 1, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) for _ in range(2))
    out = ssm.ssm_gscan_update(S, x, r, i)
    want = ssm.ssm_gscan_update(wide.view(1, B), *(t.view(1, B) for t in (x, r, i)))
    assert torch.equal(out.view(1, B), want) and torch.equal(S, wide)
