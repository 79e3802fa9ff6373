"""Offered workspaces (ssm_workspace, include/ssmblock.h) through the Python binding and the
real host layer, on the CPU: the host layer is built over the stand-ins for the runtime and
the kernel launchers (``tests/sanitize/fake_runtime.cpp``, ``fake_block.cpp``), whose device
memory is host memory and which compute nothing.  A call that asks the library's pool for
its workspace is told from one that takes offered memory by an allocation made to fail."""
import ctypes
import os
import shutil
import subprocess

import pytest

import sequence_scan_amd as ssm
from sequence_scan_amd import block
from test_sanitizers import HERE, HIP_INCLUDE, ROOT

torch = pytest.importorskip("torch")

CALLS = ("ssm_workspace", "ssm_workspace_bytes", "ssm_add_norm_bwd")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.isdir(os.path.join(HIP_INCLUDE, "hip")):
        pytest.skip("g++ or the HIP headers not found")
    so = str(tmp_path_factory.mktemp("host") / "libblockhost.so")
    csrc, fakes = os.path.join(ROOT, "sequence_scan_amd", "csrc"), os.path.join(HERE, "sanitize")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", f"-I{HIP_INCLUDE}",
                        os.path.join(csrc, "api.cpp"), os.path.join(csrc, "api_block.cpp"),
                        os.path.join(fakes, "fake_runtime.cpp"), os.path.join(fakes, "fake_block.cpp"), "-o", so],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    return ctypes.CDLL(so)


@pytest.fixture
def fake(host, monkeypatch):
    """The binding's functions from the host layer over the fake runtime."""
    block._fn("ssm_workspace")          # (looks up what the wrappers use of PyTorch)
    for name in CALLS:
        f = getattr(host, name)
        f.argtypes, f.restype = block._ARGS[name], ctypes.c_int64 if name == "ssm_workspace_bytes" else ctypes.c_int
        monkeypatch.setitem(block._fns, name, f)
    monkeypatch.setattr(block, "_wanted", {})
    block._fns["ssm_workspace"](None, 0)
    return host


def add_norm_bwd_args(rows=16, width=64, eps=1e-5):
    """Arguments of ssm_add_norm_bwd, which wants a workspace for its column sums."""
    t = {n: torch.zeros(rows, width) for n in ("dout", "r", "dx", "dres")}
    w = torch.zeros(width)
    args = [t["dout"].data_ptr(), t["r"].data_ptr(), None, None, None, width, None, 1.0, eps, 0, t["dx"].data_ptr(),
            t["dres"].data_ptr(), w.data_ptr(), None, None, rows, width, ssm.SSM_F32, ssm.SSM_F32, ssm.SSM_F32, None]
    return args, (t, w)


def takes_from_pool(host, keep, args):
    """Whether the call asks the pool for its workspace: made to fail, the pool's refusal is the call's."""
    host.fake_fail_next_alloc()
    status = block._fn("ssm_add_norm_bwd")(*args)
    if status == ssm.SSM_OK:
        # the offer was taken: spend the failure, which would meet a later call
        assert block._fn("ssm_add_norm_bwd")(*args) == ssm.SSM_ERR_HIP
    return status == ssm.SSM_ERR_HIP


def test_an_offer_is_taken_once(fake):
    args, keep = add_norm_bwd_args()
    assert takes_from_pool(fake, keep, args)
    assert block._fn("ssm_add_norm_bwd")(*args) == ssm.SSM_OK
    n = ssm.ssm_workspace_bytes()
    memory = torch.zeros(n + 16, dtype=torch.uint8)
    at = memory.data_ptr() + -memory.data_ptr() % 16
    ssm.ssm_workspace(at, n)
    assert not takes_from_pool(fake, keep, args)
    ssm.ssm_workspace(at, n)
    ssm.ssm_workspace(None, 0)
    assert takes_from_pool(fake, keep, args)


def test_no_offer_outlives_a_call_that_ctypes_refuses(fake):
    """An argument that ctypes cannot convert ends the call before the library is entered, which
    then does not take the offer; the binding has to withdraw it."""
    call, like = block._fn("ssm_add_norm_bwd"), torch.zeros(1)
    args, keep = add_norm_bwd_args()
    block._with_workspace(call, "key", like, None, args)             # learns what the call wants
    assert block._wanted["key"] > 0
    for i, bad in ((15, 16.0), (8, None), (8, "1e-5")):              # rows, eps
        with pytest.raises(ctypes.ArgumentError):
            block._with_workspace(call, "key", like, None, [*args[:i], bad, *args[i + 1:]])
        assert takes_from_pool(fake, keep, args), "the next call took memory that is no longer the offer's"


def test_no_offer_outlives_a_call_that_the_library_refuses(fake):
    call, like = block._fn("ssm_add_norm_bwd"), torch.zeros(1)
    args, keep = add_norm_bwd_args()
    block._with_workspace(call, "key", like, None, args)
    with pytest.raises(ssm.SSMError):
        block._with_workspace(call, "key", like, None, [*args[:8], -1.0, *args[9:]])
    assert takes_from_pool(fake, keep, args)


def test_bytes_are_those_of_the_last_call_whatever_is_offered(fake):
    """ssm_workspace_bytes answers for the thread's last call: an offer, or its withdrawal, is none."""
    args, keep = add_norm_bwd_args()
    assert block._fn("ssm_add_norm_bwd")(*args) == ssm.SSM_OK
    n = ssm.ssm_workspace_bytes()
    assert n > 0
    memory = torch.zeros(n + 16, dtype=torch.uint8)
    ssm.ssm_workspace(memory.data_ptr() + -memory.data_ptr() % 16, n)
    assert ssm.ssm_workspace_bytes() == n
    ssm.ssm_workspace(None, 0)
    assert ssm.ssm_workspace_bytes() == n
    with pytest.raises(ssm.SSMError):
        ssm.ssm_workspace(memory.data_ptr() + 1, n)
    assert ssm.ssm_workspace_bytes() == n
    assert block._fn("ssm_add_norm_bwd")(*args[:8], -1.0, *args[9:]) == ssm.SSM_ERR_UNSUPPORTED
    assert ssm.ssm_workspace_bytes() == 0           # (a refused call wants nothing)
