"""The bounded waits of the attention kernels on the GPU: one that runs out
reports FT_ERR_TIMEOUT, ends, and ends the block's other waits; the context
stays usable.  (The kernels themselves have no wait that a caller could hold up.)"""
import ctypes
import subprocess

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_a_wait_that_runs_out(tmp_path):
    import __graft_entry__
    from expert_cache_host_layer_gb300 import FT_ERR_TIMEOUT
    b = __graft_entry__._build_module()
    lib = str(tmp_path / "kv_waits.so")
    r = subprocess.run([b.nvcc(), *b.ARCH, *b.NVCC_FLAGS, "-shared", "-cudart", "static", "-o", lib,
                        b.ROOT + "/tests/kv_waits.cu"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    status = torch.zeros(2, dtype=torch.int32, device="cuda:0")
    result = torch.full((96,), 7, dtype=torch.int32, device="cuda:0")
    ns = torch.zeros(3, dtype=torch.int64, device="cuda:0")
    torch.cuda.synchronize()
    run = ctypes.CDLL(lib).kv_waits
    run.argtypes = [ctypes.c_void_p] * 3
    assert run(status.data_ptr(), result.data_ptr(), ns.data_ptr()) == 0
    assert status.tolist() == [FT_ERR_TIMEOUT, 0]                      # by the wait that ran out, not by the other
    assert result.tolist() == [0] * 64 + [1] * 32
    t0, t1, t2 = (t * 1e-9 for t in ns.tolist())
    assert 1.0 <= t0 < 3.0 and t0 - 0.01 < t1 < t0 + 1.0 and t2 < 0.5  # a second; ended by the first; at once
    assert int(torch.ones(5, device="cuda:0").sum()) == 5
