"""The kernels' bounded waits keep their limit in time: a barrier that nothing
arrives at, on a probe of one CTA built from the kernels' own header."""
import ctypes
import os
import subprocess

import pytest
import torch

from sparse_linear_hybrid_b200 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("probe") / "wait_probe.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "wait_probe.cu")
    subprocess.run([build.NVCC, *build.FLAGS, f"-I{build.CSRC}", "-shared", "-o", lib, src], check=True, timeout=300)
    fn = ctypes.CDLL(lib).wait_probe_run
    fn.argtypes = [ctypes.c_uint64, ctypes.c_void_p]
    return fn


@pytest.mark.parametrize("limit_ms", [0, 1, 20, 100])
def test_a_wait_ends_at_its_limit(probe, limit_ms):
    """A warp counts polls of 128 ns at most (a sleep of 40 ns at most and the look at the barrier, some 50 cycles), of
    which each takes a tenth of that or more; one thread reads the timer.  1 ms more than the limit covers the first,
    blocking look and the timer's steps."""
    out = torch.full((6,), 99, dtype=torch.int64, device="cuda")
    assert probe(limit_ms * 1_000_000, out.data_ptr()) == 0
    ok, first, later_ok, later, one_ok, one = out.tolist()
    assert (ok, later_ok, one_ok) == (0, 0, 0)
    assert limit_ms * 1e5 <= first <= limit_ms * 1e6 + 1e6
    assert limit_ms * 1e6 <= one <= limit_ms * 1e6 + 1e6
    assert later <= 1e6  # a lane that has given up only looks
