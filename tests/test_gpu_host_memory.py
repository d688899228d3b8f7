"""svdq_weights_from_codes without the host memory for its copies returns SVDQ_ERR_OOM (no C++ exception leaves the C
entry point) and the process goes on.  In a process of its own, whose address space is limited during the call."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = """
import resource
import numpy as np, torch
import rank_outlier_gemm_b200 as L
torch.zeros(1, device="cuda")
def call(N, K):
    return L.svdq_weights_from_codes(N, K, 0, 1.0, np.zeros((N, K // 2), np.uint8), np.full(N * K // 16, 0x38, np.uint8),
                                     np.ones(K, np.float32), None, None)
small = call(128, 64)
N, K = 65536, 16384   # scales of 64 MiB
args = [np.zeros((N, K // 2), np.uint8), np.full(N * K // 16, 0x38, np.uint8), np.ones(K, np.float32)]
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
soft, hard = resource.getrlimit(resource.RLIMIT_AS)
resource.setrlimit(resource.RLIMIT_AS, (used + (16 << 20), hard))
status = 0
try:
    L.svdq_weights_from_codes(N, K, 0, 1.0, *args, None, None)
except L.SvdqError as e:
    status = e.status
finally:
    resource.setrlimit(resource.RLIMIT_AS, (soft, hard))
assert status == 4, status   # SVDQ_ERR_OOM
del small
call(128, 64)
print("went on")
"""


def test_a_handle_that_does_not_fit():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "went on" in r.stdout, r.stderr[-2000:]
