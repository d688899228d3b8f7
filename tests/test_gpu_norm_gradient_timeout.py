"""A wait of the layer norm gradient that runs out: the call ends by itself, the error word says so, nothing is stored
to dZ (in place or not), and the device goes on working."""

import pytest
import torch

from rows_common import DT, f64, lib, rows
from test_gpu_layer_norm import backward, check_backward, forward

pytestmark = pytest.mark.gpu


# one warp a row, several, one row a CTA, rows that are read twice; groups with and without partial sums
@pytest.mark.parametrize("M,K,gr,dt", [(300, 256, 0, "bf16"), (1000, 640, 0, "fp32"), (700, 4096, 300, "bf16"),
                                       (400, 8192, 0, "fp16"), (500, 12288, 0, "bf16"), (40, 16384, 0, "fp32"), (9, 1024, 1, "bf16")])
def test_it_ends_with_an_error_and_without_stores(M, K, gr, dt):
    L = lib()
    Z, dY = rows(1, M, K, DT[dt]), rows(2, M, K, DT[dt], 1e-2)
    _, stats = forward(Z, None, None)
    ws = torch.empty(L.svdq_layer_norm_backward_workspace_bytes(M, K, gr), dtype=torch.uint8, device="cuda")
    da, dc = torch.empty((2, -(-M // (gr or M)), K), device="cuda")
    dZ, before = torch.full_like(dY, 7.0), dY.clone()
    assert L.svdq_check_device_errors() == 0
    L.svdq_set_wait_limit_ns(2_000_000)
    try:
        for out in (dZ, dY):
            L.svdq_debug_stalled_layer_norm_backward(dY, Z, stats, out, da, dc, ws, group_rows=gr)
            assert L.svdq_check_device_errors() == 5  # SVDQ_ERR_TIMEOUT
            assert L.svdq_check_device_errors() == 0  # read and cleared
    finally:
        L.svdq_set_wait_limit_ns(2_000_000_000)
    assert bool((dZ == 7.0).all()) and torch.equal(dY, before)
    got = backward(dY, Z, stats, None, M, K, gr)
    check_backward(f64(Z), dY, stats, 1.0, got, M, gr, DT[dt])
    assert L.svdq_check_device_errors() == 0


def test_rows_that_are_read_without_a_wait_have_no_stalled_form():
    L = lib()
    M, K = 5, 1001
    x, stats = rows(3, M, K, torch.float32), torch.ones((M, 2), device="cuda")
    with pytest.raises(L.SvdqError, match="without a wait"):
        L.svdq_debug_stalled_layer_norm_backward(x, x, stats, torch.empty_like(x), None, None, None)
