"""Layer norm gradient of rows far from zero: xh = (z - mu) rstd carries the roundings of z - mu and of the product,
2 U of its own size (from a checkpoint code * scale - mu is rounded once, too), however large mu rstd is.

A column's sum over M rows is off by at most (M + 1) U of the absolute sum in any order; a row's sums as in the
other gradient tests: fewer than 72 roundings on any path.
"""

import numpy as np
import pytest
import torch

from rows_common import DT, U, ckpt_buffers, f64, half_step, lib, ref_backward, ref_decode, rows
from test_gpu_layer_norm import backward, forward

pytestmark = pytest.mark.gpu


def check(z, dY, stats, got, dtype):
    M = z.shape[0]
    st, dy = f64(stats), f64(dY)
    dz, da, dc, xh, g = ref_backward(z, dy, st[:, :1], st[:, 1:], 1.0, 0)
    rstd, d_xh = st[:, 1:], 2.01 * U * np.abs(xh)
    gm, gx = np.abs(g).mean(1, keepdims=True), np.abs(g * xh).mean(1, keepdims=True)
    near = rstd * (72 * U * (np.abs(g) + gm + np.abs(xh) * gx) + d_xh * gx
                   + np.abs(xh) * (np.abs(g) * d_xh).mean(1, keepdims=True))
    smallest = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert np.all(np.abs(f64(got[1])[0] - da[0]) <= ((M + 1) * U * np.abs(dy * xh) + np.abs(dy) * d_xh).sum(0))
    assert np.all(np.abs(f64(got[2])[0] - dc[0]) <= M * U * np.abs(dy).sum(0))
    assert np.all(np.abs(f64(got[0]) - dz) <= near + half_step(dtype) * (np.abs(dz) + near) + smallest)


@pytest.mark.parametrize("src", ["values", "int8", "e4m3"])
@pytest.mark.parametrize("M,K,dt", [(7, 256, "fp32"), (9, 640, "fp32"), (5, 1001, "fp32"), (3, 9000, "fp32"),
                                    (3, 12800, "fp32"), (6, 1024, "bf16"), (6, 1003, "fp16"), (3, 16384, "bf16")])
@pytest.mark.parametrize("mean", [100.0, 1000.0, 3.0e4])
def test_rows_with_a_mean_far_above_their_deviation(M, K, dt, mean, src):
    Z = rows(1, M, K, torch.float32, 1.0, outliers=False)
    Z = (Z + mean).to(DT[dt])
    dY = rows(2, M, K, DT[dt], 1e-2, outliers=False)
    z = f64(Z)
    ck = None
    if src != "values":
        ck = ckpt_buffers(M, K) + (src,)
        lib().svdq_ckpt8_encode(Z, ck[0], ck[1], src)
        z = ref_decode(ck[0].cpu().numpy(), ck[1].cpu().numpy(), src)
    # the statistics of the rows that the gradient reads; a deviation of 1 at least
    rstd = 1 / np.sqrt(z.var(1) + 1.0)
    stats = torch.from_numpy(np.stack([z.mean(1), rstd], 1)).float().cuda()
    check(z, dY, stats, backward(dY, None if ck else Z, stats, None, M, K, 0, ckpt=ck), DT[dt])


@pytest.mark.parametrize("src", ["values", "int8", "e4m3"])
@pytest.mark.parametrize("M,K,dt", [(5, 640, "fp32"), (5, 640, "bf16"), (4, 1001, "fp32"), (4, 12800, "bf16"), (3, 30, "fp16")])
@pytest.mark.parametrize("value", [0.0, 1.5, 96.0, 30720.0, 1.5 * 2.0 ** 120])
def test_rows_without_variance(M, K, dt, value, src):
    """xh is exactly 0: dscale is, and dZ = rstd (g - mean(g)); mu rstd may be beyond fp32's range."""
    if dt == "fp16" and value > 65504:
        pytest.skip("no fp16 value")
    Z = torch.full((M, K), value, dtype=DT[dt], device="cuda")
    dY = rows(3, M, K, DT[dt], 1e-2, outliers=False)
    stats = torch.tensor([[value, 316.2278]], device="cuda").repeat(M, 1)
    ck = None
    if src != "values":
        ck = ckpt_buffers(M, K) + (src,)
        lib().svdq_ckpt8_encode(Z, ck[0], ck[1], src)
        assert np.all(ref_decode(ck[0].cpu().numpy(), ck[1].cpu().numpy(), src) == value)
    got = backward(dY, None if ck else Z, stats, None, M, K, 0, ckpt=ck)
    assert bool((got[1] == 0).all())
    check(np.full((M, K), value), dY, stats, got, DT[dt])


def test_forward_and_gradient_of_an_off_centre_row_agree_on_xh():
    """dscale with dY = 1 in one row is the forward's fp32 output of that row, bit for bit."""
    K = 896
    Z = rows(4, 1, K, torch.float32, outliers=False) + 3.0e4
    Y, stats = forward(Z, None, None, eps=1e-5)
    _, da, _ = backward(torch.ones_like(Z), Z, stats, None, 1, K, 0)
    assert torch.equal(da, Y)
