"""Layer norm, its gradient and the 8-bit checkpoints against float64 definitions.

Tolerances count roundings.  A thread sums up to 32 values of a row, a warp adds 5 levels, a team 16
warps: fewer than 64 fp32 additions on any path, each off by U = 2^-24 of the absolute sum.  A result
of type t is rounded once, by at most half_step(t) of its value.
"""

import numpy as np
import pytest
import torch

from rows_common import (DT, U, ckpt_buffers, code_values, f64, half_step, lib, of_group, ref_backward, ref_decode,
                         ref_encode, ref_norm, rows)

pytestmark = pytest.mark.gpu

# M, K, group_rows, dtype, parameter dtype, plus_one, extra elements between rows
CASES = [
    (1, 1, 0, "fp32", "fp32", False, 0),
    (3, 7, 2, "bf16", "fp32", True, 0),
    (5, 64, 0, "bf16", "bf16", False, 0),
    (33, 640, 16, "bf16", "bf16", True, 0),
    (40, 1152, 20, "bf16", "fp32", False, 8),
    (17, 1001, 0, "fp32", "fp32", False, 0),
    (9, 1000, 4, "fp16", "fp16", True, 24),
    (70, 1280, 1, "fp16", "fp32", False, 0),
    (19, 1288, 6, "bf16", "fp16", False, 3),
    (12, 4096, 5, "fp32", "bf16", True, 0),
    (7, 5000, 3, "bf16", "bf16", False, 0),
    (6, 9001, 0, "fp16", "fp32", False, 1),
    (4, 12288, 2, "bf16", "bf16", True, 0),
    (3, 16384, 0, "fp32", "fp32", False, 0),
    (700, 96, 300, "bf16", "fp32", False, 0),
    (2500, 24, 0, "fp16", "fp32", True, 0),
]


def params(seed, M, K, group_rows, pdt, plus_one, stride=None):
    n = -(-M // (group_rows or M))
    scale = rows(seed, n, K, DT[pdt], 0.3, stride, outliers=False)
    if not plus_one:
        scale += 1
    return scale, rows(seed + 1, n, K, DT[pdt], 0.3, stride, outliers=False)


def forward(Z, scale, shift, eps=1e-6, **kw):
    L = lib()
    M, K = Z.shape
    Y = torch.full((M, Z.stride(0) if M > 1 else K), 7.0, device="cuda", dtype=Z.dtype)[:, :K]
    stats = torch.empty((M, 2), device="cuda")
    L.svdq_layer_norm(Z, scale, shift, Y, stats, eps, **kw)
    return Y, stats


def check_forward(Z, Y, stats, m, c, eps, dtype):
    z = f64(Z)
    mu, rstd = ref_norm(z, eps)
    xh = (z - mu) * rstd
    d_mu = 64 * U * np.abs(z).mean(1, keepdims=True)
    # relative error of rstd: half of the variance's, (d_mu rstd)^2 and the sum's roundings; 4 of its own
    d_rstd = 0.5 * ((d_mu * rstd) ** 2 + 68 * U) + 4 * U
    st = f64(stats)
    assert np.all(np.abs(st[:, :1] - mu) <= d_mu + U * np.abs(mu))
    assert np.all(np.abs(st[:, 1:] - rstd) <= rstd * d_rstd)
    ref = xh * m + c
    near = np.abs(m) * rstd * d_mu + np.abs(xh * m) * (d_rstd + 6 * U) + 2 * U * np.abs(c)
    y = f64(Y)
    smallest = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert np.all(np.abs(y - ref) <= near + half_step(dtype) * (np.abs(ref) + near) + smallest)


@pytest.mark.parametrize("M,K,gr,dt,pdt,plus_one,gap", CASES)
def test_forward(M, K, gr, dt, pdt, plus_one, gap):
    Z = rows(1, M, K, DT[dt], 1.0, K + gap)
    Z += 3.0  # a mean away from zero
    scale, shift = params(5, M, K, gr, pdt, plus_one)
    Y, stats = forward(Z, scale, shift, group_rows=gr, plus_one=plus_one)
    check_forward(Z, Y, stats, of_group(f64(scale), M, gr) + plus_one, of_group(f64(shift), M, gr), 1e-6, DT[dt])
    if gap and M > 1:  # what lies between the rows stays as it was
        assert bool((Y.as_strided((M - 1, gap), (Y.stride(0), 1), Y.storage_offset() + K) == 7.0).all())


def test_forward_without_parameters_in_place_and_views():
    M, K = 21, 768
    Z = rows(2, M, K, torch.bfloat16)
    Y, stats = forward(Z, None, None)
    check_forward(Z, Y, stats, 1.0, 0.0, 1e-6, torch.bfloat16)
    # scale and shift as slices of one wider tensor, as a modulation layer returns them
    mod = rows(3, 3, 6 * K, torch.bfloat16, 0.3, outliers=False)
    scale, shift = mod[:, K:2 * K], mod[:, :K]
    Y2, stats2 = forward(Z, scale, shift, group_rows=8, plus_one=True)
    check_forward(Z, Y2, stats2, of_group(f64(scale), M, 8) + 1, of_group(f64(shift), M, 8), 1e-6, torch.bfloat16)
    Zc = Z.clone()
    lib().svdq_layer_norm(Zc, scale, shift, Zc, None, 1e-6, group_rows=8, plus_one=True)
    assert torch.equal(Zc, Y2)


def test_rows_of_special_values():
    K = 640
    Z = rows(4, 6, K, torch.float32)
    Z[0] = 5.0              # no variance: rstd = 1 / sqrt(eps)
    Z[1, 17] = float("inf")
    Z[2, 600] = float("nan")
    Z[3] = 0.0
    Z[4] = 3.0e4 + torch.randn(K, device="cuda")  # a mean far above the deviation
    Y, stats = forward(Z, None, None, eps=1e-5)
    assert bool((Y[0] == 0).all()) and bool((Y[3] == 0).all())
    assert abs(float(stats[0, 1]) / 1e-5 ** -0.5 - 1) < 1e-6
    assert bool(Y[1].isnan().all()) and bool(Y[2].isnan().all())
    keep = [4, 5]
    check_forward(Z[keep], Y[keep], stats[keep], 1.0, 0.0, 1e-5, torch.float32)


def backward(dY, Z, stats, scale, M, K, gr, plus_one=False, ckpt=None, grads=True):
    L = lib()
    n = -(-M // (gr or M))
    dZ = torch.full((M, dY.stride(0) if M > 1 else K), 7.0, device="cuda", dtype=dY.dtype)[:, :K]
    da, dc = (torch.full((n, K), 9.0, device="cuda") for _ in range(2))
    nbytes = L.svdq_layer_norm_backward_workspace_bytes(M, K, gr)
    ws = torch.full((nbytes + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    L.svdq_layer_norm_backward(dY, Z, stats, scale, dZ, da if grads else None, dc if grads else None, ws[:nbytes],
                               group_rows=gr, plus_one=plus_one, ckpt=ckpt)
    assert bool((ws[nbytes:] == 0x5A).all())
    return dZ, da, dc


def check_backward(z, dY, stats, m, got, M, gr, dtype):
    st, dy = f64(stats), f64(dY)
    mu, rstd = st[:, :1], st[:, 1:]
    dz, da, dc, xh, g = ref_backward(z, dy, mu, rstd, m, gr)
    # xh carries 2 roundings, of z - mu and of the product: absolute 2 U (|z| + |mu|) rstd at most
    d_xh = 2 * U * (np.abs(z) + np.abs(mu)) * rstd
    gm, gx = np.abs(g).mean(1, keepdims=True), np.abs(g * xh).mean(1, keepdims=True)
    near = rstd * (72 * U * (np.abs(g) + gm + np.abs(xh) * gx) + d_xh * gx
                   + np.abs(xh) * (np.abs(g) * d_xh).mean(1, keepdims=True))
    smallest = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert np.all(np.abs(f64(got[0]) - dz) <= near + half_step(dtype) * (np.abs(dz) + near) + smallest)
    # additions on a column's path: a thread's rows (M / 296 or 4), 8 teams, 37 partial sums, 8 shares
    n = M / 296 + 64
    first = np.arange(0, M, gr or M)
    total = lambda v: np.add.reduceat(v, first, axis=0)  # noqa: E731
    assert np.all(np.abs(f64(got[1]) - da) <= n * U * total(np.abs(dy * xh)) + total(np.abs(dy) * d_xh))
    assert np.all(np.abs(f64(got[2]) - dc) <= n * U * total(np.abs(dy)))


@pytest.mark.parametrize("src", ["values", "int8", "e4m3"])
@pytest.mark.parametrize("M,K,gr,dt,pdt,plus_one,gap", CASES)
def test_backward(M, K, gr, dt, pdt, plus_one, gap, src):
    Z = rows(11, M, K, DT[dt], 1.0, K + gap)
    dY = rows(12, M, K, DT[dt], 1e-2, K + gap)
    scale, _ = params(5, M, K, gr, pdt, plus_one)
    _, stats = forward(Z, None, None)
    ck, z = None, f64(Z)
    if src != "values":
        ck = ckpt_buffers(M, K) + (src,)
        lib().svdq_ckpt8_encode(Z, ck[0], ck[1], src)
        z = ref_decode(ck[0].cpu().numpy(), ck[1].cpu().numpy(), src)
    got = backward(dY, None if ck else Z, stats, scale, M, K, gr, plus_one, ck)
    check_backward(z, dY, stats, of_group(f64(scale), M, gr) + plus_one, got, M, gr, DT[dt])
    if gap and M > 1:
        dZ = got[0]
        assert bool((dZ.as_strided((M - 1, gap), (dZ.stride(0), 1), dZ.storage_offset() + K) == 7.0).all())


def test_backward_is_the_forwards_derivative():
    """Differences of the float64 forward along random directions, in Z, scale and shift."""
    M, K, gr = 24, 320, 10
    Z = rows(21, M, K, torch.float32, outliers=False)
    dY = rows(22, M, K, torch.float32, 1.0, outliers=False)
    scale, shift = params(23, M, K, gr, "fp32", True)
    _, stats = forward(Z, scale, shift, eps=1e-5, group_rows=gr, plus_one=True)
    dZ, da, dc = backward(dY, Z, stats, scale, M, K, gr, True)
    z, dy, a, c = f64(Z), f64(dY), f64(scale), f64(shift)

    def loss(z, a, c):
        mu, rstd = ref_norm(z, 1e-5)
        return float(np.sum(dy * ((z - mu) * rstd * (1 + of_group(a, M, gr)) + of_group(c, M, gr))))

    rng = np.random.default_rng(3)
    vz, va, vc = rng.standard_normal(z.shape), rng.standard_normal(a.shape), rng.standard_normal(c.shape)
    h = 1e-5
    for grad, diff in ((np.sum(f64(dZ) * vz), loss(z + h * vz, a, c) - loss(z - h * vz, a, c)),
                       (np.sum(f64(da) * va), loss(z, a + h * va, c) - loss(z, a - h * va, c)),
                       (np.sum(f64(dc) * vc), loss(z, a, c + h * vc) - loss(z, a, c - h * vc))):
        # sums of 7680 products of unit normals (root 88), each gradient off by some 1e-6 of its size, and the
        # difference's own error h^2 (its third derivatives are of order one) and 1e-16 |loss| / h
        assert abs(grad - diff / (2 * h)) < 1e-3


def test_backward_without_parameter_gradients_in_place_and_repeatable():
    M, K = 600, 1152
    Z, dY = rows(31, M, K, torch.bfloat16), rows(32, M, K, torch.bfloat16, 1e-2)
    scale, shift = params(33, M, K, 0, "fp32", False)
    _, stats = forward(Z, scale, shift)
    dZ, da, dc = backward(dY, Z, stats, scale, M, K, 0)
    again = backward(dY, Z, stats, scale, M, K, 0)
    assert torch.equal(dZ, again[0]) and torch.equal(da, again[1]) and torch.equal(dc, again[2])
    only, _, _ = backward(dY, Z, stats, scale, M, K, 0, grads=False)
    assert torch.equal(dZ, only)
    L = lib()
    ws = torch.empty(L.svdq_layer_norm_backward_workspace_bytes(M, K, 0), dtype=torch.uint8, device="cuda")
    d2, da2 = dY.clone(), torch.empty_like(da)
    L.svdq_layer_norm_backward(d2, Z, stats, scale, d2, da2, None, ws)
    assert torch.equal(d2, dZ) and torch.equal(da2, da)


def test_a_row_that_is_not_finite_stays_in_its_group():
    M, K, gr = 12, 200, 4
    Z, dY = rows(41, M, K, torch.float32), rows(42, M, K, torch.float32)
    Z[5, 3] = float("nan")
    _, stats = forward(Z, None, None)
    dZ, da, dc = backward(dY, Z, stats, None, M, K, gr)
    assert bool(dZ[5].isnan().all())
    clean = [i for i in range(M) if i != 5]
    assert bool(dZ[clean].isfinite().all())
    assert bool(da[[0, 2]].isfinite().all()) and bool(da[1].isnan().all()) and bool(dc.isfinite().all())


# ------------------------------------------------------------------ checkpoints
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("M,K,dt,gap", [(1, 1, "fp32", 0), (3, 31, "bf16", 0), (5, 33, "fp16", 2), (4, 64, "bf16", 0),
                                        (9, 1000, "bf16", 0), (300, 1152, "bf16", 0), (7, 1280, "fp32", 8),
                                        (2, 20000, "fp16", 0), (65, 4096, "fp32", 0), (3, 40, "fp16", 1)])
def test_checkpoint_codes_and_values(M, K, dt, gap, fmt):
    L = lib()
    X = rows(51, M, K, DT[dt], 1.0, K + gap)
    if dt != "fp16" and M > 1:  # very large, very small and subnormal groups, a tie, zeros
        X[0, :K // 2] *= 1e30
        X[1, :K // 2] *= 1e-36
        X[1, K // 2:] = 0.0
    codes, scales = ckpt_buffers(M, K)
    L.svdq_ckpt8_encode(X, codes, scales, fmt)
    want, sb = ref_encode(f64(X), fmt)
    assert np.array_equal(scales.cpu().numpy(), sb)
    assert np.array_equal(code_values(codes.cpu().numpy(), fmt), want)
    for out in (DT[dt], torch.float32):
        back = torch.full((M, K + gap), 3.0, dtype=out, device="cuda")
        L.svdq_ckpt8_decode(codes, scales, back[:, :K], fmt)
        v = ref_decode(codes.cpu().numpy(), scales.cpu().numpy(), fmt)
        assert torch.equal(back[:, :K], torch.from_numpy(v).cuda().to(out))
        assert bool((back[:, K:] == 3.0).all())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_checkpoint_of_edges_and_special_values(fmt):
    L = lib()
    X = torch.zeros((6, 64), device="cuda")
    for i, top in enumerate((127.49999, 127.5, 448.0, 448.00003, 1.9921875, 3.4028234e38)):
        X[i, :32] = top * torch.linspace(-1, 1, 32, device="cuda")
    X[0, 40], X[1, 33], X[2, 63] = float("inf"), float("nan"), float("-inf")
    codes, scales = ckpt_buffers(6, 64)
    L.svdq_ckpt8_encode(X, codes, scales, fmt)
    want, sb = ref_encode(f64(X), fmt)
    assert np.array_equal(scales.cpu().numpy(), sb) and list(sb[:3, 1]) == [255] * 3
    assert np.array_equal(code_values(codes.cpu().numpy(), fmt), want)
    back = torch.empty((6, 64), device="cuda")
    L.svdq_ckpt8_decode(codes, scales, back, fmt)
    assert bool(back[:3, 32:].isnan().all()) and bool(back[:, :32].isfinite().all())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("M,K,dt", [(33, 640, "bf16"), (5, 1001, "fp32"), (9, 4096, "fp16"), (3, 12288, "bf16")])
def test_forward_writes_the_encoders_checkpoint(M, K, dt, fmt):
    Z = rows(61, M, K, DT[dt])
    Z[M // 2, K // 3] = float("inf")
    ck, alone = ckpt_buffers(M, K), ckpt_buffers(M, K)
    Y, stats = forward(Z, None, None, ckpt=ck + (fmt,))
    Y0, stats0 = forward(Z, None, None)
    lib().svdq_ckpt8_encode(Z, alone[0], alone[1], fmt)
    assert torch.equal(ck[0], alone[0]) and torch.equal(ck[1], alone[1])
    assert torch.equal(Y.view(torch.uint8), Y0.view(torch.uint8))
    assert torch.equal(stats.view(torch.int32), stats0.view(torch.int32))


def test_captured_and_on_another_stream():
    """Forward with checkpoint and backward from it, captured once and replayed on new values."""
    L = lib()
    M, K, gr = 96, 640, 40
    Z, dY = rows(71, M, K, torch.bfloat16), rows(72, M, K, torch.bfloat16)
    scale, shift = params(73, M, K, gr, "bf16", True)
    Y, dZ = torch.empty_like(Z), torch.empty_like(Z)
    stats, (da, dc) = torch.empty((M, 2), device="cuda"), torch.empty((2, 3, K), device="cuda")
    ck = ckpt_buffers(M, K)
    ws = torch.empty(L.svdq_layer_norm_backward_workspace_bytes(M, K, gr), dtype=torch.uint8, device="cuda")

    def step():
        L.svdq_layer_norm(Z, scale, shift, Y, stats, 1e-6, group_rows=gr, plus_one=True, ckpt=ck + ("int8",))
        L.svdq_layer_norm_backward(dY, None, stats, scale, dZ, da, dc, ws, group_rows=gr, plus_one=True,
                                   ckpt=ck + ("int8",))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    Z.copy_(rows(81, M, K, torch.bfloat16))
    dY.copy_(rows(82, M, K, torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in (Y, stats, dZ, da, dc, *ck)]
    step()
    for a, b in zip(replayed, (Y, stats, dZ, da, dc, *ck)):
        assert torch.equal(a, b)
