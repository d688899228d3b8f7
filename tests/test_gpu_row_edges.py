"""Layer norm, checkpoints and the low-rank gradient at odd places: rows more than 2^31 elements apart,
scales and parameters at any address, buffers that end with the last row, two calls at once."""

import numpy as np
import pytest
import torch

from rows_common import DT, ckpt_buffers, f64, lib, of_group, ref_decode, rows
from test_gpu_layer_norm import backward, check_backward, check_forward, forward, params
from test_gpu_lowrank_wgrad import check, wgrad
from test_gpu_w4a16 import check as check_w4a16
from test_gpu_w4a16 import layer, run, tokens

pytestmark = pytest.mark.gpu


def test_rows_far_apart():
    """Element offsets beyond 2^31 (and byte offsets beyond 2^32)."""
    K, ld = 384, (1 << 31) // 2 + 4096
    big = torch.zeros(2 * ld + K, dtype=torch.bfloat16, device="cuda")
    Z = big.as_strided((3, K), (ld, 1))
    Z.copy_(rows(1, 3, K, torch.bfloat16))
    L = lib()
    Y, stats = torch.empty((3, K), dtype=torch.bfloat16, device="cuda"), torch.empty((3, 2), device="cuda")
    ck, alone = ckpt_buffers(3, K), ckpt_buffers(3, K)
    L.svdq_layer_norm(Z, None, None, Y, stats, 1e-6, ckpt=ck + ("int8",))
    check_forward(Z, Y, stats, 1.0, 0.0, 1e-6, torch.bfloat16)
    L.svdq_ckpt8_encode(Z, alone[0], alone[1], "int8")
    assert torch.equal(ck[0], alone[0]) and torch.equal(ck[1], alone[1])
    dY = rows(2, 3, K, torch.bfloat16)
    ws = torch.empty(L.svdq_layer_norm_backward_workspace_bytes(3, K, 0), dtype=torch.uint8, device="cuda")
    dZ, da, dc = torch.empty_like(dY), torch.empty((1, K), device="cuda"), torch.empty((1, K), device="cuda")
    L.svdq_layer_norm_backward(dY, Z, stats, None, dZ, da, dc, ws)
    check_backward(f64(Z), dY, stats, 1.0, (dZ, da, dc), 3, 0, torch.bfloat16)
    L.svdq_ckpt8_decode(ck[0], ck[1], Z, "int8")
    assert torch.equal(Z.double().cpu(), torch.from_numpy(ref_decode(ck[0].cpu().numpy(), ck[1].cpu().numpy(), "int8")))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_more_rows_than_are_at_work(dt):
    """The forward asks for rows ahead of the ones at work: of a view with gaps, in place, to the last row."""
    M, K, gr = 1301, 2056, 100
    Z = rows(6, M, K, DT[dt], 1.0, K + 24)
    before = Z.clone()
    scale, shift = params(7, M, K, gr, "fp32", True)
    L = lib()
    stats = torch.empty((M, 2), device="cuda")
    L.svdq_layer_norm(Z, scale, shift, Z, stats, 1e-6, group_rows=gr, plus_one=True)
    check_forward(before, Z, stats, of_group(f64(scale), M, gr) + 1, of_group(f64(shift), M, gr), 1e-6, DT[dt])


def test_a_checkpoint_of_more_than_2_to_31_values():
    M, K = 70000, 31008
    L = lib()
    X = torch.empty((M, K), dtype=torch.bfloat16, device="cuda").fill_(0.5)
    tail = rows(3, 64, K, torch.bfloat16)
    X[-64:] = tail
    codes, scales = ckpt_buffers(M, K)
    L.svdq_ckpt8_encode(X, codes, scales, "e4m3")
    small = ckpt_buffers(64, K)
    L.svdq_ckpt8_encode(tail, small[0], small[1], "e4m3")
    assert torch.equal(codes[-64:], small[0]) and torch.equal(scales[-64:], small[1])
    X.zero_()
    L.svdq_ckpt8_decode(codes, scales, X, "e4m3")
    assert bool((X[:-64:4999] == 0.5).all()) and float(X[-1].float().abs().max()) > 1.0


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
@pytest.mark.parametrize("M,K", [(5, 64), (37, 672), (64, 48), (300, 1040), (1, 16)])
def test_scales_at_any_address(M, K, shift):
    """The scale bytes end with their allocation's last byte and begin anywhere."""
    X = rows(4, M, K, torch.bfloat16)
    codes, _ = ckpt_buffers(M, K)
    n = M * -(-K // 32)
    scales = torch.full((n + shift,), 0xEE, dtype=torch.uint8, device="cuda")[shift:].view(M, -1)
    lib().svdq_ckpt8_encode(X, codes, scales, "int8")
    z = ref_decode(codes.cpu().numpy(), scales.cpu().numpy(), "int8")
    dY, (_, stats) = rows(5, M, K, torch.bfloat16, 1e-2), forward(X, None, None)
    scale, _ = params(6, M, K, 16, "fp32", True)
    got = backward(dY, None, stats, scale, M, K, 16, True, (codes, scales, "int8"))
    check_backward(z, dY, stats, of_group(f64(scale), M, 16) + 1, got, M, 16, torch.bfloat16)
    S = rows(7, M, 24, torch.bfloat16)
    check(wgrad(None, S, (codes, scales, "int8")), z, f64(S))


@pytest.mark.parametrize("dt,pdt,K,at", [("bf16", "bf16", 640, 1), ("fp32", "fp16", 256, 3), ("fp16", "fp32", 1153, 2),
                                         ("bf16", "fp32", 4096, 1)])
def test_parameters_and_rows_at_odd_elements(dt, pdt, K, at):
    M, gr = 45, 20
    wide = rows(8, 3, 2 * K + 7, DT[pdt], 0.3, outliers=False)
    scale, shift = wide[:, at:at + K], wide[:, K + at:2 * K + at]
    Z = rows(9, M, K + 5, DT[dt])[:, at:at + K]
    Y, stats = forward(Z, scale, shift, group_rows=gr, plus_one=True)
    check_forward(Z, Y, stats, of_group(f64(scale), M, gr) + 1, of_group(f64(shift), M, gr), 1e-6, DT[dt])
    dY = rows(10, M, K + 3, DT[dt], 1e-2)[:, 1:1 + K]
    got = backward(dY, Z, stats, scale, M, K, gr, True)
    check_backward(f64(Z), dY, stats, of_group(f64(scale), M, gr) + 1, got, M, gr, DT[dt])


def test_two_calls_at_once():
    L = lib()
    M, K = 1500, 1152
    streams = [torch.cuda.Stream() for _ in range(2)]
    data = []
    for i in range(2):
        Z, dY = rows(20 + i, M, K, torch.bfloat16), rows(30 + i, M, K, torch.bfloat16)
        _, stats = forward(Z, None, None)
        data.append(dict(Z=Z, dY=dY, stats=stats, dZ=torch.empty_like(Z), da=torch.empty((1, K), device="cuda"),
                         dc=torch.empty((1, K), device="cuda"), S=rows(40 + i, M, 16, torch.bfloat16),
                         G=torch.empty((K, 16), device="cuda"),
                         ws=torch.empty(L.svdq_layer_norm_backward_workspace_bytes(M, K), dtype=torch.uint8, device="cuda"),
                         ws2=torch.empty(L.svdq_lowrank_wgrad_workspace_bytes(M, K, 16), dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, d in zip(streams, data):
            L.svdq_layer_norm_backward(d["dY"], d["Z"], d["stats"], None, d["dZ"], d["da"], d["dc"], d["ws"], stream=s)
            L.svdq_lowrank_wgrad(d["Z"], d["S"], d["G"], d["ws2"], stream=s)
    torch.cuda.synchronize()
    for d in data:
        check_backward(f64(d["Z"]), d["dY"], d["stats"], 1.0, (d["dZ"], d["da"], d["dc"]), M, 0, torch.bfloat16)
        check(d["G"], f64(d["Z"]), f64(d["S"]))


@pytest.mark.parametrize("fmt", ["nvfp4", "int4"])
def test_few_token_layer_of_a_very_long_k(fmt):
    w, ref = layer(12, 48, 20544, 24, fmt)
    X = tokens(13, 3, 20544)
    check_w4a16(run(w, X), X, ref)


def test_tall_gradient():
    """More rows than one accumulator takes: several parts, the last one cut."""
    M, K, r = 40007, 48, 20
    X, S = rows(14, M, K, torch.bfloat16), rows(15, M, r, torch.bfloat16, 1e-2)
    check(wgrad(X, S), f64(X), f64(S))
    ck = ckpt_buffers(M, K)
    lib().svdq_ckpt8_encode(X, ck[0], ck[1], "e4m3")
    G = wgrad(None, S, ck + ("e4m3",))
    check(G, ref_decode(ck[0].cpu().numpy(), ck[1].cpu().numpy(), "e4m3"), f64(S))
    assert np.isfinite(f64(G)).all()
