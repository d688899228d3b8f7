"""Gradient of a low-rank factor, G = X^T S, against float64, from bf16 rows and from checkpoints.

The products of bf16 values are exact in fp32.  A warp adds at most 20 MMA results to one accumulator
(each off by up to 2^-22 of the absolute sum: the tensor cores truncate), 4 warps and the splits
follow with ordinary additions: 24 + splits steps, the splits at most M / 64.
"""

import numpy as np
import pytest
import torch

from rows_common import ckpt_buffers, f64, lib, ref_decode, rows

pytestmark = pytest.mark.gpu


def wgrad(X, S, ckpt=None):
    L = lib()
    M, r = S.shape
    K = ckpt[0].shape[1] if ckpt else X.shape[1]
    G = torch.full((K + 1, r), 5.0, device="cuda")
    nbytes = L.svdq_lowrank_wgrad_workspace_bytes(M, K, r)
    ws = torch.full((nbytes + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    L.svdq_lowrank_wgrad(None if ckpt else X, S, G[:K], ws[:nbytes], ckpt=ckpt)
    assert bool((ws[nbytes:] == 0x5A).all()) and bool((G[K:] == 5.0).all())
    return G[:K]


def check(G, x, s):
    ref, mag = x.T @ s, np.abs(x).T @ np.abs(s)
    steps = 24 + min(s.shape[0] / 64, 300)
    assert np.all(np.abs(f64(G) - ref) <= steps * 2.0 ** -22 * mag)


@pytest.mark.parametrize("src", ["values", "int8", "e4m3"])
@pytest.mark.parametrize("M,K,r", [(1, 16, 1), (2, 64, 8), (15, 48, 3), (17, 128, 16), (64, 80, 17), (65, 640, 32),
                                   (333, 208, 33), (500, 1152, 64), (129, 144, 65), (700, 96, 128), (4099, 1152, 16),
                                   (9000, 32, 48), (1300, 3200, 31)])
def test_values(M, K, r, src):
    X = rows(1, M, K, torch.bfloat16)
    S = rows(2, M, r, torch.bfloat16, 1e-3)
    if src == "values":
        check(wgrad(X, S), f64(X), f64(S))
        return
    ck = ckpt_buffers(M, K)
    lib().svdq_ckpt8_encode(X, ck[0], ck[1], src)
    check(wgrad(None, S, ck + (src,)), ref_decode(ck[0].cpu().numpy(), ck[1].cpu().numpy(), src), f64(S))


def test_repeatable_and_in_fp32_accuracy():
    M, K, r = 4608, 1280, 32
    X, S = rows(3, M, K, torch.bfloat16, outliers=False), rows(4, M, r, torch.bfloat16, outliers=False)
    G = wgrad(X, S)
    assert torch.equal(G, wgrad(X, S))
    ref = f64(X).T @ f64(S)
    # an fp32 sum of 4608 unit products: some 2^-24 sqrt(steps) of its own size; 1e-6 leaves a factor of about 4
    assert np.linalg.norm(f64(G) - ref) <= 1e-6 * np.linalg.norm(ref)


def test_it_is_the_branchs_derivative():
    """loss = sum dY (x A) B is linear in A and in B: its difference quotient is the gradient itself."""
    M, K, N, r = 200, 192, 160, 16
    rng = np.random.default_rng(5)
    X, dY = rows(6, M, K, torch.bfloat16, outliers=False), rows(7, M, N, torch.bfloat16, outliers=False)
    A, B = rng.standard_normal((K, r)) / 14, rng.standard_normal((r, N)) / 4
    S = torch.from_numpy(f64(dY) @ B.T).to(torch.bfloat16).cuda()
    T = torch.from_numpy(f64(X) @ A).to(torch.bfloat16).cuda()
    dA, dB = f64(wgrad(X, S)), f64(wgrad(dY, T)).T
    loss = lambda A, B: float(np.sum(f64(dY) * (f64(X) @ A @ B)))  # noqa: E731
    va, vb = rng.standard_normal(A.shape), rng.standard_normal(B.shape)
    # S and T are rounded to bf16 (2^-8 of each value): the products' sum is off by that times the root of
    # the sum of their squares, and 6 of those are never passed
    for grad, v, diff, x, s in ((dA, va, loss(A + va, B) - loss(A - va, B), f64(X), f64(S)),
                                (dB.T, vb.T, loss(A, B + vb) - loss(A, B - vb), f64(dY), f64(T))):
        spread = 2.0 ** -8 * np.sqrt(np.sum((x @ v) ** 2 * s ** 2))
        assert abs(np.sum(grad * v) - diff / 2) <= 6 * spread


def test_a_group_that_is_not_finite_stays_in_its_columns():
    M, K, r = 70, 128, 8
    X, S = rows(8, M, K, torch.bfloat16), rows(9, M, r, torch.bfloat16)
    X[13, 40] = float("inf")
    ck = ckpt_buffers(M, K)
    lib().svdq_ckpt8_encode(X, ck[0], ck[1], "int8")
    G = wgrad(None, S, ck + ("int8",))
    assert bool(G[32:64].isnan().all()) and bool(G[:32].isfinite().all()) and bool(G[64:].isfinite().all())


def test_captured():
    L = lib()
    M, K, r = 400, 320, 24
    X, S, G = rows(10, M, K, torch.bfloat16), rows(11, M, r, torch.bfloat16), torch.empty((K, r), device="cuda")
    ws = torch.empty(L.svdq_lowrank_wgrad_workspace_bytes(M, K, r), dtype=torch.uint8, device="cuda")
    L.svdq_lowrank_wgrad(X, S, G, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.svdq_lowrank_wgrad(X, S, G, ws)
    X.copy_(rows(12, M, K, torch.bfloat16))
    G.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check(G, f64(X), f64(S))
