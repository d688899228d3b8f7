"""The few-token layer with 16-bit activations against float64 on the handle's exported weights.

Activations enter with 22 bits (2^-22 of each product) and a floor of 2^-38 of the token's largest;
a sum runs over at most K / 128 MMA results per warp step group (each off by up to 2^-22 of the absolute
sum) and 8 warps; the branch's T and its up-projection are fp32 sums of r_pad and K / 16 terms.  Y is
rounded to bf16 once (2^-8).
"""

import numpy as np
import pytest
import torch

from oracle import codec as OC
from oracle.formats import e2m1_decode, e4m3_decode
from rows_common import lib
from synth import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def layer(seed, N, K, rank, fmt, bias=True):
    """A handle made from a random residual, and its weights in float64: (R / alpha_w, L1', L2, inv_lam, bias)."""
    L = lib()
    rng = np.random.default_rng(seed)
    R = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    inv = (2.0 ** rng.uniform(-3, 1, K)).astype(np.float32)
    L1 = f32_to_bf16_bits((rng.standard_normal((K, rank)) / np.sqrt(K)).astype(np.float32)) if rank else None
    L2 = f32_to_bf16_bits((rng.standard_normal((rank, N)) * 0.05).astype(np.float32)) if rank else None
    b = (rng.standard_normal(N) * 0.1).astype(np.float32) if bias else None
    w = L.svdq_weights_from_factors(N, K, rank, inv, L1, L2, R, b, fmt=fmt)
    return w, weights(w)


def weights(w):
    e = lib().svdq_weights_export(w)
    N, K = e["N"], e["K"]
    if e["format"] == "nvfp4":
        c = e["codes"]
        q = e2m1_decode(np.stack([c & 15, c >> 4], 2).reshape(N, K))
        s = e4m3_decode(OC.atoms_to_scales(e["sf"], N, K // 16))
        W = q * np.repeat(s, 16, 1)
    else:
        v = e["codes"].reshape(N, K // 8, 4)
        q = np.zeros((N, K // 8, 8))
        for byte, (a, b) in enumerate(((0, 2), (4, 6), (1, 3), (5, 7))):
            q[:, :, a], q[:, :, b] = (v[:, :, byte] & 15), v[:, :, byte] >> 4
        q = np.where(q >= 8, q - 16, q).reshape(N, K)
        s = bf16_bits_to_f32(e["sf"].view(np.uint16)).reshape(K // 64, -1)[:, :N].T.astype(np.float64)
        W = q * np.repeat(s, 64, 1)
    f = lambda v: bf16_bits_to_f32(v).astype(np.float64)  # noqa: E731
    return (W * e["alpha_w"], f(e["L1p"]), f(e["L2"]), e["inv_lam"].astype(np.float64), e["bias"].astype(np.float64))


def tokens(seed, M, K, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((M, K), generator=g, device="cuda") * scale
    x *= torch.where(torch.rand(K, generator=g, device="cuda") < 0.02, 30.0, 1.0)
    return x.to(torch.bfloat16)


def run(w, X):
    L = lib()
    M = X.shape[0]
    Y = torch.full((M + 1, w.N), 9.0, dtype=torch.bfloat16, device="cuda")
    n = L.svdq_linear_w4a16_workspace_bytes(w, M)
    ws = torch.full((n + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    L.svdq_linear_w4a16(w, X, Y[:M], ws[:n])
    assert bool((ws[n:] == 0x5A).all()) and bool((Y[M:] == 9.0).all())
    return Y[:M]


def check(Y, X, ref_weights):
    W, L1, L2, inv, b = ref_weights
    x = X.double().cpu().numpy()
    xh = x * inv
    T = x @ L1
    ref = xh @ W.T + T @ L2 + b
    K = x.shape[1]
    mag = np.abs(xh) @ np.abs(W).T + (np.abs(x) @ np.abs(L1)) @ np.abs(L2) + np.abs(b)
    floor = np.max(np.abs(xh), axis=1, keepdims=True) * 2.0 ** -38 * np.abs(W).sum(1)
    near = (K / 128 + 32) * 2.0 ** -22 * mag + floor
    y = Y.double().cpu().numpy()
    assert np.all(np.abs(y - ref) <= near + 2.0 ** -8 * (np.abs(ref) + near))


@pytest.mark.parametrize("fmt", ["nvfp4", "int4"])
@pytest.mark.parametrize("M,K,N,rank", [(1, 64, 16, 0), (1, 640, 640, 32), (2, 192, 48, 5), (3, 1152, 144, 16),
                                        (4, 128, 272, 40), (5, 1088, 528, 64), (8, 2048, 256, 128), (9, 320, 1040, 32),
                                        (13, 4608, 96, 16), (16, 1280, 640, 48), (16, 10240, 112, 0), (1, 12288, 160, 32)])
def test_values(M, K, N, rank, fmt):
    w, ref = layer(M + K + N, N, K, rank, fmt)
    X = tokens(7, M, K)
    check(run(w, X), X, ref)


@pytest.mark.parametrize("fmt", ["nvfp4", "int4"])
@pytest.mark.parametrize("scale", [1e-37, 1e-20, 1e-4, 1e4, 1e20, 1e34])
def test_any_range_of_activations(fmt, scale):
    w, ref = layer(3, 64, 256, 16, fmt, bias=False)
    X = tokens(8, 3, 256, scale)
    W, L1, L2, inv, b = ref
    if scale > 1e30:  # away from the largest bf16
        X = X.clamp(-1e36, 1e36)
    y, x = run(w, X).double().cpu().numpy(), X.double().cpu().numpy()
    want = (x * inv) @ W.T + (x @ L1) @ L2
    mag = np.abs(x * inv) @ np.abs(W).T + (np.abs(x) @ np.abs(L1)) @ np.abs(L2)
    # below 2^-126 fp32 keeps absolute steps of 2^-149 and bf16 of 2^-133
    assert np.all(np.abs(y - want) <= 34 * 2.0 ** -22 * mag + 2.0 ** -8 * np.abs(want) + 256 * 2.0 ** -133)


@pytest.mark.parametrize("fmt", ["nvfp4", "int4"])
def test_a_tokens_result_is_its_own(fmt):
    """Tokens do not depend on their company (as many columns of a tile as they need), and calls repeat."""
    w, _ = layer(4, 336, 832, 32, fmt)
    X = tokens(9, 16, 832)
    all16 = run(w, X)
    assert torch.equal(all16, run(w, X))
    for m in (0, 3, 4, 8, 15):
        assert torch.equal(run(w, X[m:m + 1].contiguous())[0], all16[m])
    bad = X.clone()
    bad[2, 5], bad[6, 0] = float("nan"), float("inf")
    Y = run(w, bad)
    keep = [m for m in range(16) if m not in (2, 6)]
    assert torch.equal(Y[keep], all16[keep])
    assert bool(Y[2].isnan().all()) and not bool(Y[6].isfinite().any())


@pytest.mark.parametrize("fmt", ["nvfp4", "int4"])
def test_handle_from_codes_is_the_exported_one(fmt):
    """svdq_weights_from_codes(export) gives the same handle, for this layer and for the W4A4 one, LoRA included."""
    L = lib()
    N, K = 272, 320
    w, _ = layer(5, N, K, 24, fmt)
    rng = np.random.default_rng(6)
    L.svdq_attach_lora(w, f32_to_bf16_bits(rng.standard_normal((K, 8)).astype(np.float32) * 0.1),
                       f32_to_bf16_bits(rng.standard_normal((8, N)).astype(np.float32) * 0.1), 0.5)
    e = L.svdq_weights_export(w)
    sf = e["sf"].copy()  # the padding rows may hold anything
    if fmt == "nvfp4":
        sf[OC.scales_to_atoms(np.ones((N, K // 16), np.uint8)) == 0] = 0x7F
    else:
        sf.view(np.uint16).reshape(K // 64, -1)[:, N:] = 0xFFFF
    assert not np.array_equal(sf, e["sf"])
    w2 = L.svdq_weights_from_codes(N, K, e["rank"], e["alpha_w"], e["codes"], sf, e["inv_lam"], e["L1p"], e["L2"],
                                   e["bias"], fmt=fmt)
    assert w2.info == w.info
    e2 = L.svdq_weights_export(w2)
    for key in ("codes", "sf", "L1p", "L2", "inv_lam", "bias"):
        assert np.array_equal(e[key], e2[key]), key
    X = tokens(10, 7, K)
    assert torch.equal(run(w, X), run(w2, X))
    check(run(w, X), X, weights(w2))
    assert torch.equal(L.linear(w, X), L.linear(w2, X))
    assert L.svdq_check_device_errors() == 0


def test_captured_and_on_two_streams():
    L = lib()
    w, ref = layer(11, 400, 640, 32, "nvfp4")
    X = tokens(12, 6, 640)
    Y = torch.empty((6, 400), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(L.svdq_linear_w4a16_workspace_bytes(w, 6), dtype=torch.uint8, device="cuda")
    L.svdq_linear_w4a16(w, X, Y, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.svdq_linear_w4a16(w, X, Y, ws)
        L.svdq_linear_w4a16(w, X, Y, ws)  # the workspace is free again once the call's kernels are done
    X.copy_(tokens(13, 6, 640))
    graph.replay()
    torch.cuda.synchronize()
    check(Y, X, ref)
    streams = [torch.cuda.Stream() for _ in range(2)]
    xs = [tokens(20 + i, 5, 640) for i in range(2)]
    outs = [torch.empty((5, 400), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    spaces = [torch.empty_like(ws) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            L.svdq_linear_w4a16(w, xs[i], outs[i], spaces[i], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        check(outs[i], xs[i], ref)
