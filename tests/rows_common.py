"""Helpers of the layer norm, checkpoint and low-rank gradient tests: float64 definitions and inputs."""

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24  # half a step of fp32, relative


def lib():
    import rank_outlier_gemm_b200 as L
    return L


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.double().cpu().numpy()


def rows(seed, M, K, dtype, scale=1.0, ld=None, outliers=True):
    """CUDA [M, K] of a wider allocation (ld elements between rows), unit normal with some large channels."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((M, ld or K), float("nan"), device="cuda", dtype=dtype)
    x = torch.randn((M, K), generator=g, device="cuda") * scale
    if outliers:
        x *= torch.where(torch.rand(K, generator=g, device="cuda") < 0.02, 20.0, 1.0)
    buf[:, :K] = x.to(dtype)
    return buf[:, :K]


def ckpt_buffers(M, K):
    return (torch.empty((M, K), dtype=torch.uint8, device="cuda"),
            torch.empty((M, -(-K // 32)), dtype=torch.uint8, device="cuda"))


E4M3 = np.array([(-1.0 if c & 128 else 1.0) * ((c & 7) / 8 * 2.0 ** -6 if not c & 120
                                               else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7))
                 for c in range(256)])
E4M3[[0x7F, 0xFF]] = np.nan


def code_values(codes, fmt):
    c = np.asarray(codes)
    return c.view(np.int8).astype(np.float64) if fmt == "int8" else E4M3[c]


def ref_encode(x, fmt):
    """(values of the codes, scale bytes) of float64 rows by the definition, group by group."""
    M, K = x.shape
    vals, scales = np.zeros((M, K)), np.zeros((M, -(-K // 32)), np.int64)
    mags = np.sort(E4M3[:127])
    for k in range(0, K, 32):
        g = x[:, k:k + 32]
        amax = np.max(np.abs(g), axis=1)
        ok = np.isfinite(amax)
        a = np.where(ok, amax, 0.0)
        b = np.zeros(M, np.int64)
        for byte in range(248 if fmt == "int8" else 246):  # the smallest exponent that holds the largest magnitude
            t = a / 2.0 ** (byte - 127)
            b += (t >= 127.5) if fmt == "int8" else (t > 448)
        v = np.where(ok[:, None], g, 0.0) / 2.0 ** (b - 127.0)[:, None]
        if fmt == "int8":
            q = np.clip(np.rint(v), -127, 127)
        else:  # nearest magnitude of the table, ties to the even code
            hi = np.clip(np.searchsorted(mags, np.abs(v)), 0, 126)
            lo = np.maximum(hi - 1, 0)
            dl, dh = np.abs(v) - mags[lo], mags[hi] - np.abs(v)
            pick = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
            q = np.copysign(mags[pick], v)
        vals[:, k:k + 32] = q
        scales[:, k // 32] = np.where(ok, b, 255)
    return vals, scales


def ref_decode(codes, scales, fmt):
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return code_values(codes, fmt) * np.repeat(s, 32, 1)[:, :codes.shape[1]]


def of_group(v, M, group_rows):
    return v[np.arange(M) // (group_rows or M)]


def ref_norm(z, eps):
    mu = z.mean(1, keepdims=True)
    return mu, 1 / np.sqrt(((z - mu) ** 2).mean(1, keepdims=True) + eps)


def ref_backward(z, dy, mu, rstd, m, group_rows):
    M = z.shape[0]
    xh = (z - mu) * rstd
    g = dy * m
    dz = rstd * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    first = np.arange(0, M, group_rows or M)
    return dz, np.add.reduceat(dy * xh, first, axis=0), np.add.reduceat(dy, first, axis=0), xh, g
