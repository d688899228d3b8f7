"""Measured cases of the few-token 4-bit product, the layer norm with its gradient, the 8-bit
activation checkpoints and the low-rank factor's gradient.

``run`` computes a case in elementary torch operations in 32 bits (``own`` false) or by the
library's entry points (``own`` true), from the same ``prepare``d inputs; ``exact`` computes it
from the definition in 64 bits.  The operators:

* ``gemv``: the layer applied to 1..16 tokens with 16-bit activations and 4-bit weights,
  Y = bf16(alpha_w * (X * inv_lam) deq(Q)^T + (X L1') L2 + b); NVFP4 (E2M1 codes, an E4M3 scale
  per 16) or INT4 (codes -7..7, a bf16 scale per 64).
* ``norm``: Y = (z - mu) * rstd * m + shift with m = scale or 1 + scale, one (scale, shift)
  vector per group of consecutive rows; gives Y, the row statistics (mu, rstd) and, on request,
  an 8-bit checkpoint of Z.
* ``norm_bwd``: its gradient from Z or from the checkpoint: with xh = (z - mu) * rstd and
  g = dY * m, dZ = rstd * (g - mean(g) - xh * mean(g * xh)), dscale = sum dY * xh and
  dshift = sum dY over each group's rows.
* ``encode`` / ``decode``: the checkpoint format: 8-bit codes (integers -127..127, or E4M3) and
  one power-of-two scale byte (exponent + 127; 0xFF marks a group with a NaN or an infinity) per
  32 consecutive values of a row; the exponent is the smallest at which the group's largest
  magnitude does not leave the codes' range.
* ``wgrad``: G = X^T S in fp32, the gradient of a low-rank factor (K x r), X bf16 or a checkpoint.
"""

import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GROUP = 32  # values per scale of the 8-bit checkpoint


def listed():
    return [
        # one token through an attention projection of a 640-wide block: a call's fixed cost
        {"name": "gemv_nvfp4_m1_640x640", "op": "gemv", "fmt": "nvfp4", "M": 1, "K": 640, "N": 640, "rank": 32},
        # the modulation layer of one image: six vectors of 4096 channels from one embedding
        {"name": "gemv_nvfp4_m1_4096x24576", "op": "gemv", "fmt": "nvfp4", "M": 1, "K": 4096, "N": 24576, "rank": 32},
        # INT4, a few images at once, a LoRA of rank 16 on the branch (32 + 16)
        {"name": "gemv_int4_m5_1280x10240", "op": "gemv", "fmt": "int4", "M": 5, "K": 1280, "N": 10240, "rank": 48},
        # the most tokens it takes, few outputs over a long K
        {"name": "gemv_nvfp4_m16_10240x1280", "op": "gemv", "fmt": "nvfp4", "M": 16, "K": 10240, "N": 1280, "rank": 32},
        # adaLN ahead of an attention, two images, keeping the checkpoint for the backward pass
        {"name": "norm_bf16_4096x1152_ckpt", "op": "norm", "dtype": "bf16", "pdtype": "bf16", "M": 4096, "K": 1152,
         "rows": 2048, "plus_one": True, "ckpt": "int8"},
        # a handful of tokens, an odd width, fp32: a call's fixed cost
        {"name": "norm_fp32_77x1001", "op": "norm", "dtype": "fp32", "pdtype": "fp32", "M": 77, "K": 1001,
         "rows": 0, "plus_one": False, "ckpt": ""},
        # plain layer norm over all tokens of a 640-wide block: the longest reduction over rows
        {"name": "norm_bwd_bf16_8192x640", "op": "norm_bwd", "dtype": "bf16", "pdtype": "fp32", "M": 8192, "K": 640,
         "rows": 0, "plus_one": False, "ckpt": ""},
        # adaLN from the checkpoint, a wide model, four images of unlike length (the last is short)
        {"name": "norm_bwd_bf16_4500x4096_ckpt", "op": "norm_bwd", "dtype": "bf16", "pdtype": "bf16", "M": 4500,
         "K": 4096, "rows": 1152, "plus_one": True, "ckpt": "int8"},
        # the checkpoint of the widest activation (the second MLP projection's input)
        {"name": "encode_int8_bf16_4608x12288", "op": "encode", "dtype": "bf16", "M": 4608, "K": 12288, "ckpt": "int8"},
        # a checkpoint read back
        {"name": "decode_e4m3_fp16_2048x1280", "op": "decode", "dtype": "fp16", "M": 2048, "K": 1280, "ckpt": "e4m3"},
        # gradient of the down factor from the checkpoint, the widest layer
        {"name": "wgrad_int8_4608x12288_r32", "op": "wgrad", "M": 4608, "K": 12288, "rank": 32, "ckpt": "int8"},
        # gradient of the up factor from bf16 rows, an odd number of tokens
        {"name": "wgrad_bf16_4099x1152_r16", "op": "wgrad", "M": 4099, "K": 1152, "rank": 16, "ckpt": ""},
    ]


def _log(rng, lo, hi, step=1):
    """An integer spread over the logarithm of [lo, hi], a multiple of step."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["gemv", "gemv", "norm", "norm_bwd", "norm_bwd", "encode", "decode", "wgrad", "wgrad"])
    if op == "gemv":
        K = _log(rng, 128, 12288, 64)
        N = min(_log(rng, 128, 24576, 16), 4096 * 24576 // K // 16 * 16)
        return {"op": op, "fmt": rng.choice(["nvfp4", "int4"]), "M": rng.randint(1, 16), "K": K, "N": N,
                "rank": rng.choice([0, 16, 32, 40, 64, 128])}
    M = _log(rng, 16, 8192)
    K = min(_log(rng, 64, 12288, rng.choice([1, 8, 64])), 4608 * 12288 // M)
    ckpt = rng.choice(["int8", "e4m3"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("encode", "decode"):
        return {"op": op, "dtype": dtype, "M": M, "K": K, "ckpt": ckpt}
    if op == "wgrad":
        return {"op": op, "M": M, "K": max(64, K // 16 * 16), "rank": rng.choice([8, 16, 24, 32, 64, 128]),
                "ckpt": rng.choice(["", ckpt])}
    return {"op": op, "dtype": dtype, "pdtype": rng.choice([dtype, "fp32"]), "M": M, "K": K,
            "rows": rng.choice([0, rng.randint(1, M), max(1, M // 4)]), "plus_one": rng.random() < 0.5,
            "ckpt": rng.choice(["", ckpt])}


def _binding():
    import rank_outlier_gemm_b200 as svdq

    return svdq


def _atoms(sf):
    """E4M3 bytes [N, K/16] in the block-scale layout of 128-row x 4-column atoms."""
    N, G = sf.shape
    n = -(-N // 128) * 128
    full = torch.zeros((n, G), dtype=torch.uint8, device=sf.device)
    full[:N] = sf
    return full.view(n // 128, 4, 32, G // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _activations(g, M, K, dtype):
    """Unit normal values with 1 % of the channels 30 times larger, as a model's activations have them."""
    x = torch.randn((M, K), generator=g, device="cuda")
    x *= torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 30.0, 1.0)
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}

    def normal(shape, std, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    op, M, K = case["op"], case["M"], case["K"]
    if op == "gemv":
        N, r = case["N"], case["rank"]
        s["X"] = _activations(g, M, K, torch.bfloat16)
        s["inv_lam"] = torch.exp2(torch.rand(K, generator=g, device="cuda") * 4 - 3)
        s["L1"] = normal((K, r), K ** -0.5, torch.bfloat16)
        s["L2"] = normal((r, N), 0.02, torch.bfloat16)
        s["bias"] = normal((N,), 0.01)
        if case["fmt"] == "nvfp4":
            s["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
            s["sf"] = (32 + 416 * torch.rand((N, K // 16), generator=g, device="cuda")).to(torch.float8_e4m3fn)
            s["alpha"] = 2.0 ** -15  # weights of about 0.02
        else:
            nib = torch.randint(-7, 8, (N, K // 8, 8), generator=g, device="cuda").to(torch.uint8) & 15
            s["codes"] = (nib[..., 0::2] | nib[..., 1::2] << 4).view(N, K // 2)
            s["sf"] = (0.002 + 0.006 * torch.rand((N, K // 64), generator=g, device="cuda")).to(torch.bfloat16)
            s["alpha"] = 1.0
        if own:
            B = _binding()
            if case["fmt"] == "nvfp4":
                sf = _atoms(s["sf"].view(torch.uint8)).cpu().numpy()
            else:
                sf = torch.zeros((K // 64, -(-N // 256) * 256), dtype=torch.bfloat16, device="cuda")
                sf[:, :N] = s["sf"].T
                sf = sf.cpu().view(torch.int16).numpy().view(np.uint8).reshape(-1)
            s["w"] = B.svdq_weights_from_codes(N, K, r, s["alpha"], s["codes"].cpu().numpy(), sf, s["inv_lam"].cpu(),
                                               s["L1"].cpu(), s["L2"].cpu(), s["bias"].cpu(), fmt=case["fmt"])
            s["Y"] = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
            s["ws"] = torch.empty(B.svdq_linear_w4a16_workspace_bytes(s["w"], M), dtype=torch.uint8, device="cuda")
        return s

    if op == "wgrad":
        X = _activations(g, M, K, torch.bfloat16)
        s["S"] = normal((M, case["rank"]), 1e-3, torch.bfloat16)
        s["X"] = _encode(X.float(), case["ckpt"]) if case["ckpt"] else X
        if own:
            B = _binding()
            s["G"] = torch.empty((K, case["rank"]), device="cuda")
            s["ws"] = torch.empty(B.svdq_lowrank_wgrad_workspace_bytes(M, K, case["rank"]), dtype=torch.uint8,
                                  device="cuda")
        return s

    dtype = DTYPES[case["dtype"]]
    Z = _activations(g, M, K, dtype)
    if op == "encode":
        s["Z"] = Z
        if own:
            s["codes"], s["scales"] = _ckpt_buffers(M, K)
        return s
    if op == "decode":
        s["ck"] = _encode(Z.float(), case["ckpt"])
        if own:
            s["out"] = torch.empty((M, K), dtype=dtype, device="cuda")
        return s

    pdtype = DTYPES[case["pdtype"]]
    rows = case["rows"] or M
    groups = -(-M // rows)
    s["scale"] = normal((groups, K), 0.2, pdtype) if case["plus_one"] else (1 + normal((groups, K), 0.2)).to(pdtype)
    s["shift"] = normal((groups, K), 0.2, pdtype)
    s["Z"] = Z
    if op == "norm_bwd":
        z = Z.double()
        mu = z.mean(1)
        s["stats"] = torch.stack([mu, 1 / ((z - mu[:, None]).square().mean(1) + 1e-6).sqrt()], 1).float()
        s["dY"] = normal((M, K), 1e-2, dtype)
        if case["ckpt"]:
            s["Z"] = _encode(Z.float(), case["ckpt"])
    if own:
        B = _binding()
        if op == "norm":
            s["Y"], s["stats"] = torch.empty_like(Z), torch.empty((M, 2), device="cuda")
            s["ck"] = _ckpt_buffers(M, K) + (case["ckpt"],) if case["ckpt"] else None
        else:
            s["dZ"] = torch.empty_like(Z)
            s["dscale"], s["dshift"] = torch.empty((2, groups, K), device="cuda")
            s["ws"] = torch.empty(B.svdq_layer_norm_backward_workspace_bytes(M, K, rows), dtype=torch.uint8,
                                  device="cuda")
    return s


def _ckpt_buffers(M, K):
    return (torch.empty((M, K), dtype=torch.uint8, device="cuda"),
            torch.empty((M, -(-K // GROUP)), dtype=torch.uint8, device="cuda"))


def _codes(codes, fmt):
    """The codes as the numbers they stand for."""
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn)


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    B, case = _binding(), s["case"]
    op = case["op"]
    if op == "gemv":
        B.svdq_linear_w4a16(s["w"], s["X"], s["Y"], s["ws"])
        return s["Y"]
    if op == "wgrad":
        if case["ckpt"]:
            codes, scales = s["X"]
            B.svdq_lowrank_wgrad(None, s["S"], s["G"], s["ws"], ckpt=(codes, scales, case["ckpt"]))
        else:
            B.svdq_lowrank_wgrad(s["X"], s["S"], s["G"], s["ws"])
        return s["G"]
    if op == "encode":
        B.svdq_ckpt8_encode(s["Z"], s["codes"], s["scales"], case["ckpt"])
        return {"codes": _codes(s["codes"], case["ckpt"]), "scales": s["scales"]}
    if op == "decode":
        B.svdq_ckpt8_decode(s["ck"][0], s["ck"][1], s["out"], case["ckpt"])
        return s["out"]
    if op == "norm":
        B.svdq_layer_norm(s["Z"], s["scale"], s["shift"], s["Y"], s["stats"], 1e-6, group_rows=case["rows"],
                          plus_one=case["plus_one"], ckpt=s["ck"])
        out = {"Y": s["Y"], "stats": s["stats"]}
        if case["ckpt"]:
            out.update(codes=_codes(s["ck"][0], case["ckpt"]), scales=s["ck"][1])
        return out
    Z, ck = (None, s["Z"] + (case["ckpt"],)) if case["ckpt"] else (s["Z"], None)
    B.svdq_layer_norm_backward(s["dY"], Z, s["stats"], s["scale"], s["dZ"], s["dscale"], s["dshift"], s["ws"],
                               group_rows=case["rows"], plus_one=case["plus_one"], ckpt=ck)
    return {"dZ": s["dZ"], "dscale": s["dscale"], "dshift": s["dshift"]}


# ------------------------------------------------------------------ plain form
def _pow2(e):
    """2^e in fp32 from its bits, e in -127..127."""
    return torch.where(e < -126, 2.0 ** -127, ((e.int() + 127) << 23).view(torch.float32))


def _encode(x, fmt):
    """(codes, scale bytes) of fp32 rows."""
    M, K = x.shape
    n = -(-K // GROUP)
    x = torch.nn.functional.pad(x, (0, n * GROUP - K)).view(M, n, GROUP)
    amax = x.abs().amax(2)
    frac, exp = torch.frexp(amax)  # amax = frac * 2^exp, frac in [0.5, 1)
    if fmt == "int8":
        e = exp - 7 + (frac >= 127.5 / 128).int()
    else:
        e = exp - 9 + (frac > 448 / 512).int()
    e = torch.where(amax == 0, -127, e.clamp(min=-127))
    bad = ~torch.isfinite(amax)
    v = torch.where(bad[..., None], 0.0, x * _pow2(-torch.where(bad, 0, e))[..., None])
    v = v.round().to(torch.int8) if fmt == "int8" else v.to(torch.float8_e4m3fn)
    scales = torch.where(bad, 255, e + 127).to(torch.uint8)
    return v.view(torch.uint8).view(M, n * GROUP)[:, :K].contiguous(), scales


def _decode(codes, scales, fmt):
    K = codes.shape[1]
    s = torch.where(scales == 255, float("nan"), _pow2(torch.where(scales == 255, 0, scales.int() - 127)))
    s = s.repeat_interleave(GROUP, 1)[:, :K]
    return _codes(codes, fmt).float() * s


def _dequantize(codes, sf, fmt):
    """The weights in fp32, not yet times alpha_w."""
    N = codes.shape[0]
    lo, hi = codes & 15, codes >> 4
    if fmt == "nvfp4":  # the low nibble comes first
        q = torch.tensor(E2M1, device=codes.device)[torch.stack([lo, hi], 2).view(N, -1).int()]
        return q * sf.float().repeat_interleave(16, 1)
    # INT4: per 8 values bytes (0, 2) (4, 6) (1, 3) (5, 7), low nibble first
    q = torch.stack([lo, hi], 2).view(N, -1, 8)[..., [0, 4, 1, 5, 2, 6, 3, 7]].view(N, -1).float()
    q = torch.where(q >= 8, q - 16, q)
    return q * sf.float().repeat_interleave(64, 1)


def _of_groups(v, M, rows, plus_one=False):
    """Each row's vector of its group, in fp32."""
    v = v.float() + 1 if plus_one else v.float()
    return v.repeat_interleave(rows, 0)[:M]


def _group_sums(v, rows):
    M, K = v.shape
    groups = -(-M // rows)
    return torch.nn.functional.pad(v, (0, 0, 0, groups * rows - M)).view(groups, rows, K).sum(1)


def _run_plain(s):
    case = s["case"]
    op, fmt = case["op"], case.get("ckpt")
    if op == "gemv":
        X = s["X"].float()
        W = _dequantize(s["codes"], s["sf"], case["fmt"])
        Y = (X * s["inv_lam"]) @ W.T * s["alpha"] + s["bias"]
        if case["rank"]:
            Y = Y + (X @ s["L1"].float()) @ s["L2"].float()
        return Y.to(torch.bfloat16)
    if op == "wgrad":
        X = _decode(*s["X"], fmt) if fmt else s["X"].float()
        return X.T @ s["S"].float()
    if op == "encode":
        codes, scales = _encode(s["Z"].float(), fmt)
        return {"codes": _codes(codes, fmt), "scales": scales}
    if op == "decode":
        return _decode(*s["ck"], fmt).to(DTYPES[case["dtype"]])
    M, dtype = case["M"], DTYPES[case["dtype"]]
    rows = case["rows"] or M
    m = _of_groups(s["scale"], M, rows, case["plus_one"])
    if op == "norm":
        z = s["Z"].float()
        mu = z.mean(1, keepdim=True)
        rstd = 1 / torch.sqrt((z - mu).square().mean(1, keepdim=True) + 1e-6)
        y = (z - mu) * rstd * m + _of_groups(s["shift"], M, rows)
        out = {"Y": y.to(dtype), "stats": torch.cat([mu, rstd], 1)}
        if fmt:
            codes, scales = _encode(z, fmt)
            out.update(codes=_codes(codes, fmt), scales=scales)
        return out
    z, dy = _decode(*s["Z"], fmt) if fmt else s["Z"].float(), s["dY"].float()
    mu, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    xh = (z - mu) * rstd
    g = dy * m
    dz = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return {"dZ": dz.to(dtype), "dscale": _group_sums(dy * xh, rows), "dshift": _group_sums(dy, rows)}


# ------------------------------------------------------------------ work and definition
def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    ck = M * K + M * -(-K // GROUP)  # bytes of a checkpoint
    if op == "gemv":
        N, r = case["N"], case["rank"]
        weights = N * K // 2 + (N * (K // 16) if case["fmt"] == "nvfp4" else N * (K // 64) * 2)
        branch = 2 * r * (K + N)
        return {"bytes": weights + branch + 4 * K + 4 * N + 2 * M * (K + N),
                "flops": 2 * M * (N * K + r * (K + N))}
    if op == "wgrad":
        r = case["rank"]
        return {"bytes": (ck if case["ckpt"] else 2 * M * K) + 2 * M * r + 4 * K * r, "flops": 2 * M * K * r}
    size = 4 if case["dtype"] == "fp32" else 2
    if op in ("encode", "decode"):
        return {"bytes": size * M * K + ck, "flops": 2 * M * K}
    groups = -(-M // (case["rows"] or M))
    vec = groups * K * (4 if case["pdtype"] == "fp32" else 2)
    if op == "norm":
        return {"bytes": 2 * size * M * K + (ck if case["ckpt"] else 0) + 2 * vec + 8 * M, "flops": 8 * M * K}
    z = ck if case["ckpt"] else size * M * K
    return {"bytes": z + 2 * size * M * K + vec + 8 * groups * K + 8 * M, "flops": 14 * M * K}


def _host(t):
    if t.dtype == torch.float8_e4m3fn:
        t = t.float()
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _exact_codes(x, fmt):
    """Codes (as numbers) and scale bytes of float64 rows, group by group of the definition."""
    top = 127.5 if fmt == "int8" else 448.0
    M, K = x.shape
    edges = np.arange(0, K, GROUP)
    amax = np.maximum.reduceat(np.abs(x), edges, axis=1)
    e = np.full(amax.shape, -127, np.int64)
    some = amax > 0
    e[some] = np.floor(np.log2(amax[some])).astype(np.int64) - (7 if fmt == "int8" else 9)
    for _ in range(3):  # up to the first exponent that holds the largest magnitude
        t = amax / np.exp2(e)
        e = np.where(t >= top if fmt == "int8" else t > top, e + 1, e)
    e = np.maximum(e, -127)
    v = x / np.exp2(np.repeat(e, GROUP, 1)[:, :K])
    if fmt == "int8":
        return np.rint(v).astype(np.int64), e + 127
    mag = np.abs(v)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(mag, 1e-300))), -6) - 3)
    return np.copysign(np.rint(mag / step) * step, v), e + 127


def _exact_values(codes, scales, fmt):
    K = codes.shape[1]
    return _host(_codes(codes, fmt)).astype(np.float64) * np.exp2(np.repeat(_host(scales) - 127.0, GROUP, 1)[:, :K])


def exact(case, seed):
    keep = globals()["own"]
    globals()["own"] = False  # the inputs alone
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = keep
    op, fmt, M, K = case["op"], case.get("ckpt"), case["M"], case["K"]
    if op == "gemv":
        # on the GPU in 64 bits, some output columns at a time
        X, N = s["X"].double(), case["N"]
        T = X @ s["L1"].double()
        Xh = X * s["inv_lam"].double()
        out = torch.empty((M, N), dtype=torch.float64, device="cuda")
        for n in range(0, N, 2048):
            c = s["codes"][n:n + 2048]
            W = torch.empty((c.shape[0], K), dtype=torch.float64, device="cuda")
            if case["fmt"] == "nvfp4":
                table = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
                W[:, 0::2], W[:, 1::2] = table[(c % 16).long()], table[(c // 16).long()]
                W = W.view(-1, K // 16, 16) * s["sf"][n:n + 2048].double()[..., None]
            else:
                for byte, (a, b) in enumerate(((0, 2), (4, 6), (1, 3), (5, 7))):
                    v = c[:, byte::4].double()
                    low, high = v % 16, torch.floor(v / 16)
                    W[:, a::8], W[:, b::8] = (low + 8) % 16 - 8, (high + 8) % 16 - 8
                W = W.view(-1, K // 64, 64) * s["sf"][n:n + 2048].double()[..., None]
            y = Xh @ W.view(-1, K).T * s["alpha"]
            out[:, n:n + 2048] = y + T @ s["L2"][:, n:n + 2048].double() + s["bias"][n:n + 2048].double()
        return out.cpu().numpy()
    if op == "wgrad":
        X = _exact_values(*s["X"], fmt) if fmt else _host(s["X"])
        return X.T @ _host(s["S"])
    if op == "encode":
        codes, scales = _exact_codes(_host(s["Z"]), fmt)
        return {"codes": codes, "scales": scales}
    if op == "decode":
        return _exact_values(*s["ck"], fmt)
    of = np.arange(M) // (case["rows"] or M)
    m = _host(s["scale"])[of] + (1.0 if case["plus_one"] else 0.0)
    if op == "norm":
        z = _host(s["Z"])
        mu, sd = z.mean(1, keepdims=True), np.sqrt(z.var(1, keepdims=True) + 1e-6)
        out = {"Y": (z - mu) / sd * m + _host(s["shift"])[of], "stats": np.concatenate([mu, 1 / sd], 1)}
        if fmt:
            out["codes"], out["scales"] = _exact_codes(z, fmt)
        return out
    z = _exact_values(*s["Z"], fmt) if fmt else _host(s["Z"])
    dy, st = _host(s["dY"]), _host(s["stats"])
    xh = (z - st[:, :1]) * st[:, 1:]
    g = dy * m
    first = np.arange(0, M, case["rows"] or M)
    return {"dZ": st[:, 1:] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True)),
            "dscale": np.add.reduceat(dy * xh, first, axis=0), "dshift": np.add.reduceat(dy, first, axis=0)}
