"""Argument checks of the few-token layer, the layer norm, the checkpoints and the low-rank gradient:
every refusal comes before any GPU work, so these run without a GPU."""

import ctypes

import numpy as np
import pytest
import torch

from rank_outlier_gemm_b200 import binding as B

P = 0x10000  # an aligned address that no refused call follows
INVALID = 1


def refused(status, text):
    assert status == INVALID
    assert text in B._lib.svdq_last_error().decode()


def desc(**kw):
    d = B.NormDesc(4, 64, 0, 0, 2, 0, 1e-6, 0, 0, 0, 0, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,text", [
    (dict(M=0), "M=0"), (dict(M=-1), "M=-1"), (dict(M=2 ** 30 + 1), "M="), (dict(K=0), "K=0"), (dict(K=16385), "K=16385"),
    (dict(dtype=3), "dtype=3"), (dict(dtype=-1), "dtype=-1"), (dict(param_dtype=5), "param_dtype=5"),
    (dict(group_rows=-2), "group_rows=-2"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(eps=float("inf")), "eps"), (dict(ld_z=63), "ld_z"), (dict(ld_y=-64), "ld_y"), (dict(ld_param=10), "ld_param"),
    (dict(ld_dz=2 ** 41), "ld_dz")])
def test_norm_desc(kw, text):
    d = desc(**kw)
    refused(B._lib.svdq_layer_norm(d, P, None, None, P, None, None, None, 0, None), text)
    refused(B._lib.svdq_layer_norm_backward(d, P, P, None, None, 0, P, None, P, None, None, P, 1 << 40, None), text)


def test_norm_pointers():
    f, b = B._lib.svdq_layer_norm, B._lib.svdq_layer_norm_backward
    d = desc()
    refused(f(None, P, None, None, P, None, None, None, 0, None), "desc is null")
    refused(f(d, None, None, None, P, None, None, None, 0, None), "Z is null")
    refused(f(d, P + 1, None, None, P, None, None, None, 0, None), "Z is not aligned")
    refused(f(d, P, P + 2, None, P, None, None, None, 0, None), "scale is not aligned")  # fp32 parameters
    refused(f(d, P, None, None, None, None, None, None, 0, None), "Y is null")
    refused(f(d, P, None, None, P, P + 4, None, None, 0, None), "stats is not 16-byte aligned")
    refused(f(d, P, None, None, P, None, P, None, 0, None), "both codes and scales")
    refused(f(d, P, None, None, P, None, P + 8, P, 0, None), "codes is not 16-byte aligned")
    refused(f(d, P, None, None, P, None, P, P, 2, None), "format=2")
    refused(b(d, P, None, None, None, 0, P, None, P, None, None, P, 1 << 40, None), "either Z or its checkpoint")
    refused(b(d, P, P, P, P, 0, P, None, P, None, None, P, 1 << 40, None), "either Z or its checkpoint")
    refused(b(d, None, P, None, None, 0, P, None, P, None, None, P, 1 << 40, None), "dY is null")
    refused(b(d, P, P, None, None, 0, None, None, P, None, None, P, 1 << 40, None), "stats is null")
    refused(b(d, P, P, None, None, 0, P, None, None, None, None, P, 1 << 40, None), "dZ is null")
    refused(b(d, P, P, None, None, 0, P, None, P, P + 2, None, P, 1 << 40, None), "dscale is not aligned")
    big = desc(M=4096)
    need = B.svdq_layer_norm_backward_workspace_bytes(4096, 64)
    assert need > 0
    refused(b(big, P, P, None, None, 0, P, None, P, P, P, None, need, None), "workspace is null")
    refused(b(big, P, P, None, None, 0, P, None, P, P, P, P, need - 1, None), "workspace has")
    refused(b(big, P, P, None, None, 0, P, None, P, P, P, P + 8, need, None), "workspace is not 16-byte aligned")


def test_checkpoint():
    e, d = B._lib.svdq_ckpt8_encode, B._lib.svdq_ckpt8_decode
    refused(e(P, 0, 0, 64, 0, 0, P, P, None), "M=0")
    refused(e(P, 0, 4, 0, 0, 0, P, P, None), "K=0")
    refused(e(P, 4, 4, 64, 0, 0, P, P, None), "dtype=4")
    refused(e(P, 0, 4, 64, 0, 3, P, P, None), "format=3")
    refused(e(P, 0, 4, 64, 32, 0, P, P, None), "ld is below")
    refused(e(P + 1, 0, 4, 64, 0, 0, P, P, None), "X is not aligned")
    refused(e(P, 0, 4, 64, 0, 0, None, P, None), "codes is null")
    refused(e(P, 0, 4, 64, 0, 0, P, None, None), "scales is null")
    refused(d(P, P, 4, 64, 0, None, 0, 0, None), "X is null")
    refused(d(P, P, 4, 64, 0, P + 2, 2, 0, None), "X is not aligned")
    refused(d(P, P, 4, 64, 9, P, 2, 0, None), "format=9")
    assert B.svdq_ckpt8_codes_bytes(3, 70) == 210 and B.svdq_ckpt8_scales_bytes(3, 70) == 9
    assert B.svdq_ckpt8_codes_bytes(0, 70) == 0 and B.svdq_ckpt8_scales_bytes(3, -1) == 0


def test_lowrank_wgrad():
    f = B._lib.svdq_lowrank_wgrad
    big = 1 << 40
    refused(f(P, None, None, 0, P, 0, 64, 8, P, P, big, None), "M=0")
    refused(f(P, None, None, 0, P, 4, 72, 8, P, P, big, None), "K=72")
    refused(f(P, None, None, 0, P, 4, 64, 0, P, P, big, None), "r=0")
    refused(f(P, None, None, 0, P, 4, 64, 129, P, P, big, None), "r=129")
    refused(f(None, None, None, 0, P, 4, 64, 8, P, P, big, None), "either X or its checkpoint")
    refused(f(P, P, P, 0, P, 4, 64, 8, P, P, big, None), "either X or its checkpoint")
    refused(f(None, P, None, 0, P, 4, 64, 8, P, P, big, None), "both codes and scales")
    refused(f(None, P, P, 5, P, 4, 64, 8, P, P, big, None), "format=5")
    refused(f(P + 8, None, None, 0, P, 4, 64, 8, P, P, big, None), "X is not 16-byte aligned")
    refused(f(P, None, None, 0, None, 4, 64, 8, P, P, big, None), "S is null")
    refused(f(P, None, None, 0, P, 4, 64, 8, None, P, big, None), "G is null")
    need = B.svdq_lowrank_wgrad_workspace_bytes(4096, 64, 8)
    assert need > 0
    refused(f(P, None, None, 0, P, 4096, 64, 8, P, P, need - 4, None), "workspace has")
    assert B.svdq_lowrank_wgrad_workspace_bytes(4096, 60, 8) == 0


def test_w4a16():
    f = B._lib.svdq_linear_w4a16
    refused(f(None, P, 1, P, P, 1 << 40, None), "null weights handle")
    assert B._lib.svdq_linear_w4a16_workspace_bytes(None, 1) == 0


def codes_args(N=16, K=64, fmt=0):
    sf = np.zeros(B.svdq_act_sf_bytes(N, K) if fmt == 0 else K // 64 * 256 * 2, np.uint8)
    return np.zeros((N, K // 2), np.uint8), sf, np.ones(K, np.float32)


@pytest.mark.parametrize("alpha,fmt,text", [(0.0, 0, "alpha_w"), (-1.0, 0, "alpha_w"), (3.0, 0, "alpha_w"),
                                            (float("nan"), 0, "alpha_w"), (float("inf"), 0, "alpha_w"),
                                            (0.5, 1, "must be 1"), (1.0, 2, "format=2")])
def test_weights_from_codes_factor(alpha, fmt, text):
    c, s, inv = codes_args(fmt=min(fmt, 1))
    h = ctypes.c_void_p(1)
    refused(B._lib.svdq_weights_from_codes(16, 64, 0, alpha, c.ctypes.data, s.ctypes.data, inv.ctypes.data, None, None,
                                           None, fmt, None, ctypes.byref(h)), text)
    assert not h.value


def test_weights_from_codes_values():
    def call(c, s, inv, fmt, rank=0, N=16, K=64):
        h = ctypes.c_void_p()
        return B._lib.svdq_weights_from_codes(N, K, rank, 1.0, c.ctypes.data, s.ctypes.data, inv.ctypes.data, None,
                                              None, None, fmt, None, ctypes.byref(h))
    c, s, inv = codes_args()
    refused(call(c, s, inv, 0, K=72), "multiple of 64")
    refused(call(c, s, inv, 0, N=24), "multiple of 16")
    refused(call(c, s, inv, 0, rank=129), "rank=129")
    refused(call(c, s, inv, 0, rank=4), "needs L1p")
    for byte in (0x7F, 0x80, 0xFF):
        bad = s.copy()
        bad[15 * 16 + 3] = byte  # row 15, group 3
        refused(call(c, bad, inv, 0), "E4M3 scale")
    inv2 = inv.copy()
    inv2[9] = np.inf
    refused(call(c, s, inv2, 0), "inv_lam")
    c, s, inv = codes_args(fmt=1)
    for at in (0, 7, 8, c.size - 1):
        for code in (0x08, 0x80, 0x18, 0x8F):
            bad = c.copy().reshape(-1)
            bad[at] = code
            refused(call(bad, s, inv, 1), "-8")
    for bits in (0x7F80, 0xBF80, 0x7FC0):
        bad = s.copy()
        bad.view(np.uint16)[15] = bits
        refused(call(c, bad, inv, 1), "scale")


def test_the_binding_refuses_tensors_of_the_wrong_kind():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)  # a host tensor
    with pytest.raises(ValueError, match="CUDA"):
        B.svdq_layer_norm(x, None, None, x, None, 1e-6)
    with pytest.raises(ValueError, match="2-D"):
        B.svdq_ckpt8_encode(x[0], x, x)
    with pytest.raises(ValueError, match="CUDA"):
        B.svdq_lowrank_wgrad(x, x, torch.zeros((64, 64)), None)
    with pytest.raises(ValueError, match="codes has"):
        B.svdq_weights_from_codes(16, 64, 0, 1.0, np.zeros(100, np.uint8), np.zeros(512, np.uint8), np.ones(64, np.float32),
                                  None, None)
