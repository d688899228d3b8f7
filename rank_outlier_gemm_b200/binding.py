"""ctypes binding of ``libsvdq.so`` (declared in ``include/svdq.h``).

Each function has the name of the C entry point it calls and only marshals
arguments: host arrays become pointers to their data, CUDA tensors become
device pointers, and the CUDA stream is PyTorch's current stream unless one is
given.  Every step of the layer runs in the library's kernels; there is no
fallback path, and importing this module fails if the library is not built.
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import numpy as np
import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsvdq.so")

SVDQ_OK = 0
STATUS_NAMES = {0: "SVDQ_OK", 1: "SVDQ_ERR_INVALID_ARG", 2: "SVDQ_ERR_UNSUPPORTED_DEVICE",
                3: "SVDQ_ERR_CUDA", 4: "SVDQ_ERR_OOM", 5: "SVDQ_ERR_TIMEOUT",
                6: "SVDQ_ERR_DEVICE_CHECK"}


class SvdqError(RuntimeError):
    def __init__(self, status: int, fn: str, msg: str):
        self.status = status
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)}: {msg}")


class PrepareOpts(ctypes.Structure):
    _fields_ = [("alpha", ctypes.c_float), ("rank", ctypes.c_int), ("power_iters", ctypes.c_int),
                ("oversample", ctypes.c_int), ("seed", ctypes.c_uint64), ("keep_residual", ctypes.c_int),
                ("refine_iters", ctypes.c_int), ("format", ctypes.c_int)]


class NormDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int), ("K", ctypes.c_int), ("group_rows", ctypes.c_int), ("dtype", ctypes.c_int),
                ("param_dtype", ctypes.c_int), ("plus_one", ctypes.c_int), ("eps", ctypes.c_float),
                ("ld_z", ctypes.c_int64), ("ld_y", ctypes.c_int64), ("ld_dy", ctypes.c_int64),
                ("ld_dz", ctypes.c_int64), ("ld_param", ctypes.c_int64)]


FORMATS = {"nvfp4": 0, "int4": 1}
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
CKPT8_FORMATS = {"int8": 0, "e4m3": 1}


_vp, _i, _sz, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_i64, _desc = ctypes.c_int64, ctypes.POINTER(NormDesc)
_SIGS = {
    "svdq_prepare_opts_default": (None, [ctypes.POINTER(PrepareOpts)]),
    "svdq_prepare_weights": (_i, [_vp, _vp, _vp, _i, _i, ctypes.POINTER(PrepareOpts), _vp, ctypes.POINTER(_vp)]),
    "svdq_weights_from_factors": (_i, [_i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.POINTER(_vp)]),
    "svdq_weights_from_factors_fmt": (_i, [_i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, ctypes.POINTER(_vp)]),
    "svdq_weights_from_codes": (_i, [_i, _i, _i, _f, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, ctypes.POINTER(_vp)]),
    "svdq_weights_format": (_i, [_vp, ctypes.POINTER(_i)]),
    "svdq_weights_sf_bytes": (_sz, [_vp]),
    "svdq_attach_lora": (_i, [_vp, _vp, _vp, _i, _f, _vp]),
    "svdq_quantize_act_lowrank_down": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _vp]),
    "svdq_linear_w4a4": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _vp]),
    "svdq_forward": (_i, [_vp, _vp, _i, _vp, _vp, _sz, _vp]),
    "svdq_forward_host": (_i, [_vp, _vp, _i, _vp, _vp, _sz, _vp]),
    "svdq_forward_noalloc": (_i, [_vp, _vp, _i, _vp, _vp]),
    "svdq_act_row_stats": (_i, [_vp, _i, _i, _f, _vp, _vp]),
    "svdq_norm_quantize_act_lowrank_down": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "svdq_forward_norm": (_i, [_vp, _vp, _i, _vp, _vp, _f, _vp, _vp, _sz, _vp]),
    "svdq_forward_norm_workspace_bytes": (_sz, [_vp, _i]),
    "svdq_linear_w4a16": (_i, [_vp, _vp, _i, _vp, _vp, _sz, _vp]),
    "svdq_linear_w4a16_workspace_bytes": (_sz, [_vp, _i]),
    "svdq_layer_norm": (_i, [_desc, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp]),
    "svdq_layer_norm_backward": (_i, [_desc, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "svdq_layer_norm_backward_workspace_bytes": (_sz, [_i, _i, _i]),
    "svdq_ckpt8_encode": (_i, [_vp, _i, _i, _i, _i64, _i, _vp, _vp, _vp]),
    "svdq_ckpt8_decode": (_i, [_vp, _vp, _i, _i, _i, _vp, _i, _i64, _vp]),
    "svdq_lowrank_wgrad": (_i, [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _vp, _vp, _sz, _vp]),
    "svdq_lowrank_wgrad_workspace_bytes": (_sz, [_i, _i, _i]),
    "svdq_ckpt8_codes_bytes": (_sz, [_i, _i]),
    "svdq_ckpt8_scales_bytes": (_sz, [_i, _i]),
    "svdq_act_codes_bytes": (_sz, [_i, _i]),
    "svdq_act_sf_bytes": (_sz, [_i, _i]),
    "svdq_lowrank_bytes": (_sz, [_vp, _i]),
    "svdq_forward_workspace_bytes": (_sz, [_vp, _i]),
    "svdq_forward_host_workspace_bytes": (_sz, [_vp, _i]),
    "svdq_weights_rank": (_i, [_vp]),
    "svdq_weights_info": (_i, [_vp, ctypes.POINTER(_i), ctypes.POINTER(_i), ctypes.POINTER(_i),
                               ctypes.POINTER(_i), ctypes.POINTER(_f)]),
    "svdq_weights_export": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "svdq_weights_destroy": (_i, [_vp]),
    "svdq_set_wait_limit_ns": (None, [ctypes.c_uint64]),
    "svdq_check_device_errors": (_i, [_vp]),
    "svdq_selftest_codec": (_i, [ctypes.POINTER(ctypes.c_uint)]),
    "svdq_weights_refine_errors": (_i, [_vp, ctypes.POINTER(ctypes.c_double), _i, ctypes.POINTER(_i)]),
    "svdq_search_alpha": (_i, [_vp, _vp, _i, _vp, _i, _i, _vp, _i, ctypes.POINTER(PrepareOpts), _vp,
                               ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_i)]),
    "svdq_debug_launch_stalled_act": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _vp]),
    "svdq_debug_stalled_layer_norm_backward": (_i, [_desc, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "svdq_debug_linear_w4a4_ksplit": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _i, _vp]),
    "svdq_debug_forward_small_m": (_i, [_vp, _vp, _i, _vp, _i, _vp]),
    "svdq_last_error": (ctypes.c_char_p, []),
    "svdq_version": (ctypes.c_char_p, []),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m rank_outlier_gemm_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()
EXPORTED = tuple(_SIGS)


def _check(status: int, fn: str):
    if status != SVDQ_OK:
        raise SvdqError(status, fn, _lib.svdq_last_error().decode())


def _host(a, dtype) -> tuple:
    """(pointer, keep-alive) of a contiguous host array of the given numpy dtype."""
    if a is None:
        return None, None
    if isinstance(a, torch.Tensor):
        if a.is_cuda:
            raise ValueError("expected a host array")
        if a.dtype == torch.bfloat16:
            a = a.view(torch.int16)
        a = a.numpy()
    arr = np.ascontiguousarray(a)
    if arr.dtype != np.dtype(dtype):
        if np.dtype(dtype) == np.uint16 and arr.dtype == np.int16:
            arr = arr.view(np.uint16)
        else:
            arr = arr.astype(dtype)
    return arr.ctypes.data, arr


def _dev(t: Optional[torch.Tensor], name: str):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# The raw current stream of a device, without the Python object torch.cuda.current_stream() builds for it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _device_and_stream(stream) -> tuple:
    """The current device and the raw stream to launch on (None: PyTorch's current stream there)."""
    dev = torch.cuda.current_device() if torch.cuda.is_initialized() else -2  # no tensor's device
    if stream is not None:
        return dev, stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if dev < 0:  # no CUDA tensor exists yet: the arguments' checks say so
        return dev, None
    return dev, _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _arg(t, name: str, shape, dtype, dev: int) -> int:
    """Address of a packed CUDA tensor of this shape and type on the current device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev and \
            t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, shape, (dtype,), dev)
    raise ValueError(f"{name} must be contiguous")


def _rows_arg(t, name: str, shape, dtypes, dev: int) -> tuple:
    """(address, elements between rows) of a CUDA matrix on the current device whose last index is contiguous."""
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == dev):
        _refuse(t, name, shape, dtypes, dev)
    rows, cols = shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"the last index of {name} must be contiguous")
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError(f"the rows of {name} overlap")
    return t.data_ptr(), ld


def _refuse(t, name: str, shape, dtypes, dev: int) -> None:
    """Raises ValueError with what is wrong with a tensor's kind, type, shape or device, if anything is."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has type {t.dtype}, not one of {', '.join(str(d) for d in dtypes)}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current device {dev}")


def _workspace(t: Optional[torch.Tensor], dev: int) -> tuple:
    """(address, bytes) of a packed CUDA workspace, or of none."""
    if t is None or t.numel() == 0:
        return None, 0
    return _arg(t, "workspace", t.shape, t.dtype, dev), t.numel() * t.element_size()


def _shape2(t, name: str) -> tuple:
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    return t.shape


def _ckpt(ckpt, M: int, K: int, dev: int) -> tuple:
    """(codes, scales, format) arguments of a checkpoint (codes, scales, "int8" or "e4m3") or of none."""
    if ckpt is None:
        return None, None, 0
    codes, scales, fmt = ckpt
    return (_arg(codes, "codes", (M, K), torch.uint8, dev),
            _arg(scales, "scales", (M, (K + 31) // 32), torch.uint8, dev), _ckpt_format(fmt))


def _ckpt_format(fmt: str) -> int:
    if fmt not in CKPT8_FORMATS:
        raise ValueError(f"checkpoint format {fmt!r} is not one of {', '.join(CKPT8_FORMATS)}")
    return CKPT8_FORMATS[fmt]


class Weights:
    """Owns an svdq_weights handle; destroyed with the object."""

    def __init__(self, handle: int):
        self.handle = handle
        self.N, self.K = self.info["N"], self.info["K"]  # fixed for the handle's life

    @property
    def info(self) -> dict:
        N, K, r, rp, aw = _i(), _i(), _i(), _i(), _f()
        _check(_lib.svdq_weights_info(self.handle, ctypes.byref(N), ctypes.byref(K), ctypes.byref(r),
                                      ctypes.byref(rp), ctypes.byref(aw)), "svdq_weights_info")
        fmt = _i()
        _check(_lib.svdq_weights_format(self.handle, ctypes.byref(fmt)), "svdq_weights_format")
        return {"N": N.value, "K": K.value, "rank": r.value, "r_pad": rp.value, "alpha_w": aw.value,
                "format": {v: k for k, v in FORMATS.items()}[fmt.value]}

    def __del__(self):
        # at interpreter exit the module globals may already be gone
        if getattr(self, "handle", None) and _lib is not None:
            _lib.svdq_weights_destroy(self.handle)
            self.handle = None


def svdq_prepare_opts_default() -> PrepareOpts:
    o = PrepareOpts()
    _lib.svdq_prepare_opts_default(ctypes.byref(o))
    return o


def svdq_prepare_weights(W_bf16, act_absmax, bias_bf16=None, rank: int = 32, alpha: float = 0.5,
                         power_iters: int = 4, oversample: int = 16, seed: int = 0,
                         keep_residual: bool = False, refine_iters: int = 1, fmt: str = "nvfp4",
                         stream=None) -> Weights:
    Wp, Wk = _host(W_bf16, np.uint16)
    N, K = Wk.shape
    ap, ak = _host(act_absmax, np.float32)
    bp, bk = _host(bias_bf16, np.uint16)
    o = svdq_prepare_opts_default()
    o.alpha, o.rank, o.power_iters, o.oversample, o.seed = alpha, rank, power_iters, oversample, seed
    o.keep_residual = int(keep_residual)
    o.refine_iters = int(refine_iters)
    o.format = FORMATS[fmt]
    h = _vp()
    _check(_lib.svdq_prepare_weights(Wp, ap, bp, N, K, ctypes.byref(o), _stream(stream), ctypes.byref(h)),
           "svdq_prepare_weights")
    return Weights(h.value)


def svdq_weights_from_factors(N: int, K: int, rank: int, inv_lam, L1p_bf16, L2_bf16, R, bias=None,
                              stream=None, fmt: str = "nvfp4") -> Weights:
    ip, ik = _host(inv_lam, np.float32)
    lp, lk = _host(L1p_bf16, np.uint16) if rank else (None, None)
    l2p, l2k = _host(L2_bf16, np.uint16) if rank else (None, None)
    rp, rk = _host(R, np.float32)
    bp, bk = _host(bias, np.float32)
    h = _vp()
    _check(_lib.svdq_weights_from_factors_fmt(N, K, rank, ip, lp, l2p, rp, bp, FORMATS[fmt], _stream(stream),
                                              ctypes.byref(h)), "svdq_weights_from_factors_fmt")
    return Weights(h.value)


def svdq_weights_from_codes(N: int, K: int, rank: int, alpha_w: float, codes, sf, inv_lam, L1p_bf16, L2_bf16,
                            bias=None, fmt: str = "nvfp4", stream=None) -> Weights:
    """A handle from what svdq_weights_export gives (host arrays)."""
    cp, ck = _host(codes, np.uint8)
    sp, sk = _host(sf, np.uint8)
    ip, ik = _host(inv_lam, np.float32)
    lp, lk = _host(L1p_bf16, np.uint16) if rank else (None, None)
    l2p, l2k = _host(L2_bf16, np.uint16) if rank else (None, None)
    bp, bk = _host(bias, np.float32)
    n_sf = (K // 64) * (-(-N // 256) * 256) * 2 if fmt == "int4" else svdq_act_sf_bytes(N, K)
    for a, n, name in ((ck, N * K // 2, "codes"), (sk, n_sf, "sf"), (ik, K, "inv_lam"), (lk, K * rank, "L1p"),
                       (l2k, rank * N, "L2"), (bk, N, "bias")):
        if a is not None and a.size != n:
            raise ValueError(f"{name} has {a.size} elements, not {n}")
    h = _vp()
    _check(_lib.svdq_weights_from_codes(N, K, rank, alpha_w, cp, sp, ip, lp, l2p, bp, FORMATS[fmt], _stream(stream),
                                        ctypes.byref(h)), "svdq_weights_from_codes")
    return Weights(h.value)


def svdq_attach_lora(w: Weights, A_bf16, B_bf16, scale: float = 1.0, stream=None) -> None:
    Ap, Ak = _host(A_bf16, np.uint16)
    Bp, Bk = _host(B_bf16, np.uint16)
    _check(_lib.svdq_attach_lora(w.handle, Ap, Bp, Ak.shape[1], scale, _stream(stream)), "svdq_attach_lora")


def svdq_quantize_act_lowrank_down(w: Weights, X: torch.Tensor, xq: torch.Tensor, xsf: torch.Tensor,
                                   T: Optional[torch.Tensor], stream=None) -> None:
    _check(_lib.svdq_quantize_act_lowrank_down(w.handle, _dev(X, "X"), X.shape[0], _dev(xq, "xq"),
                                               _dev(xsf, "xsf"), _dev(T, "T"), _stream(stream)),
           "svdq_quantize_act_lowrank_down")


def svdq_debug_launch_stalled_act(w: Weights, X, xq, xsf, T, stream=None) -> None:
    _check(_lib.svdq_debug_launch_stalled_act(w.handle, _dev(X, "X"), X.shape[0], _dev(xq, "xq"),
                                              _dev(xsf, "xsf"), _dev(T, "T"), _stream(stream)),
           "svdq_debug_launch_stalled_act")


def svdq_linear_w4a4(w: Weights, xq, xsf, T, M: int, Y: torch.Tensor, stream=None) -> None:
    _check(_lib.svdq_linear_w4a4(w.handle, _dev(xq, "xq"), _dev(xsf, "xsf"), _dev(T, "T"), M, _dev(Y, "Y"),
                                 _stream(stream)), "svdq_linear_w4a4")


def svdq_debug_stalled_layer_norm_backward(dY, Z, stats, dZ, dscale, dshift, workspace, group_rows: int = 0,
                                           stream=None) -> None:
    dev, s = _device_and_stream(stream)
    M, K = _shape2(dY, "dY")
    dyp, ld_dy = _rows_arg(dY, "dY", (M, K), DTYPES, dev)
    zp, ld_z = _rows_arg(Z, "Z", (M, K), (dY.dtype,), dev)
    dzp, ld_dz = _rows_arg(dZ, "dZ", (M, K), (dY.dtype,), dev)
    shape = (-(-M // (group_rows or M)), K)
    da = _arg(dscale, "dscale", shape, torch.float32, dev) if dscale is not None else None
    dc = _arg(dshift, "dshift", shape, torch.float32, dev) if dshift is not None else None
    stp = _arg(stats, "stats", (M, 2), torch.float32, dev)
    ws, n = _workspace(workspace, dev)
    d = _norm_desc(M, K, group_rows, DTYPES[dY.dtype], 2, False, 0.0, ld_z, 0, ld_dy, ld_dz, 0)
    _check(_lib.svdq_debug_stalled_layer_norm_backward(d, dyp, zp, stp, dzp, da, dc, ws, n, s),
           "svdq_debug_stalled_layer_norm_backward")


def svdq_debug_linear_w4a4_ksplit(w: Weights, xq, xsf, T, M: int, Y: torch.Tensor, ksplit: int,
                                  stream=None) -> None:
    _check(_lib.svdq_debug_linear_w4a4_ksplit(w.handle, _dev(xq, "xq"), _dev(xsf, "xsf"), _dev(T, "T"), M,
                                              _dev(Y, "Y"), ksplit, _stream(stream)),
           "svdq_debug_linear_w4a4_ksplit")


def svdq_debug_forward_small_m(w: Weights, X: torch.Tensor, Y: torch.Tensor, ksplit: int = 0, stream=None) -> None:
    _check(_lib.svdq_debug_forward_small_m(w.handle, _dev(X, "X"), X.shape[0], _dev(Y, "Y"), ksplit, _stream(stream)),
           "svdq_debug_forward_small_m")


def svdq_forward(w: Weights, X: torch.Tensor, Y: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    _check(_lib.svdq_forward(w.handle, _dev(X, "X"), X.shape[0], _dev(Y, "Y"), _dev(workspace, "workspace"),
                             workspace.numel() * workspace.element_size(), _stream(stream)), "svdq_forward")


def svdq_forward_host(w: Weights, X_host: torch.Tensor, Y_host: torch.Tensor, workspace: torch.Tensor,
                      stream=None) -> None:
    if X_host.is_cuda or Y_host.is_cuda:
        raise ValueError("X_host and Y_host must be host tensors")
    _check(_lib.svdq_forward_host(w.handle, X_host.data_ptr(), X_host.shape[0], Y_host.data_ptr(),
                                  _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
                                  _stream(stream)), "svdq_forward_host")


def svdq_forward_noalloc(w: Weights, X: torch.Tensor, Y: torch.Tensor, stream=None) -> None:
    """svdq_forward with the intermediates in the library's static device block (no allocation)."""
    _check(_lib.svdq_forward_noalloc(w.handle, _dev(X, "X"), X.shape[0], _dev(Y, "Y"), _stream(stream)),
           "svdq_forward_noalloc")


def svdq_act_row_stats(Z: torch.Tensor, eps: float, stats: torch.Tensor, stream=None) -> None:
    """(mu, rstd) per row of a CUDA bf16 [M, K] tensor into a CUDA float32 [M, 2] tensor."""
    _check(_lib.svdq_act_row_stats(_dev(Z, "Z"), Z.shape[0], Z.shape[1], float(eps), _dev(stats, "stats"),
                                   _stream(stream)), "svdq_act_row_stats")


def svdq_norm_quantize_act_lowrank_down(w: Weights, Z: torch.Tensor, stats: torch.Tensor, norm_a: torch.Tensor,
                                        norm_c: torch.Tensor, xq, xsf, T, stream=None) -> None:
    _check(_lib.svdq_norm_quantize_act_lowrank_down(w.handle, _dev(Z, "Z"), Z.shape[0], _dev(stats, "stats"),
                                                    _dev(norm_a, "norm_a"), _dev(norm_c, "norm_c"), _dev(xq, "xq"),
                                                    _dev(xsf, "xsf"), _dev(T, "T"), _stream(stream)),
           "svdq_norm_quantize_act_lowrank_down")


def svdq_forward_norm(w: Weights, Z: torch.Tensor, norm_a: torch.Tensor, norm_c: torch.Tensor, eps: float,
                      Y: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    _check(_lib.svdq_forward_norm(w.handle, _dev(Z, "Z"), Z.shape[0], _dev(norm_a, "norm_a"), _dev(norm_c, "norm_c"),
                                  float(eps), _dev(Y, "Y"), _dev(workspace, "workspace"),
                                  workspace.numel() * workspace.element_size(), _stream(stream)), "svdq_forward_norm")


def svdq_forward_norm_workspace_bytes(w: Weights, M: int) -> int:
    return _lib.svdq_forward_norm_workspace_bytes(w.handle, M)


def svdq_linear_w4a16(w: Weights, X: torch.Tensor, Y: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """The layer on 1..16 tokens with 16-bit activations: X [M, K], Y [M, N], CUDA bf16."""
    dev, s = _device_and_stream(stream)
    M, K = _shape2(X, "X")
    if K != w.K:
        raise ValueError(f"X has {K} columns, the layer takes {w.K}")
    ws, n = _workspace(workspace, dev)
    st = _lib.svdq_linear_w4a16(w.handle, _arg(X, "X", (M, K), torch.bfloat16, dev), M,
                                _arg(Y, "Y", (M, w.N), torch.bfloat16, dev), ws, n, s)
    if st:
        _check(st, "svdq_linear_w4a16")


def svdq_linear_w4a16_workspace_bytes(w: Weights, M: int) -> int:
    return _lib.svdq_linear_w4a16_workspace_bytes(w.handle, M)


def _norm_params(scale, shift, M: int, K: int, group_rows: int, dev: int) -> tuple:
    """(svdq_dtype, elements between groups, addresses) of the per-group vectors [groups, K]."""
    shape = (-(-M // (group_rows or M)) if M else 0, K)
    if scale is None and shift is None:
        return 2, 0, None, None
    sp, ld = _rows_arg(scale, "scale", shape, DTYPES, dev) if scale is not None else (None, 0)
    if shift is None:
        return DTYPES[scale.dtype], ld, sp, None
    hp, ld_shift = _rows_arg(shift, "shift", shape, DTYPES, dev)
    if sp is not None and (scale.dtype != shift.dtype or ld != ld_shift):
        raise ValueError("scale and shift must have the same type and stride")
    return DTYPES[shift.dtype], ld_shift, sp, hp


@functools.lru_cache(maxsize=256)
def _norm_desc(*fields) -> NormDesc:
    return NormDesc(*fields)


def svdq_layer_norm(Z: torch.Tensor, scale: Optional[torch.Tensor], shift: Optional[torch.Tensor], Y: torch.Tensor,
                    stats: Optional[torch.Tensor], eps: float, group_rows: int = 0, plus_one: bool = False, ckpt=None,
                    stream=None) -> None:
    """Layer norm of the rows of a CUDA [M, K] tensor (bf16, fp16 or fp32) into Y.

    scale and shift are [groups, K] (one row per group_rows rows of Z, 0: all), stats float32 [M, 2];
    ckpt = (codes, scales, "int8" or "e4m3") also writes Z's 8-bit checkpoint (uint8 [M, K] and
    [M, ceil(K/32)]).
    """
    dev, s = _device_and_stream(stream)
    M, K = _shape2(Z, "Z")
    zp, ld_z = _rows_arg(Z, "Z", (M, K), DTYPES, dev)
    yp, ld_y = _rows_arg(Y, "Y", (M, K), (Z.dtype,), dev)
    pd, ld_p, sp, hp = _norm_params(scale, shift, M, K, group_rows, dev)
    stp = _arg(stats, "stats", (M, 2), torch.float32, dev) if stats is not None else None
    codes, scales, fmt = _ckpt(ckpt, M, K, dev)
    d = _norm_desc(M, K, group_rows, DTYPES[Z.dtype], pd, bool(plus_one), eps, ld_z, ld_y, 0, 0, ld_p)
    st = _lib.svdq_layer_norm(d, zp, sp, hp, yp, stp, codes, scales, fmt, s)
    if st:
        _check(st, "svdq_layer_norm")


def svdq_layer_norm_backward(dY: torch.Tensor, Z: Optional[torch.Tensor], stats: torch.Tensor,
                             scale: Optional[torch.Tensor], dZ: torch.Tensor, dscale: Optional[torch.Tensor],
                             dshift: Optional[torch.Tensor], workspace: Optional[torch.Tensor], group_rows: int = 0,
                             plus_one: bool = False, ckpt=None, stream=None) -> None:
    """Gradient of svdq_layer_norm from Z or (Z None) from its checkpoint; dscale and dshift float32 [groups, K]."""
    dev, s = _device_and_stream(stream)
    M, K = _shape2(dY, "dY")
    dyp, ld_dy = _rows_arg(dY, "dY", (M, K), DTYPES, dev)
    dzp, ld_dz = _rows_arg(dZ, "dZ", (M, K), (dY.dtype,), dev)
    zp, ld_z = _rows_arg(Z, "Z", (M, K), (dY.dtype,), dev) if Z is not None else (None, 0)
    pd, ld_p, sp, _ = _norm_params(scale, None, M, K, group_rows, dev)
    shape = (-(-M // (group_rows or M)) if M else 0, K)
    da = _arg(dscale, "dscale", shape, torch.float32, dev) if dscale is not None else None
    dc = _arg(dshift, "dshift", shape, torch.float32, dev) if dshift is not None else None
    stp = _arg(stats, "stats", (M, 2), torch.float32, dev)
    codes, scales, fmt = _ckpt(ckpt, M, K, dev)
    ws, n = _workspace(workspace, dev)
    d = _norm_desc(M, K, group_rows, DTYPES[dY.dtype], pd, bool(plus_one), 0.0, ld_z, 0, ld_dy, ld_dz, ld_p)
    st = _lib.svdq_layer_norm_backward(d, dyp, zp, codes, scales, fmt, stp, sp, dzp, da, dc, ws, n, s)
    if st:
        _check(st, "svdq_layer_norm_backward")


def svdq_layer_norm_backward_workspace_bytes(M: int, K: int, group_rows: int = 0) -> int:
    return _lib.svdq_layer_norm_backward_workspace_bytes(M, K, group_rows)


def svdq_ckpt8_encode(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, fmt: str = "int8",
                      stream=None) -> None:
    """8-bit checkpoint of a CUDA [M, K] tensor (bf16, fp16 or fp32) into uint8 [M, K] and [M, ceil(K/32)]."""
    dev, s = _device_and_stream(stream)
    M, K = _shape2(X, "X")
    xp, ld = _rows_arg(X, "X", (M, K), DTYPES, dev)
    cp, sp, f = _ckpt((codes, scales, fmt), M, K, dev)
    st = _lib.svdq_ckpt8_encode(xp, DTYPES[X.dtype], M, K, ld, f, cp, sp, s)
    if st:
        _check(st, "svdq_ckpt8_encode")


def svdq_ckpt8_decode(codes: torch.Tensor, scales: torch.Tensor, X: torch.Tensor, fmt: str = "int8",
                      stream=None) -> None:
    """The values of a checkpoint into a CUDA [M, K] tensor (bf16, fp16 or fp32)."""
    dev, s = _device_and_stream(stream)
    M, K = _shape2(X, "X")
    xp, ld = _rows_arg(X, "X", (M, K), DTYPES, dev)
    cp, sp, f = _ckpt((codes, scales, fmt), M, K, dev)
    st = _lib.svdq_ckpt8_decode(cp, sp, M, K, f, xp, DTYPES[X.dtype], ld, s)
    if st:
        _check(st, "svdq_ckpt8_decode")


def svdq_lowrank_wgrad(X: Optional[torch.Tensor], S: torch.Tensor, G: torch.Tensor, workspace: Optional[torch.Tensor],
                       ckpt=None, stream=None) -> None:
    """G [K, r] float32 = X^T S for CUDA bf16 X [M, K] (or, X None, its checkpoint) and S [M, r]."""
    dev, s = _device_and_stream(stream)
    M, r = _shape2(S, "S")
    K = _shape2(G, "G")[0]
    xp = _arg(X, "X", (M, K), torch.bfloat16, dev) if X is not None else None
    codes, scales, fmt = _ckpt(ckpt, M, K, dev)
    ws, n = _workspace(workspace, dev)
    st = _lib.svdq_lowrank_wgrad(xp, codes, scales, fmt, _arg(S, "S", (M, r), torch.bfloat16, dev), M, K, r,
                                 _arg(G, "G", (K, r), torch.float32, dev), ws, n, s)
    if st:
        _check(st, "svdq_lowrank_wgrad")


def svdq_lowrank_wgrad_workspace_bytes(M: int, K: int, r: int) -> int:
    return _lib.svdq_lowrank_wgrad_workspace_bytes(M, K, r)


def svdq_ckpt8_codes_bytes(M: int, K: int) -> int:
    return _lib.svdq_ckpt8_codes_bytes(M, K)


def svdq_ckpt8_scales_bytes(M: int, K: int) -> int:
    return _lib.svdq_ckpt8_scales_bytes(M, K)


def svdq_act_codes_bytes(M: int, K: int) -> int:
    return _lib.svdq_act_codes_bytes(M, K)


def svdq_act_sf_bytes(M: int, K: int) -> int:
    return _lib.svdq_act_sf_bytes(M, K)


def svdq_lowrank_bytes(w: Weights, M: int) -> int:
    return _lib.svdq_lowrank_bytes(w.handle, M)


def svdq_forward_workspace_bytes(w: Weights, M: int) -> int:
    return _lib.svdq_forward_workspace_bytes(w.handle, M)


def svdq_forward_host_workspace_bytes(w: Weights, M: int) -> int:
    return _lib.svdq_forward_host_workspace_bytes(w.handle, M)


def svdq_weights_info(w: Weights) -> dict:
    return w.info


def svdq_weights_rank(w: Weights) -> int:
    return int(_lib.svdq_weights_rank(w.handle))


def svdq_weights_export(w: Weights, residual: bool = False) -> dict:
    i = w.info
    N, K, r = i["N"], i["K"], i["rank"]
    out = {"codes": np.empty((N, K // 2), np.uint8), "sf": np.empty(_lib.svdq_weights_sf_bytes(w.handle), np.uint8),
           "L1p": np.empty((K, r), np.uint16), "L2": np.empty((r, N), np.uint16),
           "inv_lam": np.empty(K, np.float32), "bias": np.empty(N, np.float32)}
    if residual:
        out["residual"] = np.empty((N, K), np.float32)
    _check(_lib.svdq_weights_export(w.handle, out["codes"].ctypes.data, out["sf"].ctypes.data,
                                    out["L1p"].ctypes.data if r else None, out["L2"].ctypes.data if r else None,
                                    out["inv_lam"].ctypes.data, out["bias"].ctypes.data,
                                    out["residual"].ctypes.data if residual else None), "svdq_weights_export")
    out.update(i)
    return out


def svdq_set_wait_limit_ns(ns: int) -> None:
    _lib.svdq_set_wait_limit_ns(int(ns))


def svdq_search_alpha(W_bf16, X_bf16, bias_bf16=None, alphas=(0.3, 0.4, 0.5, 0.6, 0.7, 0.8), rank: int = 32,
                      refine_iters: int = 1, fmt: str = "nvfp4", stream=None):
    """(relative output error per alpha, index of the best) on the calibration batch X."""
    Wp, Wk = _host(W_bf16, np.uint16)
    Xp, Xk = _host(X_bf16, np.uint16)
    bp, bk = _host(bias_bf16, np.uint16)
    N, K = Wk.shape
    a = np.ascontiguousarray(np.asarray(alphas, np.float32))
    o = svdq_prepare_opts_default()
    o.rank, o.refine_iters = rank, refine_iters
    o.format = FORMATS[fmt]
    err = (ctypes.c_double * len(a))()
    best = ctypes.c_int(0)
    _check(_lib.svdq_search_alpha(Wp, Xp, Xk.shape[0], bp, N, K, a.ctypes.data, len(a), ctypes.byref(o),
                                  _stream(stream), err, ctypes.byref(best)), "svdq_search_alpha")
    return [float(err[i]) for i in range(len(a))], int(best.value)


def svdq_weights_refine_errors(w: Weights) -> list:
    """Residual quantization error of each split prepare tried (the kept one is the smallest)."""
    n = ctypes.c_int(0)
    _check(_lib.svdq_weights_refine_errors(w.handle, None, 0, ctypes.byref(n)), "svdq_weights_refine_errors")
    buf = (ctypes.c_double * max(1, n.value))()
    _check(_lib.svdq_weights_refine_errors(w.handle, buf, n.value, ctypes.byref(n)), "svdq_weights_refine_errors")
    return [float(buf[i]) for i in range(n.value)]


def svdq_selftest_codec() -> int:
    """Mismatch count of the encoder's exact division/reciprocal shortcuts on the current device."""
    out = ctypes.c_uint(0)
    _check(_lib.svdq_selftest_codec(ctypes.byref(out)), "svdq_selftest_codec")
    return int(out.value)


def svdq_check_device_errors(stream=None) -> int:
    """Returns the device error status (0 = none) after synchronizing the stream."""
    return _lib.svdq_check_device_errors(_stream(stream))


def svdq_last_error() -> str:
    return _lib.svdq_last_error().decode()


def svdq_version() -> str:
    return _lib.svdq_version().decode()


# ---------------------------------------------------------------- helpers
def act_buffers(w: Weights, M: int, device="cuda"):
    """Device buffers (xq, xsf, T) for one activation batch of M rows."""
    i = w.info
    xq = torch.empty(max(1, svdq_act_codes_bytes(M, i["K"])), dtype=torch.uint8, device=device)
    xsf = torch.empty(svdq_act_sf_bytes(M, i["K"]), dtype=torch.uint8, device=device)
    T = torch.empty((M, 2 * i["r_pad"]), dtype=torch.bfloat16, device=device) if i["r_pad"] else None
    return xq, xsf, T


def linear(w: Weights, X: torch.Tensor, stream=None) -> torch.Tensor:
    """Y = layer(X) for a CUDA bf16 X of shape [M, K] (both kernels)."""
    M = X.shape[0]
    xq, xsf, T = act_buffers(w, M, X.device)
    Y = torch.empty((M, w.info["N"]), dtype=torch.bfloat16, device=X.device)
    svdq_quantize_act_lowrank_down(w, X, xq, xsf, T, stream)
    svdq_linear_w4a4(w, xq, xsf, T, M, Y, stream)
    return Y
