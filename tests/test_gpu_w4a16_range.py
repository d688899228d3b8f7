"""The few-token layer where the branch and the 4-bit part are of very unlike size, and at the ends of the range."""

import numpy as np
import pytest
import torch

from rows_common import lib
from test_gpu_w4a16 import layer, run, tokens, weights

pytestmark = pytest.mark.gpu


def with_smoothing(w, inv, alpha=None):
    """The handle `w` with other smoothing factors (and, on request, another alpha_w)."""
    L = lib()
    e = L.svdq_weights_export(w)
    return L.svdq_weights_from_codes(e["N"], e["K"], e["rank"], alpha or e["alpha_w"], e["codes"], e["sf"],
                                     inv.astype(np.float32), e["L1p"], e["L2"], e["bias"], fmt=e["format"])


@pytest.mark.parametrize("fmt", ["nvfp4", "int4"])
@pytest.mark.parametrize("factor", [0.0, 2.0 ** -149, 2.0 ** -120, 2.0 ** -60])
@pytest.mark.parametrize("scale", [1.0, 1e6, 1e30])
def test_tokens_that_the_smoothing_leaves_nothing_of(fmt, factor, scale):
    """x inv_lam is zero or tiny where x is not (the branch sees x alone): Y is T L2 + b and whatever is left."""
    N, K = 272, 320
    w, _ = layer(21, N, K, 24, fmt)
    inv = np.full(K, factor)
    inv[64:128] = 1.0
    w = with_smoothing(w, inv)
    W, L1, L2, inv, b = weights(w)
    X = tokens(22, 5, K, scale).clamp(-1e34, 1e34)
    X[:4, 64:128] = 0.0  # the last token has ordinary channels
    X[3] = 0.0
    x = X.double().cpu().numpy()
    ref = (x * inv) @ W.T + (x @ L1) @ L2 + b
    mag = np.abs(x * inv) @ np.abs(W).T + (np.abs(x) @ np.abs(L1)) @ np.abs(L2) + np.abs(b)
    # K / 128 + 32 MMA results of 2^-22 as for any token; activations to 2^-38 of the token's largest
    floor = np.max(np.abs(x * inv), axis=1, keepdims=True) * 2.0 ** -38 * np.abs(W).sum(1)
    near = (K / 128 + 32) * 2.0 ** -22 * mag + floor
    y = run(w, X).double().cpu().numpy()
    assert np.isfinite(y).all()
    assert np.all(np.abs(y - ref) <= near + 2.0 ** -8 * (np.abs(ref) + near))


@pytest.mark.parametrize("alpha,x", [(2.0 ** -100, 2.0 ** -37), (2.0 ** -60, 2.0 ** -80), (2.0 ** -40, 1.0), (2.0 ** -14, 1.0),
                                     (2.0 ** 20, 2.0 ** 60), (2.0 ** 40, 2.0 ** 60)])
def test_factors_of_the_weights_at_the_ends_of_the_range(alpha, x):
    """Every weight is 6 * 448 alpha_w and every activation x: Y is exact.  alpha_w times the token's power of two
    (x 2^-13) leaves fp32's range at the first two, where Y is 2^-116 and 2^-119."""
    N, K = 16, 1024
    w = lib().svdq_weights_from_codes(N, K, 0, alpha, np.full((N, K // 2), 0x77, np.uint8), np.full(128 * K // 16, 0x7E, np.uint8),
                                      np.ones(K, np.float32), None, None, None, fmt="nvfp4")
    X = torch.full((3, K), x, dtype=torch.bfloat16, device="cuda")
    X[1] = 0.0
    X[2, 1:] = 0.0
    want = X.double().sum(1, keepdim=True) * 2688.0 * alpha
    assert float(want[0, 0]) > 2.0 ** -120
    assert torch.equal(run(w, X).double(), want.expand(3, N))
