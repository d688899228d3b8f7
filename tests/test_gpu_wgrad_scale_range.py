"""The low-rank gradient from checkpoints whose scale times S leaves bf16's range although code * scale does not."""

import numpy as np
import pytest
import torch

from rows_common import f64, ref_decode, rows
from test_gpu_lowrank_wgrad import check, wgrad

pytestmark = pytest.mark.gpu


def codes_of(values, fmt):
    v = torch.as_tensor(values, dtype=torch.float32)
    return (v.to(torch.int8) if fmt == "int8" else v.to(torch.float8_e4m3fn)).view(torch.uint8).cuda()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("r", [3, 8, 16, 40])
def test_a_zero_next_to_a_very_large_value(r, fmt):
    """scale * S beyond 2^128: columns whose code is 0 there keep their sums."""
    M, K = 70, 128
    rng = np.random.default_rng(r)
    codes = codes_of(rng.integers(-15, 16, (M, K)), fmt)
    scales = torch.full((M, K // 32), 120, dtype=torch.uint8, device="cuda")
    row = 37
    codes[row] = 0
    codes[row, 5] = codes_of([8.0], fmt)[0]  # 2^100 times 2^40: beyond fp32, in this column alone
    scales[row, 0] = 127 + 97
    S = rows(5, M, r, torch.bfloat16, outliers=False)
    S[row] = 2.0 ** 40
    G = wgrad(None, S, (codes, scales, fmt))
    keep = [k for k in range(K) if k != 5]
    x = ref_decode(codes.cpu().numpy(), scales.cpu().numpy(), fmt)
    assert bool(G[keep].isfinite().all()) and bool((G[5] == float("inf")).all())
    check(G[keep], x[:, keep], f64(S))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("r", [3, 8, 16, 40])
def test_small_values_times_small_ones(r, fmt):
    """scale * S below 2^-126: the products (2^-121) and the sums are ordinary fp32 values and keep their bits."""
    M, K = 96, 64
    codes = codes_of(np.full((M, K), 120.0), fmt)
    scales = torch.full((M, K // 32), 127 - 76, dtype=torch.uint8, device="cuda")
    S = torch.full((M, r), (1 + 127 / 128) * 2.0 ** -53, dtype=torch.bfloat16, device="cuda")
    check(wgrad(None, S, (codes, scales, fmt)), ref_decode(codes.cpu().numpy(), scales.cpu().numpy(), fmt), f64(S))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_the_largest_and_smallest_values(fmt):
    """Values next to 2^128 and at 2^-120 in the same sums, each where S brings its products into range."""
    M, K, r = 64, 64, 16
    top = 127.0 if fmt == "int8" else 448.0
    codes = codes_of(np.where(np.arange(M)[:, None] % 2, top, 64.0) * np.ones((M, K)), fmt)
    cap = 248 if fmt == "int8" else 246
    scales = torch.where(torch.arange(M) % 2 == 1, cap, 127 - 126)[:, None].repeat(1, 2).to(torch.uint8).cuda()
    S = torch.where(torch.arange(M) % 2 == 1, 2.0 ** -124, 2.0 ** 120)[:, None].repeat(1, r).to(torch.bfloat16).cuda()
    check(wgrad(None, S, (codes, scales, fmt)), ref_decode(codes.cpu().numpy(), scales.cpu().numpy(), fmt), f64(S))
