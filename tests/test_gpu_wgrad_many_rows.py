"""The low-rank gradient of more rows than 65535 parts of them hold."""

import numpy as np
import pytest
import torch

from rows_common import lib

pytestmark = pytest.mark.gpu


def test_half_a_billion_rows():
    """Whole numbers at a few rows, the first and the last among them: every sum is exact."""
    M, K, r = 537_000_003, 16, 2
    L = lib()
    rng = np.random.default_rng(1)
    at = np.unique(np.concatenate([[0, 1, M // 2, M - 2, M - 1], rng.integers(0, M, 3000)]))
    v = rng.integers(-100, 101, (len(at), K)).astype(np.int8)
    codes = torch.zeros((M, K), dtype=torch.uint8, device="cuda")
    scales = torch.full((M, 1), 127, dtype=torch.uint8, device="cuda")
    S = torch.ones((M, r), dtype=torch.bfloat16, device="cuda")
    S[:, 1] = -2.0
    codes[torch.from_numpy(at).cuda()] = torch.from_numpy(v).view(torch.uint8).cuda()
    G = torch.full((K, r), 5.0, device="cuda")
    ws = torch.empty(L.svdq_lowrank_wgrad_workspace_bytes(M, K, r), dtype=torch.uint8, device="cuda")
    L.svdq_lowrank_wgrad(None, S, G, ws, ckpt=(codes, scales, "int8"))
    want = v.astype(np.int64).sum(0)[:, None] * np.array([1, -2])
    assert np.array_equal(G.double().cpu().numpy(), want.astype(np.float64))
