"""Long sums against bounds counted from how the kernels share them out, tight enough that a row left out or taken twice
always shows: every term is between 1 and 4, and the bounds are below 1.

Low-rank gradient: a warp adds the rows of one accumulator by at most 32 products of 16 rows each, each off by up to
2^-22 of the absolute sum (the tensor cores truncate); the CTA's row warps (16, 8 or 4) and the parts of the rows follow
by ordinary additions.  Column sums of the layer norm's gradient: a thread's rows, the CTA's teams, the splits.
"""

import pytest
import torch

from rows_common import U, ckpt_buffers, lib
from test_gpu_layer_norm import backward
from test_gpu_lowrank_wgrad import wgrad

pytestmark = pytest.mark.gpu


def between_1_and_2(seed, M, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1 + torch.rand((M, K), generator=g, device="cuda")).clamp(max=1.99).to(dtype)


@pytest.mark.parametrize("src", ["values", "int8", "e4m3"])
@pytest.mark.parametrize("M,K,r", [(20003, 4400, 2), (9001, 48, 20), (8197, 2304, 33), (4608, 12288, 8)])
def test_low_rank_gradient(M, K, r, src):
    X, S = between_1_and_2(1, M, K, torch.bfloat16), between_1_and_2(2, M, r, torch.bfloat16)
    ck = None
    if src != "values":
        ck = ckpt_buffers(M, K)
        lib().svdq_ckpt8_encode(X, ck[0], ck[1], src)
        lib().svdq_ckpt8_decode(ck[0], ck[1], X, src)
        assert float(X.min()) >= 1.0
    G = wgrad(None if ck else X, S, ck and ck + (src,))
    ref = X.double().T @ S.double()
    parts = max(1, lib().svdq_lowrank_wgrad_workspace_bytes(M, K, r) // (K * r * 4))
    row_warps = 4 if K > 17 * 256 else 8 if K > 17 * 128 else 16
    bound = (32 * 2.0 ** -22 + (row_warps + parts) * U) * ref
    assert float(bound.max()) < 1.0
    assert bool(((G.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("M,K,gr", [(3001, 8192, 0), (8192, 640, 0), (5000, 4096, 1300), (2999, 1001, 0), (2048, 12288, 0),
                                    (6000, 64, 5000)])
def test_column_sums(M, K, gr):
    rows = gr or M
    groups = -(-M // rows)
    Z, dY = between_1_and_2(3, M, K, torch.float32), between_1_and_2(4, M, K, torch.float32)
    stats = torch.tensor([[-1.0, 0.5]], device="cuda").repeat(M, 1)  # xh in [1, 1.5]
    _, da, dc = backward(dY, Z, stats, None, M, K, gr)
    xh = (Z.double() + 1) * 0.5
    chunks = -(-K // 8)
    nv = 1 if chunks <= 32 else 2 if chunks <= 1024 else 3 if chunks <= 1536 else 4
    warps = -(-chunks // (32 * nv))
    teams = min(max(1, 16 // warps), rows)
    splits = max(1, lib().svdq_layer_norm_backward_workspace_bytes(M, K, gr) // (groups * 2 * K * 4))
    n = -(-rows // (splits * teams)) + teams + splits
    for g in range(groups):
        at = slice(g * rows, min(M, (g + 1) * rows))
        for got, terms, own in ((da[g], dY.double()[at] * xh[at], 3), (dc[g], dY.double()[at], 0)):
            ref = terms.sum(0)  # `own`: roundings of z - mu, of xh and of the product
            bound = (n + own) * U * ref
            assert float(bound.max()) < 1.0
            assert bool(((got.double() - ref).abs() <= bound).all())
