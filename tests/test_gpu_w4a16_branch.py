"""The few-token layer's low-rank branch holds T = X L1' in fp32 up to the product with L2.

Whole numbers make every step exact: x and L1' are integers of at most 8 bits, T an integer below 2^23 (its
sums are exact in fp32 in any order), L2 / alpha_w is 1 or -1, the 4-bit weights and the bias are 0.  Two ranks
whose T differ by a small integer then give that integer, and nothing else: a T of fewer than 23 bits is off by
whole steps.
"""

import numpy as np
import pytest
import torch

from rows_common import lib
from synth import f32_to_bf16_bits
from test_gpu_w4a16 import run

pytestmark = pytest.mark.gpu


def empty_handle(N, K, rank, L1, L2, fmt, inv=None, alpha=1.0, bias=None):
    """A handle without a 4-bit part."""
    n = 256 if fmt == "int4" else 128
    sf = np.zeros(-(-N // n) * n * (K // 64 * 2 if fmt == "int4" else K // 16), np.uint8)
    return lib().svdq_weights_from_codes(N, K, rank, alpha, np.zeros((N, K // 2), np.uint8), sf,
                                         np.ones(K, np.float32) if inv is None else inv,
                                         f32_to_bf16_bits(L1.astype(np.float32)), f32_to_bf16_bits(L2.astype(np.float32)),
                                         bias, fmt=fmt)


@pytest.mark.parametrize("fmt", ["nvfp4", "int4"])
@pytest.mark.parametrize("M,K,N,pairs", [(1, 64, 16, 1), (3, 256, 144, 8), (5, 512, 272, 16), (16, 128, 640, 40),
                                         (8, 448, 4112, 64)])
def test_differences_of_the_branch(M, K, N, pairs, fmt):
    rng = np.random.default_rng(M + K + N)
    x = rng.integers(-255, 256, (M, K))
    L1 = np.zeros((K, 2 * pairs), np.int64)
    L1[:, 0::2] = rng.integers(-127, 128, (K, pairs))
    L1[:, 1::2] = L1[:, 0::2]
    k = rng.integers(0, K, pairs)
    step = rng.integers(1, 3, pairs)  # the second rank of a pair: one entry less by 1 or 2
    L1[k, 2 * np.arange(pairs) + 1] -= step
    T = x @ L1
    assert np.abs(T).max() < 2 ** 23 and (M * K < 500 or np.abs(T).max() > 2 ** 17)
    L2 = np.zeros((2 * pairs, N), np.int64)
    of = rng.integers(0, pairs, N)
    L2[2 * of, np.arange(N)], L2[2 * of + 1, np.arange(N)] = 1, -1
    w = empty_handle(N, K, 2 * pairs, L1, L2, fmt)
    X = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()
    want = T @ L2
    assert np.abs(want).max() <= 2 * 255
    got = run(w, X).double().cpu().numpy()
    # the integers have at most 9 bits: bf16 keeps 8
    assert np.all(np.abs(got - want) <= np.abs(want) * 2.0 ** -8)
