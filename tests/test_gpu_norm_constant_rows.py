"""Layer norm of rows without variance: where the row's sum is exact in fp32 (bf16 and fp16 values, whole numbers) the
mean is the value itself, so Y is the offset exactly, at every width."""

import pytest
import torch

from rows_common import DT
from test_gpu_layer_norm import forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("K", [1, 7, 60, 97, 448, 640, 896, 960, 1001, 1792, 1920, 2056, 3584, 7168, 10496, 16376])
def test_values_of_eight_bits(K, dt):
    Z = (torch.arange(128, 256, device="cuda").float() / 16)[:, None].repeat(1, K).to(DT[dt])
    Z[::2] *= -1
    shift = torch.linspace(-1, 1, K, device="cuda")[None]
    Y, stats = forward(Z, None, shift, eps=1e-6)
    assert torch.equal(stats[:, 0], Z[:, 0].float())
    assert torch.equal(Y, shift.to(DT[dt]).expand_as(Y))
