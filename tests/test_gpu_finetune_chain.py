"""The operators as they are used together: fine-tuning a LoRA around a frozen 4-bit layer.

An embedding per image goes through a 4-bit modulation layer (few tokens, 16-bit activations) to the
(shift, scale) of an adaLN; the tokens' layer norm keeps an 8-bit checkpoint of its input; the W4A4
layer follows.  Backwards: the LoRA's factors from checkpoints, the layer norm from its checkpoint,
(scale, shift) gradients reduced over each image's tokens.  Three images of 40 tokens, the last one cut.
"""

import numpy as np
import pytest
import torch

from rows_common import U, ckpt_buffers, f64, half_step, lib, of_group, ref_backward, ref_norm, rows
from synth import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu

IMAGES, TOKENS, M, E, K, N, RANK, LORA = 3, 40, 113, 128, 256, 320, 16, 8


def handle(seed, n, k, rank):
    rng = np.random.default_rng(seed)
    L1 = f32_to_bf16_bits((rng.standard_normal((k, rank)) / np.sqrt(k)).astype(np.float32))
    L2 = f32_to_bf16_bits((rng.standard_normal((rank, n)) * 0.1).astype(np.float32))
    return lib().svdq_weights_from_factors(n, k, rank, np.ones(k, np.float32), L1, L2,
                                           (rng.standard_normal((n, k)) * 0.03).astype(np.float32),
                                           (rng.standard_normal(n) * 0.1).astype(np.float32))


class Chain:
    def __init__(self):
        L = lib()
        self.mod, self.w = handle(1, 2 * K, E, 8), handle(2, N, K, RANK)
        rng = np.random.default_rng(3)
        L.svdq_attach_lora(self.w, f32_to_bf16_bits((rng.standard_normal((K, LORA)) / 16).astype(np.float32)),
                           f32_to_bf16_bits((rng.standard_normal((LORA, N)) * 0.1).astype(np.float32)), 1.0)
        e = L.svdq_weights_export(self.w)
        self.A = torch.from_numpy(bf16_bits_to_f32(e["L1p"])[:, RANK:].copy()).cuda()
        self.B = torch.from_numpy(bf16_bits_to_f32(e["L2"])[RANK:].copy()).cuda()
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.emb, self.Z, self.dY = rows(4, IMAGES, E, torch.bfloat16), rows(5, M, K, torch.bfloat16), \
            rows(6, M, N, torch.bfloat16, 1e-2)
        self.dX = rows(7, M, K, torch.bfloat16, 1e-2)  # stands for what the layer hands back
        self.vec, self.X, self.Y, self.dZ = (torch.empty(s, **bf) for s in ((IMAGES, 2 * K), (M, K), (M, N), (M, K)))
        self.stats = torch.empty((M, 2), device="cuda")
        self.ck_z, self.ck_x = ckpt_buffers(M, K), ckpt_buffers(M, K)
        self.dA, self.dBt = torch.empty((K, LORA), device="cuda"), torch.empty((N, LORA), device="cuda")
        self.dscale, self.dshift = torch.empty((2, IMAGES, K), device="cuda")
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.ws = [torch.empty(n, **u8) for n in (L.svdq_linear_w4a16_workspace_bytes(self.mod, IMAGES),
                                                  L.svdq_forward_workspace_bytes(self.w, M),
                                                  L.svdq_lowrank_wgrad_workspace_bytes(M, K, LORA),
                                                  L.svdq_lowrank_wgrad_workspace_bytes(M, N, LORA),
                                                  L.svdq_layer_norm_backward_workspace_bytes(M, K, TOKENS))]

    def step(self):
        L = lib()
        L.svdq_linear_w4a16(self.mod, self.emb, self.vec, self.ws[0])
        shift, scale = self.vec[:, :K], self.vec[:, K:]
        L.svdq_layer_norm(self.Z, scale, shift, self.X, self.stats, 1e-6, group_rows=TOKENS, plus_one=True,
                          ckpt=self.ck_z + ("int8",))
        L.svdq_forward(self.w, self.X, self.Y, self.ws[1])
        L.svdq_ckpt8_encode(self.X, self.ck_x[0], self.ck_x[1], "int8")
        self.S = (self.dY.float() @ self.B.T).to(torch.bfloat16)
        self.T = (self.X.float() @ self.A).to(torch.bfloat16)
        L.svdq_lowrank_wgrad(None, self.S, self.dA, self.ws[2], ckpt=self.ck_x + ("int8",))
        L.svdq_lowrank_wgrad(self.dY, self.T, self.dBt, self.ws[3])
        L.svdq_layer_norm_backward(self.dX, None, self.stats, scale, self.dZ, self.dscale, self.dshift, self.ws[4],
                                   group_rows=TOKENS, plus_one=True, ckpt=self.ck_z + ("int8",))

    def results(self):
        return [t.clone() for t in (self.vec, self.X, self.Y, self.dA, self.dBt, self.dZ, self.dscale, self.dshift)]


def group_max(x):
    """Each value's group's largest magnitude."""
    return np.repeat(np.abs(x).reshape(x.shape[0], -1, 32).max(2), 32, 1)


def test_against_the_formulas_without_checkpoints():
    """Every result against float64 on unquantized inputs: the checkpoints' part in the difference is at most
    half a step, 2^-7 of a group's largest magnitude, carried through the formula."""
    c = Chain()
    c.step()
    assert lib().svdq_check_device_errors() == 0
    z, dx, x, vec = f64(c.Z), f64(c.dX), f64(c.X), f64(c.vec)
    m, shift = 1 + of_group(vec[:, K:], M, TOKENS), of_group(vec[:, :K], M, TOKENS)
    mu, rstd = ref_norm(z, 1e-6)
    xh = (z - mu) * rstd
    assert np.all(np.abs(x - (xh * m + shift)) <= 2.0 ** -8 * (np.abs(x) + 1e-3) + 1e-4 * np.abs(m))
    assert bool(c.Y.isfinite().all())

    off = group_max(x) * 2.0 ** -7
    s, t, dy = f64(c.S), f64(c.T), f64(c.dY)
    assert np.all(np.abs(f64(c.dA) - x.T @ s) <= off.T @ np.abs(s) + 64 * 2.0 ** -22 * np.abs(x).T @ np.abs(s))
    assert np.all(np.abs(f64(c.dBt) - dy.T @ t) <= 64 * 2.0 ** -22 * np.abs(dy).T @ np.abs(t))

    dz, da, dc, xh, g = ref_backward(z, dx, mu, rstd, m, TOKENS)
    d_xh = group_max(z) * 2.0 ** -7 * rstd + 80 * U * (np.abs(z) + np.abs(mu)) * rstd
    gx, gd = np.abs(g * xh).mean(1, keepdims=True), (np.abs(g) * d_xh).mean(1, keepdims=True)
    near = rstd * (d_xh * gx + np.abs(xh) * gd + d_xh * gd + 100 * U * (np.abs(g) + np.abs(g).mean(1, keepdims=True)
                                                                        + np.abs(xh) * gx))
    assert np.all(np.abs(f64(c.dZ) - dz) <= near + half_step(torch.bfloat16) * (np.abs(dz) + near))
    first = np.arange(0, M, TOKENS)
    total = lambda v: np.add.reduceat(v, first, axis=0)  # noqa: E731
    assert np.all(np.abs(f64(c.dscale) - da) <= total(np.abs(dx) * d_xh) + 64 * U * total(np.abs(dx * xh)))
    assert np.all(np.abs(f64(c.dshift) - dc) <= 64 * U * total(np.abs(dx)))
    # and no more than rounding to the nearest code costs: an error of variance step^2 / 12 in each value, where
    # the step is 2^(k - 6) for a group maximum in [2^k, 2^(k + 1)) (twice that from 1.992 2^k on); the norms
    # of some two thousand independent sums of such errors stay within a factor 1.5 of what that gives
    def spread(v, weights):  # expected norm of (errors of v)^T weights
        step = 2.0 ** (np.floor(np.log2(group_max(v))) - 5)  # the larger one
        return np.sqrt(np.sum((step ** 2 / 12).T @ weights ** 2))
    assert np.linalg.norm(f64(c.dA) - x.T @ s) <= 1.5 * spread(x, s)
    scatter = np.sqrt(np.sum(total((2.0 ** (np.floor(np.log2(group_max(z))) - 5) * rstd * dx) ** 2 / 12)))
    assert np.linalg.norm(f64(c.dscale) - da) <= 1.5 * scatter


def test_one_graph_of_the_whole_run():
    c = Chain()
    c.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.step()
    for t, seed in ((c.emb, 14), (c.Z, 15), (c.dY, 16), (c.dX, 17)):
        t.copy_(rows(seed, *t.shape, torch.bfloat16, 1e-2 if t is c.dY or t is c.dX else 1.0))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    replayed = c.results()
    c.step()
    for a, b in zip(replayed, c.results()):
        assert torch.equal(a, b)
    assert lib().svdq_check_device_errors() == 0
