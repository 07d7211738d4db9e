"""The sums over rows of rms_norm_backward, held to the roundings that their order
has: the rows of a group that one lane adds in turn, the lanes of a workgroup that
share a group, 64 runs of groups in turn, and a tree over the runs."""

import numpy as np
import pytest

import fp8_block_scaled_04_amd as fb
from oracle import bf16, layer
from tests.gpu_util import bf16_dev, f32_dev, require_gpu
from tests.layer_util import rows_bits, weight_of

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def setup_module(module):
    require_gpu()


@pytest.mark.parametrize("m,k", [(3, 256), (64, 128), (513, 2048), (1100, 384), (1025, 2048), (4097, 512), (9001, 128),
                                 (2053, 1024), (700, 4224), (5000, 2176)])
def test_dweight_within_its_chain_of_additions(m, k):
    rng = np.random.default_rng(m + 2 * k)
    w, raw = weight_of(rng, k, "bf16")
    h, dy = rows_bits(rng, m, k), rows_bits(rng, m, k, 1e-3)
    rstd = layer.norm(h, None, w, 1e-6)[1].astype(np.float32)
    dw = fb.rms_norm_backward(bf16_dev(dy), bf16_dev(h), f32_dev(rstd), bf16_dev(raw))[1].cpu().numpy()
    groups = fb.rms_norm_backward_workspace_bytes(m, k) // (4 * k)
    # rows at once: up to 512 lanes of 8 columns, whole waves, as long as every group has that many rows
    lanes, rows = -(-k // 512) * 64, 1
    while k <= 2048 and 2 * rows * lanes <= 512 and 2 * rows * groups <= m:
        rows *= 2
    # roundings: h rstd, one per addition (the product with dy is exact inside its fma)
    chain = 1 + -(-m // (groups * rows)) + (rows - 1) + -(-groups // 64) + 6
    n = np.abs(bf16.to_f32(h).astype(np.float64) * rstd[:, None].astype(np.float64))
    size = (np.abs(bf16.to_f32(dy).astype(np.float64)) * n).sum(0)
    err = np.abs(dw - layer.norm_backward(dy, h, rstd, w)[1])
    print(f"{m} x {k}: {rows} rows at once, {chain} roundings, used {float((err / (size * U)).max()):.2f}")
    assert np.all(err <= chain * U * size * (1 + chain * U))
