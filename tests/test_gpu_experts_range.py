"""moe_experts with weighted activations next to the largest that its header allows,
2^112: the sums of a chunk's products stay finite before the scale makes them
ordinary numbers."""

import pytest
import torch

import fp8_block_scaled_04_amd as fb
from tests.gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_gpu()


# every form of the second product
@pytest.mark.parametrize("tile,T,H,I,E", [
    ((16, 8, 16, 8), 3, 2048, 256, 9), ((16, 16, 16, 4), 16, 128, 2304, 3), ((16, 8, 32, 1), 17, 2048, 256, 9),
    ((16, 16, 32, 4), 40, 256, 1152, 40), ((16, 16, 64, 4), 50, 1024, 640, 40), ((16, 16, 64, 1), 60, 4096, 128, 100),
    ((64, 128, 256, 4), 128, 384, 1024, 8)])
def test_experts_of_large_activations(tile, T, H, I, E):
    assert fb.moe_experts_tile(T, H, I, E, 1) == tile
    # gates of 127 (1 / (1 + exp(-127)) is 1), u = 1, weights 2^105: activations of 127 2^105 < 2^112, exact in BF16;
    # 128 of them times 448 are 889 2^118 < 2^128
    x = torch.zeros(T, H, device=DEV)
    x[:, :127] = 1
    w13 = torch.ones(E, 2 * I, H, device=DEV)
    w13[:, I:] = 0
    w13[:, I:, 0] = 1
    codes = lambda t: t.to(torch.float8_e4m3fn)  # noqa: E731
    one = lambda *n: torch.ones(*n, device=DEV)  # noqa: E731
    ids = (torch.arange(T, device=DEV, dtype=torch.int32) % E).view(T, 1)
    got = fb.moe_experts(codes(x), one(H // 128, T), ids, one(T, 1) * 2.0 ** 105, codes(w13), one(E, 2 * I // 128, H // 128),
                         codes(one(E, H, I) * 448), one(E, H // 128, I // 128) * 2.0 ** -20, out_dtype=torch.float32)
    # whole multiples (I / 128 of them) of 889 2^98: exact
    assert (got == 889.0 * 2.0 ** 98 * (I // 128)).all()
