"""moe_experts, exactly, where workgroups walk several items of the narrow kernels:
the next item's scales, accumulators, activations and the sum over waves in LDS
used again."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_04_amd as fb
from oracle import layer
from tests.gpu_util import DEV, require_gpu
from tests.layer_util import expert_dev
from tests.test_gpu_experts import check_exact, exact_case

pytestmark = pytest.mark.gpu
CUS = 256


def setup_module(module):
    require_gpu()


def items(w, tile):
    """(items, items that all workgroups hold at once) of the two products: a job
    is up to 16 rows of an expert; four workgroups per CU, three in the second."""
    rows, up, down, waves = tile
    ids, I, H = w["ids"], w["w2"].shape[2], w["w2"].shape[1]
    jobs = sum(-(-int((ids == e).any(1).sum()) // rows) for e in range(w["w2"].shape[0]))
    return (jobs * (I // up), 4 * CUS), (jobs * (H // down), 3 * CUS * 4 // waves)


# each form of the second product, with 8 and 16 columns in the first
@pytest.mark.parametrize("tile,T,H,I,E,topk", [
    ((16, 8, 16, 4), 128, 1024, 384, 4, 4), ((16, 8, 32, 4), 128, 1024, 384, 8, 8), ((16, 16, 64, 4), 100, 1024, 384, 20, 8),
    ((16, 8, 32, 1), 128, 4096, 128, 7, 7), ((16, 16, 64, 1), 128, 2048, 128, 60, 16)])
def test_experts_with_more_items_than_workgroups(tile, T, H, I, E, topk):
    assert fb.moe_experts_tile(T, H, I, E, topk) == tile
    w = exact_case(T, H, I, E, topk, seed=T + H + I)
    (up, most_up), (down, most_down) = items(w, tile)
    assert down > most_down and (up > most_up or I == 128)
    got = check_exact(w)
    assert torch.equal(check_exact(w), got)
    # and with places outside, so that jobs are cut short
    w["ids"][np.random.default_rng(1).random((T, topk)) < 0.1] = -1
    check_exact(w)


@pytest.mark.parametrize("T,H,I,E,topk", [(128, 1024, 384, 4, 4), (100, 1024, 384, 20, 8)])
def test_experts_with_more_items_into_bf16(T, H, I, E, topk):
    w = exact_case(T, H, I, E, topk, seed=T + E)
    want = torch.from_numpy(layer.experts(**w)[0]).to(DEV).to(torch.bfloat16)      # (exact in FP32: rounded once)
    assert torch.equal(fb.moe_experts(*expert_dev(w)), want)
