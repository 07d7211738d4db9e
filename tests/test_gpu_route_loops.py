"""moe_route and moe_route_backward with more tokens than all workgroups hold at
once, every kernel: each row bit for bit that of a call that needs no second turn."""

import pytest
import torch

import fp8_block_scaled_04_amd as fb
from tests.gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu
WORKGROUPS = 2048


def setup_module(module):
    require_gpu()


# 16 tokens per workgroup up to 256 experts and 16 places, else four
@pytest.mark.parametrize("e,topk,tokens", [(8, 2, 16), (100, 5, 16), (256, 8, 16), (256, 16, 16), (257, 4, 4), (1024, 64, 4),
                                           (64, 20, 4), (200, 17, 4)])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_of_more_tokens_than_workgroups(e, topk, tokens, kind, renorm):
    once = WORKGROUPS * tokens
    t = 2 * once + 3
    gen = torch.Generator(device=DEV).manual_seed(e)
    x = (2 * torch.randn(t, e, generator=gen, device=DEV)).to(kind)
    x[torch.rand(t, e, generator=gen, device=DEV) < 0.02] = -torch.inf
    x[1::97] = torch.nan                                # (rows without any expert)
    dw = torch.randn(t, topk, generator=gen, device=DEV)
    ids, w = fb.moe_route(x, topk, renormalize=renorm)
    back = fb.moe_route_backward(x, ids, dw, renormalize=renorm)
    part = once // 2 - 8
    for t0 in range(0, t, part):
        s = slice(t0, min(t, t0 + part))
        i1, w1 = fb.moe_route(x[s].clone(), topk, renormalize=renorm)
        assert torch.equal(ids[s], i1) and torch.equal(w[s], w1)
        b1 = fb.moe_route_backward(x[s].clone(), i1, dw[s].clone(), renormalize=renorm)
        assert torch.equal(back[s], b1)
    assert (ids[1::97] == -1).all() and (w[1::97] == 0).all() and (back[1::97] == 0).all()
