"""moe_route and moe_route_backward against the float64 oracle.

u = 2^-24.  exp(x - top) is off by the rounding of x - top, |x - top| u, and at
most 2 steps (4 u) of expf; a sum of up to 1024 such terms passes 16 additions in
a lane and 6 in a wave (22 u, and the terms' own error, at most 0.4 u from x - top
in the sum, as d exp(-d) < 0.4), and a division rounds once: (|x - top| + 32) u.
The gradient adds two products and a sum over the places, 64 + 2 roundings at
most, 2 |x - top| more for the second weight.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_04_amd as fb
from oracle import bf16, layer
from tests.gpu_util import DEV, bf16_dev, f32_dev, i32_dev, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def setup_module(module):
    require_gpu()


def make(rng, t, e, kind, spread=2.0):
    x = rng.standard_normal((t, e)) * spread
    if kind == "bf16":
        b = bf16.from_f64_rne(x)
        return bf16.to_f32(b).astype(np.float64), bf16_dev(b)
    x = x.astype(np.float32)
    return x.astype(np.float64), f32_dev(x)


def distance(x):
    """top - x of the logits that count, 0 elsewhere."""
    live = np.where(np.isfinite(x), x, -np.inf)
    top = live.max(1, keepdims=True)
    known = np.isfinite(x) & np.isfinite(top)
    return np.where(known, np.where(known, top, 0.0) - np.where(known, x, 0.0), 0.0)


def check(x, dev, topk, renorm, seed=0):
    ids, w = fb.moe_route(dev, topk, renormalize=renorm)
    ids_ref, w_ref = layer.route(x, topk, renorm)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    d = distance(x)
    at = np.where(ids_ref >= 0, np.take_along_axis(d, np.maximum(ids_ref, 0), 1), 0)
    got = w.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - w_ref) <= (at + 32) * U * w_ref + 2.0 ** -126)
    dw = np.random.default_rng(seed).standard_normal(ids_ref.shape).astype(np.float32)
    dl = fb.moe_route_backward(dev, ids, f32_dev(dw), renormalize=renorm)
    assert dl.dtype == dev.dtype
    ref = layer.route_backward(x, ids_ref, dw, renorm)
    # p_i (|G_i| + sum p |G|)
    size = np.zeros(x.shape)
    for t in range(x.shape[0]):
        v = np.where(np.isnan(x[t]), -np.inf, x[t])
        on = [e for e in ids_ref[t] if e >= 0]
        p = np.zeros(v.size)
        if renorm:
            p[on] = layer._softmax(v[on])
        else:
            p = layer._softmax(v)
        g = np.zeros(v.size)
        g[on] = np.abs(dw[t, :len(on)])
        size[t] = p * (g + np.dot(p, g))
    half = 2.0 ** -8 if dev.dtype == torch.bfloat16 else U
    assert np.all(np.abs(dl.float().cpu().numpy() - ref) <= half * np.abs(ref) + (3 * d + 128) * U * size + 2.0 ** -126)


@pytest.mark.parametrize("t,e,topk", [(1, 1, 1), (1, 8, 2), (3, 64, 6), (5, 65, 1), (37, 128, 8), (9, 256, 8), (4, 257, 16),
                                      (2, 1024, 64), (7, 60, 60), (6, 64, 64), (130, 32, 4), (3, 200, 9),
                                      (18, 256, 16), (5, 256, 17), (66, 16, 16), (3, 5, 4), (33, 100, 1)])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route(t, e, topk, kind, renorm):
    x, dev = make(np.random.default_rng(t * 1000 + e), t, e, kind)
    check(x, dev, topk, renorm)


# Rows that are whole pieces of 4 and 8 logits and rows that are not, for each number of experts per lane; a last piece
# in the middle of the lanes.
@pytest.mark.parametrize("t,e,topk", [(5, 4, 4), (17, 12, 3), (2, 62, 7), (19, 72, 5), (4, 76, 16), (6, 127, 8), (21, 131, 8),
                                      (7, 132, 2), (16, 136, 16), (3, 252, 10), (15, 248, 8), (9, 254, 1), (40000, 8, 2)])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_of_whole_and_broken_pieces(t, e, topk, kind, renorm):
    x, dev = make(np.random.default_rng(t * 1000 + e), t, e, kind)
    check(x, dev, topk, renorm)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_ties_and_signed_zeros(renorm):
    rng = np.random.default_rng(1)
    x = rng.integers(-1, 2, (20, 96)).astype(np.float32)
    x[x == 0] *= -1.0                                   # -0 here, +0 there: equal
    x[::2][x[::2] == 0] = 0.0
    x[3] = 0.0
    x[3, ::3] = -0.0
    check(x.astype(np.float64), f32_dev(x), 10, renorm)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_left_out(kind, renorm):
    # -inf and NaN experts, rows with fewer than topk left, rows with none
    rng = np.random.default_rng(2)
    x = rng.standard_normal((12, 70))
    x = bf16.to_f32(bf16.from_f64_rne(x)).astype(np.float64)
    x[0, ::2] = -np.inf
    x[1, 5:] = -np.inf
    x[2, 2:] = np.nan
    x[3] = -np.inf
    x[4] = np.nan
    x[5, :] = -np.inf
    x[5, 69] = -200.0
    x[6] = np.finfo(np.float32).min if kind == "fp32" else bf16.to_f32(np.uint16(0xFF7F))   # the type's lowest value
    x[7] = x[6, 0]
    x[7, 40] = 1.0
    dev = f32_dev(x) if kind == "fp32" else bf16_dev(bf16.from_f64_rne(x))
    check(x, dev, 6, renorm)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_infinite_and_far_logits(renorm):
    x = np.zeros((4, 40))
    x[0, [3, 17]] = np.inf
    x[1, 9] = np.inf
    x[2] = np.linspace(-1e30, 1e30, 40)
    x[3] = np.linspace(-90, 0, 40)
    x = x.astype(np.float32)
    ids, w = fb.moe_route(f32_dev(x), 4, renormalize=renorm)
    ids_ref, w_ref = layer.route(x, 4, renorm)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    assert np.allclose(w.cpu().numpy(), w_ref, rtol=200 * U, atol=2.0 ** -126)
    dl = fb.moe_route_backward(f32_dev(x), ids, torch.ones(4, 4, device=DEV), renormalize=renorm)
    assert torch.isfinite(dl).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_of_other_ids(renorm, wide):
    # an id twice, ids outside, places without one
    rng = np.random.default_rng(4)
    x = rng.standard_normal((6, 10)).astype(np.float32)
    ids = np.array([[1, 1, 3], [-1, -1, -1], [9, 10, 2], [4, -5, 4], [1 << 30, 0, -1], [7, 7, 7]], np.int32)
    if wide:                                            # (more experts than 16 lanes hold)
        x = np.concatenate([x, np.full((6, 290), -np.inf, np.float32)], 1)
        ids[2, 1] = 300
    dw = rng.standard_normal((6, 3)).astype(np.float32)
    dl = fb.moe_route_backward(f32_dev(x), i32_dev(ids), f32_dev(dw), renormalize=renorm).cpu().numpy()
    assert np.allclose(dl, layer.route_backward(x, ids, dw, renorm), rtol=0, atol=400 * U)


def test_route_of_no_tokens_and_many():
    ids, w = fb.moe_route(torch.empty(0, 8, device=DEV), 2)
    assert ids.shape == w.shape == (0, 2)
    assert fb.moe_route_backward(torch.empty(0, 8, device=DEV), ids, w).shape == (0, 8)
    t = 4 * (1 << 20) + 9                                # more tokens than workgroups hold at once
    x = torch.randn(t, 8, device=DEV)
    ids, w = fb.moe_route(x, 2)
    pick = [0, 1, 4 * (1 << 20) - 1, 4 * (1 << 20), t - 1]
    i1, w1 = fb.moe_route(x[pick].contiguous(), 2)
    assert torch.equal(ids[pick], i1) and torch.equal(w[pick], w1)
    g = fb.moe_route_backward(x, ids, w)
    assert torch.equal(g[pick], fb.moe_route_backward(x[pick].contiguous(), i1, w1))


def test_route_refuses():
    x = torch.zeros(4, 8, device=DEV)
    i = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    for call in (lambda: fb.moe_route(x, 0), lambda: fb.moe_route(x, 9), lambda: fb.moe_route(x[:, ::2], 2),
                 lambda: fb.moe_route(x, (1 << 32) + 2), lambda: fb.moe_route_backward(x, i[:3], x[:3, :2].contiguous()),
                 lambda: fb.moe_route_backward(x, i, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        fb.moe_route(x.half(), 2)
    with pytest.raises(TypeError):
        fb.moe_route_backward(x, i.long(), x[:, :2].contiguous())
    with pytest.raises(fb.Fp8bsError):
        fb.moe_route(torch.zeros(2, 1025, device=DEV), 2)
