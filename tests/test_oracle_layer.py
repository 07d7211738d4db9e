"""Pins of the norm, router and expert oracle (oracle/layer.py): closed forms,
torch's autograd in float64 on the CPU, differences."""

import numpy as np
import pytest
import torch

from oracle import bf16, e4m3, layer
from tests.layer_util import expert_case, rows_bits


def test_norm_by_hand():
    # 3, 4 in a row of otherwise zeros: mean square 25 / 128
    x = np.zeros((1, 128))
    x[0, :2] = 3, 4
    h, rstd, y = layer.norm(bf16.from_f64_rne(x), None, np.full(128, 2.0), 2.0 ** -60)
    assert np.isclose(rstd[0], np.sqrt(128 / 25), rtol=1e-12)
    assert np.allclose(y[0, :3], [6 * np.sqrt(128) / 5, 8 * np.sqrt(128) / 5, 0], rtol=1e-12)
    s = layer.tile_scales(y)
    assert s.shape == (1, 1) and np.isclose(s[0, 0], 8 * np.sqrt(128) / 5 / 448)
    assert layer.tile_scales(np.zeros((2, 256))).tolist() == [[1, 1], [1, 1]]


def test_norm_rounds_the_sum_once():
    x, r = bf16.from_f64_rne(np.full((1, 128), 256.0)), bf16.from_f64_rne(np.full((1, 128), 1.0))
    h, _, _ = layer.norm(x, r, np.ones(128), 1e-6)
    assert (bf16.to_f32(h) == 256).all()               # 257 has no BF16 value; the tie goes to the even one


def test_norm_backward_is_the_norms_gradient():
    rng = np.random.default_rng(1)
    hb, dyb, dhb = rows_bits(rng, 5, 256), rows_bits(rng, 5, 256), rows_bits(rng, 5, 256)
    w = rng.standard_normal(256)
    h = torch.tensor(bf16.to_f32(hb), dtype=torch.float64, requires_grad=True)
    wt = torch.tensor(w, requires_grad=True)
    eps = float(np.float32(1e-5))
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * wt
    (y * torch.tensor(bf16.to_f32(dyb).astype(np.float64))).sum().backward()
    _, rstd, _ = layer.norm(hb, None, w, 1e-5)
    dx, dw = layer.norm_backward(dyb, hb, rstd, w, dhb)
    assert np.allclose(dx, h.grad.numpy() + bf16.to_f32(dhb), rtol=1e-10, atol=1e-10)
    assert np.allclose(dw, wt.grad.numpy(), rtol=1e-10, atol=1e-10)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_and_its_gradient(renorm):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((7, 12))
    ids, w = layer.route(x, 4, renorm)
    p = torch.softmax(torch.tensor(x), 1)
    top = torch.topk(p, 4, 1)
    assert np.array_equal(ids, top.indices.numpy())
    want = top.values / top.values.sum(1, keepdim=True) if renorm else top.values
    assert np.allclose(w, want.numpy(), rtol=1e-12)
    dw = rng.standard_normal((7, 4))
    got = layer.route_backward(x, ids, dw, renorm)
    step = 1e-6                                        # differences, the choice held fixed
    for t in range(7):
        for e in range(12):
            d = []
            for sign in (1, -1):
                z = x.copy()
                z[t, e] += sign * step
                q = np.exp(z[t])
                v = q[ids[t]]
                d.append(np.dot(v / (v if renorm else q).sum(), dw[t]))
            assert abs((d[0] - d[1]) / (2 * step) - got[t, e]) < 1e-8


def test_route_leaves_out_and_ties():
    inf, nan = np.inf, np.nan
    x = np.array([[1, 3, 3, -inf], [nan, -inf, 2, nan], [-inf, nan, -inf, -inf], [inf, 0, inf, 1]])
    ids, w = layer.route(x, 3, True)
    assert ids.tolist() == [[1, 2, 0], [2, -1, -1], [-1, -1, -1], [0, 2, 3]]
    assert w[1].tolist() == [1, 0, 0] and w[2].tolist() == [0, 0, 0] and w[3].tolist() == [0.5, 0.5, 0]
    assert np.isclose(w[0].sum(), 1) and w[0, 0] == w[0, 1]
    assert (layer.route_backward(x, ids, np.ones((4, 3)), False)[2] == 0).all()


def test_experts_by_rows():
    w = expert_case(5, 256, 128, 4, 2, seed=3, pad=1)
    out, size = layer.experts(**w)
    x = layer.dequantize_rows(w["x"], w["sx"])
    for t in range(5):
        want = np.zeros(256)
        for j in range(2):
            e = w["ids"][t, j]
            if e < 0:
                continue
            up = layer.dequantize_blocks(w["w13"][e], w["s13"][e]) @ x[t]
            act = up[:128] * torch.sigmoid(torch.tensor(up[:128])).numpy() * up[128:]
            want += float(w["weights"][t, j]) * (layer.dequantize_blocks(w["w2"][e], w["s2"][e]) @ act)
        assert np.allclose(out[t], want, rtol=1e-10, atol=1e-12)
        assert (size[t] >= np.abs(want) - 1e-12).all()
    assert (out[4] == 0).all()


def test_experts_twice_in_a_row():
    w = expert_case(2, 128, 128, 3, 3, seed=4, ids=[[1, 1, 2], [0, 0, 0]])
    out, _ = layer.experts(**w)
    w["weights"][:, 0] += w["weights"][:, 1]
    w["ids"][:, 1] = -1
    w["weights"][1, 0] += w["weights"][1, 2]
    w["ids"][1, 2] = 77
    again, _ = layer.experts(**w)
    assert np.allclose(out, again, rtol=1e-6)


def test_dequantization():
    q = e4m3.encode(np.float32([[1.5] * 128 + [-448] * 128]))
    assert layer.dequantize_rows(q, np.float32([[2], [0.5]])).tolist() == [[3.0] * 128 + [-224.0] * 128]
    b = layer.dequantize_blocks(np.repeat(q, 128, 0), np.float32([[2, 0.5]]))
    assert b.shape == (128, 256) and b[127, 0] == 3 and b[0, 255] == -224
