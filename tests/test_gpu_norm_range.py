"""rms_norm_quantize where FP32 is short: tiles of subnormal y, whose scale is a few
steps of 2^-149, and products of h and weight that leave FP32's normal range."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_04_amd as fb
from oracle import bf16, quantize
from tests.gpu_util import bf16_dev, codes_host, f32_bits_host, f32_dev, require_gpu
from tests.layer_util import rows_bits, weight_of
from tests.test_gpu_norm import check

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_gpu()


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("k", [2048, 16384])
def test_norm_of_subnormal_tiles_is_the_quantizer(k, pow2):
    # Rows of +-1: the mean square is 1, eps is absorbed, rstd = 1 and y = +-weight, so codes and scales are bit for bit
    # those of the rule.  One tile per amax, from one step of 2^-149 up to normal numbers: a scale rounded down to n
    # steps leaves quotients up to 448 (1 + 1 / (2 n)), which saturate.
    rng = np.random.default_rng(k)
    steps = np.unique(np.round(np.exp2(np.linspace(0, 23.5, k // 128))).astype(np.int64))
    known = np.array([500, 671, 672, 1120, 3808, 6496])       # (past 464, or next to it, with one or both kinds of scales)
    steps = np.concatenate([known, rng.permutation(steps)])[:k // 128]
    steps = np.concatenate([steps, rng.integers(1, 9000, k // 128 - steps.size)])
    n = np.floor(rng.random((k // 128, 128)) * (steps[:, None] + 1)).astype(np.int64)
    n[np.arange(k // 128), rng.integers(0, 128, k // 128)] = steps
    w = (n * 2.0 ** -149).astype(np.float32).reshape(k)
    sign = np.where(rng.random((9, k)) < 0.5, -1.0, 1.0)
    q, s, _, rstd = fb.rms_norm_quantize(bf16_dev(bf16.from_f64_rne(sign)), f32_dev(w), 2.0 ** -126, pow2=pow2)
    assert (rstd == 1).all()
    got = codes_host(q)
    assert not (got & 0x7F == 0x7F).any()
    q_ref, s_ref = quantize.quantize_rows_f32(sign.astype(np.float32) * w, pow2)
    assert np.array_equal(f32_bits_host(s), s_ref.view(np.uint32)) and np.array_equal(got, q_ref)


@pytest.mark.parametrize("pow2", [False, True])
def test_norm_of_a_small_tile_among_ones(pow2):
    # BF16 weights: 31 tiles of 1 and one of 2^-130, there with weights of 2^-10.  y = (h weight) rstd, rounded once
    x = np.ones((3, 4096))
    x[:, 640:768] = 2.0 ** -130
    w = np.ones(4096)
    w[640:768] = 2.0 ** -10
    q, s, _, rstd = fb.rms_norm_quantize(bf16_dev(bf16.from_f64_rne(x)), bf16_dev(bf16.from_f64_rne(w)), pow2=pow2)
    y = (x * w * rstd.cpu().numpy().astype(np.float64)[:, None]).astype(np.float32)
    q_ref, s_ref = quantize.quantize_rows_f32(y, pow2)
    assert np.array_equal(f32_bits_host(s), s_ref.view(np.uint32)) and np.array_equal(codes_host(q), q_ref)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("h,weight", [(-80, -80), (-70, -64), (34, 100), (55, 73), (-100, 40), (-100, -24), (0, 0)])
def test_norm_of_products_past_the_normal_range(h, weight, kind):
    # h weight below 2^-126 or past 2^128 (below 2^144) where y is neither: the bounds of test_gpu_norm.py hold as
    # anywhere
    rng = np.random.default_rng(200 + h)
    w, raw = weight_of(rng, 768, kind)
    w = w * 2.0 ** weight
    dev = f32_dev(w) if kind == "fp32" else bf16_dev(bf16.from_f64_rne(w))
    check(rows_bits(rng, 7, 768, 2.0 ** h), None, w, dev, 2.0 ** -126)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_norm_of_rows_with_both_ends(kind):
    # one row: large h with ordinary weights, tiny h with very large ones, zeros of either
    rng = np.random.default_rng(77)
    w, raw = weight_of(rng, 1024, kind)
    size = np.exp2(np.repeat([0, 100, 110, -100, -10, 0, 80, 0], 128).astype(np.float64))
    x = rng.standard_normal((5, 1024)) * np.exp2(np.repeat([55, -100, -118, 50, -40, 0, 55, 55], 128).astype(np.float64))
    x[:, 640:704] = 0
    w = w * size
    w[700:768] = 0
    dev = f32_dev(w) if kind == "fp32" else bf16_dev(bf16.from_f64_rne(w))
    check(bf16.from_f64_rne(x), None, w, dev, 1e-6)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_norm_of_rows_out_of_range_leaves_the_others(kind):
    # NaN, infinities and sums of squares past 2^128 in rows of their own; the sum of squares gives rstd 0 and codes of 0
    rng = np.random.default_rng(21)
    w, raw = weight_of(rng, 1152, kind)
    dev = f32_dev(raw) if kind == "fp32" else bf16_dev(raw)
    x = rng.standard_normal((40, 1152))
    clean = fb.rms_norm_quantize(bf16_dev(bf16.from_f64_rne(x)), dev, return_y=True)
    bad = x.copy()
    bad[3, 700] = np.nan
    bad[17, 0], bad[18, 1151] = np.inf, -np.inf
    bad[30] = 2.0 ** 70
    got = fb.rms_norm_quantize(bf16_dev(bf16.from_f64_rne(bad)), dev, return_y=True)
    rest = [m for m in range(40) if m not in (3, 17, 18, 30)]
    for a, b in zip(clean, got):
        pick = (lambda t: t[:, rest]) if a.shape == (9, 40) else (lambda t: t[rest])
        assert torch.equal(pick(a.view(torch.uint8) if a.element_size() == 1 else a), pick(b.view(torch.uint8) if b.element_size() == 1 else b))
    assert got[3][30] == 0 and (codes_host(got[0])[30] & 0x7F == 0).all() and (got[4][30] == 0).all()
    assert got[3][3].isnan() and got[4][3].isnan().all()
