"""rms_norm_quantize where FP32 is short: tiles of subnormal y, whose scale is a few
steps of 2^-149, and products of h and weight that leave FP32's normal range."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_04_amd as fb
from oracle import bf16, quantize
from tests.gpu_util import bf16_dev, codes_host, f32_bits_host, f32_dev, require_gpu

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
