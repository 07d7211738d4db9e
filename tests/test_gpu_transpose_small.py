"""quantize_transpose_128x1 where the new scales are a few steps of 2^-149, bit for
bit: rounded down, they leave quotients past 464, which have to saturate."""

import numpy as np
import pytest

import fp8_block_scaled_04_amd as fb
from oracle import bf16, quantize
from tests.gpu_util import assert_codes_equal, bf16_dev, codes_dev, codes_host, f32_bits_host, f32_dev, require_gpu

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_gpu()


def check(q, s, pow2):
    qt, st = fb.quantize_transpose_128x1(codes_dev(q), f32_dev(s), pow2=pow2)
    qt_ref, st_ref = quantize.quantize_transpose_128x1(q, s, pow2=pow2)
    assert not (codes_host(qt) & 0x7F == 0x7F).any()
    assert_codes_equal(f32_bits_host(st), st_ref.view(np.uint32), "scales")
    assert_codes_equal(codes_host(qt), qt_ref, "codes")


@pytest.mark.parametrize("pow2", [False, True])
def test_transpose_requant_of_subnormal_scales(pow2):
    rng = np.random.default_rng(3)
    q = rng.integers(0, 256, (256, 1024), dtype=np.uint8)
    q[:, ::3] &= 0xBF                                   # columns of small codes only
    q[:, 1::3] &= 0x9F
    q[(q & 0x7F) == 0x7F] = 0x11
    s = (np.round(np.exp2(rng.uniform(0, 12, (8, 256)))) * 2.0 ** -149).astype(np.float32)
    s[0, :128], s[1, :128], s[2, :128] = 2.0 ** -149, 2.0 ** -148, 3 * 2.0 ** -149
    check(q, s, pow2)


@pytest.mark.parametrize("pow2", [False, True])
def test_transpose_requant_behind_the_norm(pow2):
    # rows of +-1 have rstd 1, so y = +-weight: tiles of up to 2^11 steps of 2^-149, their columns from one step on
    rng = np.random.default_rng(4)
    w = (np.round(np.exp2(rng.uniform(0, 11, 1024))) * 2.0 ** -149).astype(np.float32)
    x = rng.choice([-1.0, 1.0], (256, 1024))
    q, s, _, _ = fb.rms_norm_quantize(bf16_dev(bf16.from_f64_rne(x)), f32_dev(w), 2.0 ** -126, pow2=pow2)
    check(codes_host(q), s.cpu().numpy(), pow2)
