"""rms_norm_quantize and rms_norm_backward against the float64 oracle.

u = 2^-24 is half a step of FP32, 2^-8 of BF16, 2^-4 of E4M3 (relative).  A sum
over a row of K values passes at most 16 values in one lane, 6 steps in a wave
and 16 waves: 38 roundings, halved by the square root, and 4 more up to rstd:
23 u.  y takes two products more, a scale three roundings: 28 u covers both.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_04_amd as fb
from oracle import bf16, layer, quantize
from tests.gpu_util import DEV, bf16_dev, codes_host, f32_bits_host, f32_dev, require_gpu
from tests.layer_util import rows_bits, weight_of

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def setup_module(module):
    require_gpu()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def check(x, r, w, wdev, eps, **kw):
    """One call against the oracle; -> its outputs."""
    got = fb.rms_norm_quantize(bf16_dev(x), wdev, eps, residual=None if r is None else bf16_dev(r), return_y=True, **kw)
    q, s, h, rstd, y = got
    h_ref, rstd_ref, y_ref = layer.norm(x, r, w, eps)
    assert np.array_equal(bits(h), h_ref)
    assert np.all(np.abs(rstd.cpu().numpy() - rstd_ref) <= 24 * U * rstd_ref)
    err = np.abs(y.float().cpu().numpy().astype(np.float64) - y_ref)
    assert np.all(err <= (2.0 ** -8 + 30 * U) * np.abs(y_ref) + 2.0 ** -134)
    want, s = layer.tile_scales(y_ref), s.cpu().numpy().astype(np.float64)
    if kw.get("pow2"):
        assert np.all(np.frexp(s)[0] == 0.5)
        assert np.all(s >= want * (1 - 28 * U)) and np.all(s <= 2 * want * (1 + 28 * U))
    else:
        assert np.all(np.abs(s - want) <= 28 * U * want + 2.0 ** -149)
    back = layer.dequantize_rows(codes_host(q), s)
    step = np.repeat(s.T, 128, 1) * 2.0 ** -10
    assert np.all(np.abs(back - y_ref) <= (2.0 ** -4 + 60 * U) * np.abs(y_ref) + step * 1.0001)
    return got


@pytest.mark.parametrize("m,k", [(1, 128), (1, 7168), (3, 256), (17, 1536), (5, 2048), (6, 2176), (33, 4224), (9, 8320),
                                 (4, 16384), (130, 896)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_norm(m, k, residual, kind):
    rng = np.random.default_rng(m * 7 + k)
    w, raw = weight_of(rng, k, kind)
    check(rows_bits(rng, m, k), rows_bits(rng, m, k, 3.0) if residual else None, w,
          f32_dev(raw) if kind == "fp32" else bf16_dev(raw), 1e-6)


@pytest.mark.parametrize("m,k", [(2, 128), (7, 7168)])
def test_norm_power_of_two_scales(m, k):
    rng = np.random.default_rng(k)
    w, raw = weight_of(rng, k, "fp32")
    check(rows_bits(rng, m, k), rows_bits(rng, m, k), w, f32_dev(raw), 1e-6, pow2=True)


def test_norm_of_rows_of_ones_is_the_quantizer():
    # mean square 1 and an eps that 1 absorbs: rstd = 1, y = +-weight, so codes and scales are bit for bit those
    # of the quantizer
    rng = np.random.default_rng(5)
    sign = np.where(rng.random((40, 1024)) < 0.5, -1.0, 1.0)
    w, raw = weight_of(rng, 1024, "bf16")
    w[256:384] = raw[256:384] = 0                      # one tile of zeros: scale 1
    for pow2 in (False, True):
        q, s, _, rstd, y = fb.rms_norm_quantize(bf16_dev(bf16.from_f64_rne(sign)), bf16_dev(raw), 2.0 ** -100, pow2=pow2,
                                                return_y=True)
        y_bits = bf16.from_f64_rne(sign * w)
        q_ref, s_ref = quantize.quantize_1x128(y_bits, pow2=pow2)
        assert np.array_equal(codes_host(q), q_ref) and np.array_equal(f32_bits_host(s), s_ref.view(np.uint32))
        assert (rstd == 1).all() and np.array_equal(bits(y), y_bits)


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e15])
def test_norm_of_extreme_rows(size):
    # (1e-30: the mean square underflows and eps alone counts; y is around 1e-27)
    rng = np.random.default_rng(11)
    w, raw = weight_of(rng, 512, "fp32")
    x = bf16.from_f64_rne(rng.standard_normal((3, 512)) * size)
    check(x, None, w, f32_dev(raw), 1e-6)


def test_norm_of_zeros():
    x = torch.zeros(3, 256, dtype=torch.bfloat16, device=DEV)
    q, s, h, rstd = fb.rms_norm_quantize(x, torch.ones(256, device=DEV), 1e-4, residual=x)
    assert (codes_host(q) & 0x7F == 0).all() and (s == 1).all() and (h == 0).all()
    assert np.allclose(rstd.cpu().numpy(), 100, rtol=24 * U)
    q, s, h, rstd = fb.rms_norm_quantize(x[:0], torch.ones(256, device=DEV))
    assert q.shape == (0, 256) and s.shape == (2, 0) and rstd.shape == (0,)


@pytest.mark.parametrize("where", ["x", "residual"])
def test_norm_in_place(where):
    rng = np.random.default_rng(3)
    x, r = rows_bits(rng, 19, 1152), rows_bits(rng, 19, 1152)
    w, raw = weight_of(rng, 1152, "bf16")
    want = fb.rms_norm_quantize(bf16_dev(x), bf16_dev(raw), residual=bf16_dev(r))
    a, b = bf16_dev(x), bf16_dev(r)
    to = a if where == "x" else b
    got = fb.rms_norm_quantize(a, bf16_dev(raw), residual=b, h=to)
    assert got[2] is to
    for p, q in zip(want, got):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_norm_of_more_rows_than_workgroups():
    m = (1 << 20) + 5
    x = torch.randn(m, 128, device=DEV, dtype=torch.bfloat16)
    w = torch.ones(128, device=DEV)
    q, s, _, rstd = fb.rms_norm_quantize(x, w)
    pick = [0, 1, 7, (1 << 20) - 1, 1 << 20, m - 1]
    q1, s1, _, rstd1 = fb.rms_norm_quantize(x[pick].contiguous(), w)
    assert torch.equal(q[pick].view(torch.uint8), q1.view(torch.uint8))
    assert torch.equal(s[:, pick], s1) and torch.equal(rstd[pick], rstd1)


def back_bound(dy, h, rstd, w, dh):
    """Error bounds of dx and dweight: roundings times the sizes of what is added."""
    dy, h = bf16.to_f32(dy).astype(np.float64), bf16.to_f32(h).astype(np.float64)
    n, g, inv = np.abs(h * rstd[:, None]), np.abs(dy * w), np.abs(rstd)[:, None]
    extra = 0 if dh is None else np.abs(bf16.to_f32(dh).astype(np.float64))
    return 48 * U * (inv * (g + n * (n * g).mean(1, keepdims=True)) + extra), np.abs(dy * n).sum(0) * U


@pytest.mark.parametrize("m,k", [(1, 128), (1, 7168), (3, 256), (17, 1536), (513, 2048), (6, 2176), (1100, 384), (2, 16384)])
@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_norm_backward(m, k, with_dh, kind):
    rng = np.random.default_rng(m + k)
    w, raw = weight_of(rng, k, kind)
    wdev = f32_dev(raw) if kind == "fp32" else bf16_dev(raw)
    h, dy = rows_bits(rng, m, k), rows_bits(rng, m, k, 1e-3)
    dh = rows_bits(rng, m, k, 1e-3) if with_dh else None
    rstd = layer.norm(h, None, w, 1e-6)[1].astype(np.float32)
    args = (bf16_dev(dy), bf16_dev(h), f32_dev(rstd), wdev)
    dhd = bf16_dev(dh) if with_dh else None
    dx, dw = fb.rms_norm_backward(*args, dh=dhd)
    dx_ref, dw_ref = layer.norm_backward(dy, h, rstd, w, dh)
    bx, bw = back_bound(dy, h, rstd.astype(np.float64), w, dh)
    assert np.all(np.abs(dx.float().cpu().numpy() - dx_ref) <= 2.0 ** -8 * np.abs(dx_ref) + bx * 1.01 + 2.0 ** -134)
    # rows of one group in turn, then 16 runs of groups, then the runs; three roundings of a term
    groups = fb.rms_norm_backward_workspace_bytes(m, k) // (4 * k)
    chain = -(-m // groups) + -(-groups // 16) + 16 + 3
    assert np.all(np.abs(dw.cpu().numpy() - dw_ref) <= chain * bw * 1.01)
    again = fb.rms_norm_backward(*args, dh=dhd)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    # accumulated, and in place of dy
    acc = torch.full((k,), 0.25, device=DEV)
    dx2, dw2 = fb.rms_norm_backward(args[0], args[1], args[2], wdev, dh=dhd, dx=args[0], dweight=acc, accumulate=True)
    assert dx2 is args[0] and torch.equal(dx2, dx)
    assert dw2 is acc and torch.equal(acc, dw + 0.25)
    if with_dh:
        assert torch.equal(fb.rms_norm_backward(bf16_dev(dy), args[1], args[2], wdev, dh=dhd, dx=dhd)[0], dx)


@pytest.mark.parametrize("m,k", [(1023, 2048), (1025, 2048), (2053, 1024), (4095, 512), (4097, 512), (4103, 640), (9001, 128)])
def test_norm_backward_of_many_narrow_rows(m, k):
    # several rows of a workgroup at once, the last run of rows cut short.  A row's gradient depends on nothing else:
    # bit for bit that of the same row in a call of a few.  dweight within the roundings of test_norm_backward (a lane's
    # rows, then the lanes' sums, are no longer chain than the group's rows)
    rng = np.random.default_rng(m * 3 + k)
    w, raw = weight_of(rng, k, "bf16")
    h, dy, dh = rows_bits(rng, m, k), rows_bits(rng, m, k, 1e-3), rows_bits(rng, m, k, 1e-3)
    rstd = layer.norm(h, None, w, 1e-6)[1].astype(np.float32)
    out = torch.full((m + 2, k), -7.0, dtype=torch.bfloat16, device=DEV)
    dx, dw = fb.rms_norm_backward(bf16_dev(dy), bf16_dev(h), f32_dev(rstd), bf16_dev(raw), dh=bf16_dev(dh), dx=out[:m])
    assert (out[m:] == -7).all()
    dx_ref, dw_ref = layer.norm_backward(dy, h, rstd, w, dh)
    bx, bw = back_bound(dy, h, rstd.astype(np.float64), w, dh)
    assert np.all(np.abs(dx.float().cpu().numpy() - dx_ref) <= 2.0 ** -8 * np.abs(dx_ref) + bx * 1.01 + 2.0 ** -134)
    groups = fb.rms_norm_backward_workspace_bytes(m, k) // (4 * k)
    chain = -(-m // groups) + -(-groups // 16) + 16 + 3
    assert np.all(np.abs(dw.cpu().numpy() - dw_ref) <= chain * bw * 1.01)
    few = slice(m - 37, m)
    assert torch.equal(fb.rms_norm_backward(bf16_dev(dy[few]), bf16_dev(h[few]), f32_dev(rstd[few]), bf16_dev(raw),
                                            dh=bf16_dev(dh[few]))[0], dx[m - 37:])


def test_norm_backward_of_no_rows():
    e = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, device=DEV)
    acc = torch.full((256,), 3.0, device=DEV)
    dx, dw = fb.rms_norm_backward(e, e, w[:0], w)
    assert dx.shape == (0, 256) and (dw == 0).all()
    fb.rms_norm_backward(e, e, w[:0], w, dweight=acc, accumulate=True)
    assert (acc == 3).all()


def test_norm_backward_against_differences():
    # of L = sum dy y(h), float64 differences of the oracle's norm
    rng = np.random.default_rng(9)
    h, dy = bf16.from_f64_rne(rng.standard_normal((2, 256))), bf16.from_f64_rne(rng.standard_normal((2, 256)))
    w, raw = weight_of(rng, 256, "fp32")
    rstd = layer.norm(h, None, w, 1e-5)[1].astype(np.float32)
    dx, dw = fb.rms_norm_backward(bf16_dev(dy), bf16_dev(h), f32_dev(rstd), f32_dev(raw))
    hv, dv = bf16.to_f32(h).astype(np.float64), bf16.to_f32(dy).astype(np.float64)

    def loss(a, b):
        return (a / np.sqrt((a * a).mean(1, keepdims=True) + 1e-5) * b * dv).sum()
    for k in (0, 1, 100, 255):
        for m in (0, 1):
            d = np.zeros((2, 256))
            d[m, k] = 1e-5
            want = (loss(hv + d, w) - loss(hv - d, w)) / 2e-5
            assert abs(float(dx[m, k]) - want) <= 2.0 ** -8 * abs(want) + 1e-6
        d = np.zeros(256)
        d[k] = 1e-5
        want = (loss(hv, w + d) - loss(hv, w - d)) / 2e-5
        assert abs(float(dw[k]) - want) <= 1e-5 * max(1, abs(want))


def test_norm_refuses():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, device=DEV)
    for call in (lambda: fb.rms_norm_quantize(x[:, ::2], w[:128]), lambda: fb.rms_norm_quantize(x, w[:128]),
                 lambda: fb.rms_norm_quantize(x, w, residual=x[:2]), lambda: fb.rms_norm_quantize(x, w, h=x),
                 lambda: fb.rms_norm_backward(x, x, w[:3], w), lambda: fb.rms_norm_backward(x[:2], x, w[:4], w),
                 lambda: fb.rms_norm_backward(x, x, w[:4], w, accumulate=True),
                 lambda: fb.rms_norm_backward(x, x, w[:4], w, workspace=torch.zeros(8, device=DEV))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fb.rms_norm_quantize(x.float(), w), lambda: fb.rms_norm_quantize(x, w.double())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: fb.rms_norm_quantize(x[:, :192].contiguous(), w[:192]), lambda: fb.rms_norm_quantize(x, w, 0.0),
                 lambda: fb.rms_norm_backward(x, x, w[:4], w, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(fb.Fp8bsError):
            call()
