"""moe_experts against the float64 oracle.

Exact cases: small whole numbers for which every step of the kernels is exact
(gates of at least 64, where 1 / (1 + exp(-g)) is 1 in FP32), so any wrong row,
column, chunk, scale or expert shows as a difference.

General cases, error of an output: of the first product, per expert, the matrix
core's own truncation (gpu_util.py: 8 * 2^(E - 13) per group of eight products, E
the exponent of the largest) and FP32 additions, carried through the activation
(|silu'| <= 1.1, |silu(g)| <= |g|) and the second product; of the two-part
activations 2^-16 of a term; of FP32 sums 2^-24 per addition; 2^-8 for a BF16
output.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_04_amd as fb
from oracle import e4m3, layer
from tests.gpu_util import DEV, require_gpu
from tests.layer_util import EXPERT_ARGS, expert_case, expert_dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def setup_module(module):
    require_gpu()


def product_error(xq, sx, wq, sw):
    """(product, error bound) [T][N] of E4M3 rows and block-scaled weights."""
    x, w = e4m3.decode(xq), e4m3.decode(wq)
    T, K = x.shape
    value = layer.dequantize_rows(xq, sx) @ layer.dequantize_blocks(wq, sw).T
    err = np.zeros(value.shape)
    for t in range(T):
        top = np.abs(x[t] * w).reshape(-1, K // 8, 8).max(2)
        _, e = np.frexp(top)
        group = np.where(top > 0, 8 * np.exp2(e - 1.0 - 13), 0).reshape(-1, K // 128, 16).sum(2)
        sizes = np.abs(x[t] * w).reshape(-1, K // 128, 128).sum(2)
        scale = np.asarray(sx, np.float64)[:, t][None] * np.repeat(np.asarray(sw, np.float64), 128, 0)
        err[t] = ((group + sizes * U * (K // 128 + 12)) * scale).sum(1)
    return value, err


def bound(w, half):
    """Error bound of the whole layer [T][H] and its oracle."""
    out, size = layer.experts(**w)
    T, H = out.shape
    err = np.zeros((T, H))
    for e in range(w["w13"].shape[0]):
        tok = sorted({int(t) for t in np.argwhere(w["ids"] == e)[:, 0]})
        if not tok:
            continue
        up, d = product_error(w["x"][tok], w["sx"][:, tok], w["w13"][e], w["s13"][e])
        g, u = np.split(up, 2, axis=1)
        dg, du = np.split(d, 2, axis=1)
        share = np.array([np.abs(w["weights"][t][w["ids"][t] == e]).sum() for t in tok])[:, None]
        dact = share * (1.1 * dg * (np.abs(u) + du) + np.abs(g) * du + 12 * U * np.abs(g * u))
        err[tok] += dact @ np.abs(layer.dequantize_blocks(w["w2"][e], w["s2"][e])).T
    K = w["w2"].shape[2] * w["ids"].shape[1]
    return out, err + size * (2.0 ** -16 + U * (K // 128 + 24)) + half * np.abs(out) + 2.0 ** -130


@pytest.mark.parametrize("T,H,I,E,topk,pad", [(1, 128, 128, 1, 1, 0), (1, 1024, 256, 8, 2, 0), (3, 256, 384, 5, 3, 1),
                                              (16, 640, 128, 16, 4, 3), (17, 256, 256, 6, 2, 0), (40, 384, 128, 4, 3, 7),
                                              (64, 256, 256, 8, 4, 0), (128, 128, 128, 3, 2, 5), (2, 128, 128, 40, 16, 0)])
def test_experts(T, H, I, E, topk, pad):
    w = expert_case(T, H, I, E, topk, seed=T + H, pad=pad)
    dev = expert_dev(w)
    ref, tol = bound(w, U)
    got = fb.moe_experts(*dev, out_dtype=torch.float32)
    assert np.all(np.abs(got.cpu().numpy() - ref) <= tol)
    assert T == pad or float(np.sqrt(((got.cpu().numpy() - ref) ** 2).sum() / (ref ** 2).sum())) < 2.0 ** -10
    half = fb.moe_experts(*dev)
    assert torch.equal(half, got.to(torch.bfloat16))     # one rounding of the same sums
    assert (got[T - pad:] == 0).all()
    assert torch.equal(fb.moe_experts(*dev, out_dtype=torch.float32), got)


def exact_case(T, H, I, E, topk, seed, ids=None):
    """Whole numbers: x in {0, 1}, at least 64 ones in each row; gate weights 1;
    up weights in {-1, 0, 1}, nine of ten 0, so that no sum passes 24 bits; w2 in
    {-1, 0, 1}, more 0 where many terms are added; scales and weights powers of
    two.  At most 16 experts differ (in their codes; all do in their scales)."""
    rng = np.random.default_rng(seed)
    w = {}
    x = (rng.random((T, H)) < (0.55 if H <= 640 else 80 / H)).astype(np.float32)
    x[:, :64] = 1
    w["x"] = e4m3.encode(x)
    w["sx"] = np.ones((H // 128, T), np.float32)
    few = min(E, 16)
    w13 = np.ones((few, 2 * I, H), np.float32)
    w13[:, I:] = rng.choice([-1, 0, 1], (few, I, H), p=[0.05, 0.9, 0.05])
    w["w13"] = e4m3.encode(w13)[np.arange(E) % few]
    w["s13"] = np.exp2(rng.integers(0, 2, (E, 2 * I // 128, H // 128))).astype(np.float32)
    p = min(1 / 3, 500 / (I * topk) * (134 / float(x.sum(1).mean())) ** 1.5)
    w["w2"] = e4m3.encode(rng.choice([-1, 0, 1], (few, H, I), p=[p, 1 - 2 * p, p]).astype(np.float32))[np.arange(E) % few]
    w["s2"] = np.exp2(rng.integers(-1, 2, (E, H // 128, I // 128))).astype(np.float32)
    if ids is None:
        ids = np.stack([rng.permutation(E)[:topk] for _ in range(T)])
    w["ids"] = np.asarray(ids, np.int32)
    w["weights"] = np.exp2(rng.integers(-2, 1, (T, topk))).astype(np.float32)
    return {n: w[n] for n in EXPERT_ARGS}


def check_exact(w, **kw):
    ref, size = layer.experts(**w)
    # g, u: whole numbers below 2^24; activations g u times a power of two (below 2^16: two BF16 parts); sums below 2^24
    assert np.all(size * 8 < 2.0 ** 24)
    got = fb.moe_experts(*expert_dev(w), out_dtype=torch.float32, **kw)
    assert np.array_equal(got.cpu().numpy().astype(np.float64), ref)
    return got


@pytest.mark.parametrize("T,H,I,E,topk", [(1, 128, 128, 4, 2), (1, 256, 256, 2, 2), (2, 128, 384, 9, 3), (5, 384, 128, 3, 1),
                                          (15, 128, 128, 1, 1), (16, 128, 128, 2, 2), (17, 128, 128, 1, 1),
                                          (31, 256, 128, 2, 1), (33, 128, 128, 2, 2), (49, 128, 256, 3, 2),
                                          (64, 128, 128, 1, 1), (65, 128, 128, 1, 1), (100, 256, 128, 2, 1),
                                          (128, 128, 128, 2, 2), (128, 128, 128, 20, 16), (7, 640, 128, 64, 4),
                                          (128, 128, 128, 1024, 16), (128, 128, 128, 512, 16)])
def test_experts_exactly(T, H, I, E, topk):
    check_exact(exact_case(T, H, I, E, topk, seed=T * 3 + H))


# Every kernel, pinned: rows per pass, columns of the two products, waves that share the second's.
@pytest.mark.parametrize("tile,T,H,I,E,topk", [
    ((16, 8, 16, 4), 1, 128, 1152, 9, 2), ((16, 8, 32, 1), 17, 2048, 256, 9, 1), ((16, 8, 32, 4), 2, 1152, 384, 9, 3),
    ((16, 16, 32, 4), 40, 256, 1152, 40, 2), ((16, 16, 64, 4), 3, 2048, 384, 40, 4), ((16, 16, 64, 4), 50, 1024, 640, 40, 6),
    ((16, 16, 64, 1), 4, 2176, 640, 30, 6), ((16, 16, 64, 1), 60, 4096, 128, 100, 2),
    # all experts at once: fewer chunks than waves, as many, more; one token, 16; a row for every expert, one expert for all
    ((16, 8, 16, 8), 1, 128, 128, 1, 1), ((16, 8, 16, 8), 3, 2048, 256, 9, 1), ((16, 8, 16, 8), 16, 128, 128, 16, 16),
    ((16, 8, 16, 8), 16, 256, 2048, 1, 1), ((16, 16, 16, 8), 2, 2048, 128, 64, 14), ((16, 16, 16, 8), 16, 2304, 1024, 4, 2),
    ((16, 8, 16, 8), 13, 4224, 640, 3, 2), ((16, 8, 16, 8), 15, 3968, 256, 12, 5),
    # many rows: halves of units alone; whole units of the first product, of the second (its last one half empty); up to
    # 16, 32 and 64 rows each, and more
    ((64, 128, 256, 4), 64, 256, 384, 24, 8), ((64, 128, 256, 4), 64, 128, 1024, 64, 8),
    ((64, 128, 256, 4), 64, 1920, 128, 64, 8), ((64, 128, 256, 4), 128, 128, 1024, 64, 16),
    ((64, 128, 256, 4), 128, 1920, 128, 64, 16), ((64, 128, 256, 4), 128, 384, 640, 16, 8),
    ((64, 128, 256, 4), 128, 640, 1024, 16, 16), ((64, 128, 256, 4), 128, 4096, 512, 2, 2)])
def test_experts_exactly_on_every_kernel(tile, T, H, I, E, topk):
    assert fb.moe_experts_tile(T, H, I, E, topk) == tile
    check_exact(exact_case(T, H, I, E, topk, seed=T + H + I))


# One place per token, a fifth of them outside: no sum over places is left.  On every kernel of the second product.
@pytest.mark.parametrize("tile,T,H,I,E", [
    ((16, 8, 16, 8), 16, 128, 128, 3), ((16, 16, 16, 4), 16, 128, 2304, 3), ((16, 8, 32, 1), 17, 2048, 256, 9),
    ((16, 16, 32, 4), 40, 256, 1152, 40), ((16, 16, 64, 4), 50, 1024, 640, 40), ((16, 16, 64, 1), 60, 4096, 128, 100),
    ((64, 128, 256, 4), 128, 384, 1024, 8), ((64, 128, 256, 4), 128, 4096, 512, 2)])
def test_experts_of_one_place(tile, T, H, I, E):
    assert fb.moe_experts_tile(T, H, I, E, 1) == tile
    rng = np.random.default_rng(T + E)
    ids = np.where(rng.random((T, 1)) < 0.2, rng.choice([-1, E, -(1 << 31), 1 << 30], (T, 1)), rng.integers(0, E, (T, 1)))
    ids[-1] = -1
    w = exact_case(T, H, I, E, 1, seed=T + H + I, ids=ids)
    more = torch.full((T + 1, H), float("nan"), device=DEV)
    check_exact(w, out=more[:T])
    assert more[T].isnan().all()
    half = torch.full((T + 1, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    fb.moe_experts(*expert_dev(w), out=half[:T])
    assert torch.equal(half[:T], more[:T].to(torch.bfloat16)) and half[T].isnan().all()
    w["ids"][:] = E
    assert (fb.moe_experts(*expert_dev(w), out=half[:T]) == 0).all()


@pytest.mark.parametrize("T,H,I,E,topk", [(5, 256, 384, 4, 1), (16, 256, 384, 16, 1), (40, 256, 384, 4, 1), (64, 256, 640, 16, 2)])
@pytest.mark.parametrize("where", ["w2", "s2", "w13"])
def test_experts_of_others_do_not_matter(T, H, I, E, topk, where):
    # NaN codes or scales of an expert reach its own tokens and no others
    w = exact_case(T, H, I, E, topk, seed=T + E)
    clean = fb.moe_experts(*expert_dev(w), out_dtype=torch.float32)
    bad = int(w["ids"][T // 2][0])
    mine = torch.from_numpy((w["ids"] == bad).any(1)).to(DEV)
    w[where] = w[where].copy()
    w[where][bad] = np.float32(np.nan) if where == "s2" else 0x7F
    got = fb.moe_experts(*expert_dev(w), out_dtype=torch.float32)
    assert got[mine].isnan().all() and torch.equal(got[~mine], clean[~mine])


@pytest.mark.parametrize("T,H,I,E,topk", [(64, 256, 512, 20, 8), (128, 128, 1024, 24, 3), (100, 256, 640, 16, 10)])
def test_experts_with_many_rows(T, H, I, E, topk):
    assert fb.moe_experts_tile(T, H, I, E, topk)[0] == 64
    w = expert_case(T, H, I, E, topk, seed=T, pad=3)
    ref, tol = bound(w, U)
    got = fb.moe_experts(*expert_dev(w), out_dtype=torch.float32)
    assert np.all(np.abs(got.cpu().numpy() - ref) <= tol)
    assert float(np.sqrt(((got.cpu().numpy() - ref) ** 2).sum() / (ref ** 2).sum())) < 2.0 ** -10


@pytest.mark.parametrize("places", [2, 40])
def test_experts_that_stand_twice_or_outside(places):
    # (more places than experts, and fewer: the two ways the experts with work are found)
    E = 6 if places == 40 else 90
    ids = np.random.default_rng(8).integers(-2, E + 2, (max(2, places // 4), 4))
    ids[0] = [3, 3, 5, 3]
    ids[1] = [-1, E, 1 << 30, -(1 << 31)]
    w = exact_case(ids.shape[0], 128, 128, E, 4, seed=5, ids=ids)
    got = check_exact(w)
    assert (got[1] == 0).all()


def test_experts_more_places_than_experts():
    ids = np.random.default_rng(3).integers(0, 2, (20, 16))
    check_exact(exact_case(20, 128, 128, 2, 16, seed=2, ids=ids))


def test_experts_all_tokens_one_expert():
    ids = np.full((128, 1), 6)
    check_exact(exact_case(128, 128, 128, 7, 1, seed=6, ids=ids))


def test_experts_without_any():
    w = exact_case(3, 128, 128, 4, 2, seed=7, ids=np.full((3, 2), -1))
    assert (check_exact(w) == 0).all()
    dev = expert_dev(w)
    none = [dev[0][:0], dev[1][:, :0].contiguous(), dev[2][:0], dev[3][:0]] + dev[4:]
    assert fb.moe_experts(*none).shape == (0, 128)


def test_experts_workspace_contents_do_not_matter():
    w = exact_case(9, 256, 128, 5, 3, seed=9)
    n = fb.moe_experts_workspace_bytes(9, 256, 128, 5, 3)
    want = check_exact(w)
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((n + 64,), fill, dtype=torch.uint8, device=DEV)
        out = torch.full((9, 256), float("nan"), device=DEV)
        assert torch.equal(check_exact(w, workspace=ws[:n], out=out), want)
        assert (ws[n:] == fill).all()


def test_experts_gates_of_either_sign():
    # silu far from 0: -0 for gates of -500, the gate itself for +500; u = 1
    x = torch.ones(1, 128, device=DEV).to(torch.float8_e4m3fn)
    w13 = torch.zeros(1, 256, 128, device=DEV)
    w13[0, :64, :100] = 5.0
    w13[0, 64:128, :100] = -5.0
    w13[0, 128:, 0] = 1.0
    w2 = torch.eye(128, device=DEV)[None].to(torch.float8_e4m3fn)
    one = torch.ones(1, 1, device=DEV)
    got = fb.moe_experts(x, one, torch.zeros(1, 1, dtype=torch.int32, device=DEV), one, w13.to(torch.float8_e4m3fn),
                         torch.ones(1, 2, 1, device=DEV), w2, torch.ones(1, 1, 1, device=DEV), out_dtype=torch.float32)
    assert (got[0, :64] == 500).all() and (got[0, 64:] == 0).all()


def test_experts_refuse():
    w = expert_dev(exact_case(3, 256, 128, 4, 2, seed=1))
    x, sx, ids, wt, w13, s13, w2, s2 = w

    def put(i, t):
        return w[:i] + [t] + w[i + 1:]
    for args in (put(0, x[:, :128].contiguous()), put(1, sx[:, :2].contiguous()), put(2, ids[:2]), put(3, wt[:, :1].contiguous()),
                 put(4, w13[:, :200].contiguous()), put(5, s13[:, :1].contiguous()), put(6, w2[:3]),
                 put(7, s2[:, :1].contiguous()), put(2, ids.t().contiguous().t())):
        with pytest.raises(ValueError):
            fb.moe_experts(*args)
    for args in (put(0, x.float()), put(2, ids.long()), put(4, w13.float())):
        with pytest.raises(TypeError):
            fb.moe_experts(*args)
    with pytest.raises(TypeError):
        fb.moe_experts(*w, out_dtype=torch.float16)
    with pytest.raises(fb.Fp8bsError):
        fb.moe_experts(*w, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    many = [t.expand(130, *t.shape[1:]).contiguous() if i in (0, 2, 3) else t
            for i, t in enumerate([x[:1], torch.ones(2, 130, device=DEV), ids[:1], wt[:1]] + w[4:])]
    with pytest.raises(fb.Fp8bsError):
        fb.moe_experts(*many)
