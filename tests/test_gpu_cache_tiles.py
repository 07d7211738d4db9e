"""The cache's attention on every row tile, and its weights and eviction, where
the paths of the kernels differ: scores in the hundreds, negative scales, strided
queries, absent pages, small pages.  Every attention case is pinned to the tile it
is meant for.  Tolerances are those of tests/test_gpu_cache.py.
"""

import numpy as np
import pytest
import torch

from fp8_block_scaled_04_amd import fp8bs
from oracle import bf16, cache as oracle
from tests import cache_util
from tests.gpu_util import f32_bits_host, f32_dev, i32_dev, out_host_f64, require_gpu
from tests.test_gpu_cache import LENS, SHAPES, cache_dev, check_attention, same_cache, score_error

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_gpu()


# name: tile, D, heads, group, P, cached tokens, rows, max_new, max_kv; a bound of
# 2^20 cached tokens sends few pairs to the larger tiles, in splits
BOUND = 1 << 20
FORMS = {
    "16 rows": (16, 128, 2, 4, 16, [300, 90, 200], [2, 7, 1], 7, 300),
    "16 rows, D = 64": (16, 64, 2, 4, 16, [300, 90, 200], [2, 7, 1], 7, 300),
    "128 rows": (128, 128, 2, 4, 16, [300, 90, 200], [2, 30, 20], 30, BOUND),
    "128 rows, one split": (128, 128, 4, 16, 32, [250, 90, 200] * 16, [2, 7, 5] * 16, 7, 256),
    "128 rows, D = 64": (128, 64, 2, 4, 16, [300, 90, 200], [2, 30, 20], 30, BOUND),
    "128 rows, D = 64, one split": (128, 64, 2, 40, 64, [256, 190], [240, 190], 250, 256),
    "256 rows": (256, 128, 2, 8, 16, [300, 90, 200], [2, 80, 20], 80, BOUND),
    "256 rows, one split": (256, 128, 8, 4, 64, [300, 190] * 16, [100, 160] * 16, 160, 300),
}


def case(name, seed=0):
    tile, D, H, G, P, kv, new, max_new, max_kv = FORMS[name]
    w = cache_util.make(kv, new, H, G, D, P, seed=seed)
    return w, tile, D, G, max_new, max_kv


def attend(w, d, q, tile, max_new, max_kv, scale, **kw):
    cache = cache_dev(d)
    assert fp8bs.cache_attention_tile(cache, d["table"], q.shape[1], q.shape[0], max_new, max_kv) == tile
    out, lse = fp8bs.cache_attention(q, cache, d["table"], d["q_offsets"], d["kv_lens"], max_new, max_kv, scale,
                                     return_lse=True, **kw)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("name", FORMS)
def test_large_scores_negative_scales_and_strided_queries(name):
    w, tile, D, G, max_new, max_kv = case(name, seed=9)
    w["q"] = cache_util.bits(bf16.to_f32(w["q"]).astype(np.float64) * 12)
    d = cache_util.dev(w)
    joint = torch.cat([d["q"], torch.zeros_like(d["q"])], dim=1).contiguous()
    for scale, cap in ((0.4, 0.0), (-0.4, 0.0), (-0.4, 20.0)):
        print(f"{name} scale={scale} cap={cap}", flush=True)
        out, lse = attend(w, d, joint[:, :d["q"].shape[1]], tile, max_new, max_kv, scale, softcap=cap)
        check_attention(w, out, lse, scale, cap, False, f"{name} scale={scale} cap={cap}")


@pytest.mark.parametrize("name", FORMS)
def test_scores_that_grow_along_the_cache(name):
    # every later page outweighs all before it: the running maximum moves at each step
    w, tile, D, G, max_new, max_kv = case(name, seed=10)
    w["q"] = cache_util.bits(np.abs(bf16.to_f32(w["q"]).astype(np.float64)) + 0.5)
    w["k"] = np.where(w["k"] == 0x7F, w["k"], w["k"] & 0x7F)
    for b in range(len(w["kv_lens"])):
        n = -(-int(w["kv_lens"][b]) // w["P"])
        for j in range(n):
            w["ks"][w["table"][b, j]] *= np.float32((j + 1) / n)
    d = cache_util.dev(w)
    for scale in (0.05, -0.05):
        print(f"{name} growing scores scale={scale}", flush=True)
        out, lse = attend(w, d, d["q"], tile, max_new, max_kv, scale)
        check_attention(w, out, lse, scale, 0.0, False, f"{name} growing scores")


def absent(w):
    """Table entries outside the pool: single pages, the first ones, a whole sequence."""
    table = w["table"]
    table[0, 1] = -1
    table[1, :] = 1 << 20
    table[2 % len(table), 2:4] = -(1 << 31)
    table[-1, 0] = w["k"].shape[0]


@pytest.mark.parametrize("name", FORMS)
def test_absent_pages(name):
    w, tile, D, G, max_new, max_kv = case(name, seed=11)
    absent(w)
    d = cache_util.dev(w)
    for cap, full in ((0.0, False), (5.0, True)):
        print(f"{name} absent pages cap={cap}", flush=True)
        out, lse = attend(w, d, d["q"], tile, max_new, max_kv, 0.1, softcap=cap, full=full)
        check_attention(w, out, lse, 0.1, cap, full, f"{name} absent pages")
    lo, hi = w["q_offsets"][1:3]
    assert torch.isneginf(lse[lo:hi]).all() and (out[lo:hi] == 0).all()


@pytest.mark.parametrize("lens", ["ragged", "overrun", "prompt", "empty"])
@pytest.mark.parametrize("H,G,D,P", SHAPES)
def test_shapes_on_larger_tiles(lens, H, G, D, P):
    kv, new = LENS[lens]
    w = cache_util.make(kv, new, H, G, D, P, seed=H + G + D + 2)
    d = cache_util.dev(w)
    for rows in (65, 129):
        max_new = max(-(-rows // G), w["max_new"])
        tile = 256 if D == 128 and max_new * G > 128 else 128
        for cap, full in ((0.0, False), (3.0, True)):
            print(f"tile {tile} {lens} H={H} G={G} D={D} P={P} cap={cap}", flush=True)
            out, lse = attend(w, d, d["q"], tile, max_new, BOUND * 16, D ** -0.5, softcap=cap, full=full)
            check_attention(w, out, lse, D ** -0.5, cap, full, f"tile {tile} {lens} H={H} G={G} D={D} P={P}")


@pytest.mark.parametrize("D,H,G,P,kv,new,tiles", [
    (128, 2, 4, 16, [300, 90, 200], [2, 4, 1], False),
    (64, 2, 4, 32, [300, 90, 200], [2, 4, 1], False),
    (128, 2, 4, 16, [300, 90, 400], [40, 90, 300], True),
    (64, 2, 5, 32, [300, 90, 400], [40, 90, 300], True),
])
def test_weights_negative_scales_strided_queries_and_absent_pages(D, H, G, P, kv, new, tiles):
    for what in ("scale", "absent"):
        w = cache_util.make(kv, new, H, G, D, P, seed=D + G)
        if what == "absent":
            absent(w)
        else:
            w["q"] = cache_util.bits(bf16.to_f32(w["q"]).astype(np.float64) * 6)
        d = cache_util.dev(w)
        joint = torch.cat([torch.zeros_like(d["q"]), d["q"]], dim=1).contiguous()
        acc = np.random.default_rng(4).random((len(kv), H, max(kv) + 2)).astype(np.float32)
        need = fp8bs.cache_attention_weights_workspace_bytes(cache_dev(d), d["table"], H * G, max(new), acc.shape[2])
        assert (need > 0) == tiles
        for scale, cap in ((-0.1, 0.0), (0.1, 0.0), (-0.1, 8.0)):
            print(f"weights {what} D={D} tiles={tiles} scale={scale} cap={cap}", flush=True)
            args = (w["table"], w["q_offsets"], w["kv_lens"], scale)
            lse = oracle.attention(w["q"], cache_util.cache_of(w), *args, cap)[1].astype(np.float32)
            ref = oracle.weights(w["q"], lse, cache_util.cache_of(w), *args, acc, acc.shape[2], cap)
            out = fp8bs.cache_attention_weights(joint[:, H * G:], f32_dev(lse), cache_dev(d), d["table"], d["q_offsets"],
                                                d["kv_lens"], max(new), max(kv), scale, f32_dev(acc), softcap=cap)
            torch.cuda.synchronize()
            # the largest |lse| is rounded to FP32 on its way in: 2^-24 of it in a weight's exponent, and
            # again where it is taken to base 2
            top = np.abs(lse[np.isfinite(lse)]).max()
            e = 2 * score_error(w, scale, cap) + 2.0 ** -19 + 2.0 ** -22 * top + 2.0 ** -24 * max(new) * G / 2
            err = np.abs(out_host_f64(out) - ref)
            assert (err <= e * ref + 1e-30).all(), f"worst {np.max(err / (e * ref + 1e-30)):.3g}"


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64)])
def test_evict_from_absent_pages(D, P):
    # kept tokens of an absent page move as zeros and do not count for the scale
    kv, budget, recent, H = [400, 130, 260], 150, 20, 2
    w = cache_util.make(kv, [0] * 3, H, 1, D, P, seed=D, spare=3 * -(-budget // P))
    free = [p for p in range(w["k"].shape[0]) if p not in set(w["table"].ravel().tolist())]
    dst = np.array(free[:3 * -(-budget // P)], np.int32).reshape(3, -1)
    absent(w)
    acc = np.random.default_rng(6).random((3, H, 400)).astype(np.float32)
    d = cache_util.dev(w)
    print(f"evict from absent pages D={D} P={P}", flush=True)
    kept, lens, out = fp8bs.cache_evict(f32_dev(acc), cache_dev(d), d["table"], i32_dev(dst), d["kv_lens"], 400, budget,
                                        recent)
    torch.cuda.synchronize()
    rk, rl, ra = oracle.evict(acc, cache_util.cache_of(w), w["table"], dst, w["kv_lens"], budget, recent)
    assert np.array_equal(kept.cpu().numpy(), rk) and np.array_equal(lens.cpu().numpy(), rl)
    assert np.array_equal(f32_bits_host(out), ra.view(np.uint32))
    same_cache(d, w, "evict from absent pages")
