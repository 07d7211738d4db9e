"""GPU parity of the paged FP8 key/value cache against the float64 oracle.

Append and eviction are exact functions of their inputs: codes, scales,
indexes, lengths and sums are compared bit for bit.

Attention, elementwise.  With S the largest sum of |q_d k_d| * |scale| of the
case and A_j = sum over tokens of weight * |v|:
- a score is a sum of at most 128 exact products in FP32, then a few FP32
  operations: its error is at most 2^-17 S + 2^-19 (S enters capped scores with
  slope <= 1; the cap's own form adds cap * 2^-21);
- a weight's relative error is twice that (its own score, and the sum it is
  divided by), plus 2^-8 where it meets the codes in BF16 (round to nearest:
  2^-9, doubled);
- the output rounding is 2^-9 |out| for BF16 (2^-8 taken).
lse: the score error plus 2^-21 |lse|.  weights: the score error twice (score
and lse) plus FP32 rounding of score - lse, relative, plus 2^-20 relative for
the sum.
"""

import numpy as np
import pytest
import torch

from fp8_block_scaled_04_amd import fp8bs
from oracle import bf16, cache as oracle, e4m3
from tests import cache_util
from tests.gpu_util import assert_codes_equal, codes_host, f32_bits_host, f32_dev, out_host_f64, require_gpu

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_gpu()


# (cached tokens, rows) per sequence: one token and none at all; page ends
# inside and at the end of a matrix tile; more rows than cached tokens; whole
# prompts; chunks behind a prefix
LENS = {
    "one": ([1], [1]),
    "empty": ([0, 5, 0], [0, 1, 2]),
    "step": ([1, 15, 16, 17, 31, 33, 64, 100, 257], [1] * 9),
    "ragged": ([40, 130, 3, 77, 300], [7, 1, 3, 0, 45]),
    "overrun": ([4, 20], [9, 20]),
    "prompt": ([129, 64], [129, 64]),
    "long": ([1500, 2311], [1, 3]),
}
SHAPES = [  # heads, group, D, P
    (2, 1, 64, 16), (1, 4, 128, 16), (2, 3, 128, 32), (3, 5, 64, 64), (2, 8, 128, 128), (1, 16, 64, 32), (1, 17, 128, 64),
]


def cache_dev(d):
    return d["k"], d["ks"], d["v"], d["vs"]


def same_cache(d, w, what, pages=None):
    """Codes and scales equal bit for bit (on `pages`, else everywhere)."""
    sel = slice(None) if pages is None else pages
    for n in ("k", "v"):
        assert_codes_equal(codes_host(d[n])[sel], w[n][sel], f"{what} {n} codes")
        got, ref = f32_bits_host(d[n + "s"])[sel], w[n + "s"].view(np.uint32)[sel]
        nan = np.isnan(w[n + "s"])[sel]
        assert np.array_equal(got[~nan], ref[~nan]), f"{what} {n} scales"


def score_error(w, scale, cap):
    q = np.abs(bf16.to_f32(w["q"]).astype(np.float64))
    S = 0.0
    for b in range(len(w["kv_lens"])):
        lo, hi = w["q_offsets"][b], w["q_offsets"][b + 1]
        for hq in range(q.shape[1] if hi > lo else 0):
            k, _ = oracle.values(w["k"], w["ks"], w["table"][b], int(w["kv_lens"][b]), hq // w["G"])
            if k.size:
                S = max(S, float((q[lo:hi, hq] @ np.abs(k).T).max()) * abs(scale))
    return 2.0 ** -17 * S + 2.0 ** -19 + cap * 2.0 ** -21


def abs_values(w):
    w2 = dict(w)
    w2["v"] = w["v"] & 0x7F
    return cache_util.cache_of(w2)


def check_attention(w, out, lse, scale, cap, full, what):
    args = (w["table"], w["q_offsets"], w["kv_lens"], scale, cap, full)
    ref, ref_lse = oracle.attention(w["q"], cache_util.cache_of(w), *args)
    size, _ = oracle.attention(w["q"], abs_values(w), *args)
    e = score_error(w, scale, cap)
    got = out_host_f64(out)
    tol = (2 * e + 2.0 ** -8) * size + 1e-30
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of tolerance, first {np.argwhere(bad)[:3].tolist()}"
    none = np.isneginf(ref_lse)
    assert (got[none] == 0).all(), f"{what}: rows that see nothing"
    if lse is not None:
        z = lse.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isneginf(z), none), f"{what}: lse of empty rows"
        assert (np.abs(z[~none] - ref_lse[~none]) <= e + 2.0 ** -21 * np.abs(ref_lse[~none])).all(), f"{what}: lse"
    return ref_lse


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,G,D,P", SHAPES)
def test_append(lens, H, G, D, P):
    kv, new = LENS[lens]
    for pow2 in (False, True):
        print(f"append {lens} H={H} D={D} P={P} pow2={pow2}", flush=True)
        w = cache_util.make(kv, new, H, 1, D, P, seed=H + D + P)
        d = cache_util.dev(w)
        fp8bs.cache_append(d["k_new"], d["v_new"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], w["max_new"],
                           pow2)
        torch.cuda.synchronize()
        oracle.append(cache_util.cache_of(w), w["k_new"], w["v_new"], w["table"], w["q_offsets"], w["kv_lens"], pow2)
        same_cache(d, w, f"append {lens}")


def test_append_special_values_token_by_token():
    # one token per call: zeros first (scale 0), subnormals, tiny, ordinary and
    # the largest BF16 values; every step grows the page's scale
    D, P, H = 64, 16, 2
    rows = [0.0, 2.0 ** -133, 2.0 ** -100, 2.0 ** -70, 2.0 ** -60, 1e-3, 0.0, 1.0, 300.0, 3.3e38]
    rng = np.random.default_rng(3)
    for pow2 in (False, True):
        w = cache_util.make([len(rows)], [1], H, 1, D, P)
        w["ks"][:], w["vs"][:] = 7.0, 7.0                     # a page's old contents do not matter
        d = cache_util.dev(w)
        for i, size in enumerate(rows):
            x = rng.standard_normal((1, H, D))
            w["k_new"] = cache_util.bits(size * x / np.abs(x).max())
            w["v_new"] = cache_util.bits(-size * x / np.abs(x).max())
            w["kv_lens"][:] = i + 1
            e = cache_util.dev(w)
            fp8bs.cache_append(e["k_new"], e["v_new"], cache_dev(d), d["table"], d["q_offsets"], e["kv_lens"], 1, pow2)
            torch.cuda.synchronize()
            oracle.append(cache_util.cache_of(w), w["k_new"], w["v_new"], w["table"], w["q_offsets"], w["kv_lens"], pow2)
            same_cache(d, w, f"token {i}")


def test_append_strided_rows_and_absent_pages():
    # keys and values as slices of one projection; a table entry outside the pool
    w = cache_util.make([40, 50], [40, 30], 3, 1, 128, 16, seed=5)
    w["table"][1, 2] = 10 ** 6
    w["table"][1, 3] = -1
    d = cache_util.dev(w)
    joint = torch.cat([torch.zeros_like(d["k_new"]), d["k_new"], d["v_new"]], dim=1).contiguous()
    fp8bs.cache_append(joint[:, 3:6], joint[:, 6:9], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], 40)
    torch.cuda.synchronize()
    oracle.append(cache_util.cache_of(w), w["k_new"], w["v_new"], w["table"], w["q_offsets"], w["kv_lens"])
    same_cache(d, w, "strided append")


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,G,D,P", SHAPES)
def test_attention(lens, H, G, D, P):
    kv, new = LENS[lens]
    w = cache_util.make(kv, new, H, G, D, P, seed=H + G + D)
    d = cache_util.dev(w)
    scale = D ** -0.5
    for cap, full, dtype in ((0.0, False, torch.bfloat16), (3.0, False, torch.float32), (0.0, True, torch.float32)):
        what = f"attention {lens} H={H} G={G} D={D} P={P} cap={cap} full={full}"
        print(what, flush=True)
        out, lse = fp8bs.cache_attention(d["q"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], w["max_new"],
                                         w["max_kv"], scale, softcap=cap, full=full, out_dtype=dtype, return_lse=True)
        torch.cuda.synchronize()
        check_attention(w, out, lse, scale, cap, full, what)


@pytest.mark.parametrize("G,D", [(1, 128), (4, 64), (16, 128)])
def test_attention_many_rows_behind_a_prefix(G, D):
    # row counts around the row tiles, lengths around the token tiles
    w = cache_util.make([700, 513, 260, 129], [150, 64, 33, 129], 1, G, D, 32, seed=G)
    d = cache_util.dev(w)
    for cap in (0.0, 20.0):
        print(f"many rows G={G} D={D} cap={cap}", flush=True)
        out, lse = fp8bs.cache_attention(d["q"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], 150, 700,
                                         D ** -0.5, softcap=cap, return_lse=True)
        torch.cuda.synchronize()
        check_attention(w, out, lse, D ** -0.5, cap, False, f"many rows G={G} D={D}")


BOUND = 1 << 16                                      # of cached tokens: with it few rows go to the larger row tiles


@pytest.mark.parametrize("lens", ["ragged", "overrun", "prompt"])
@pytest.mark.parametrize("H,G,D,P", SHAPES)
def test_attention_on_larger_row_tiles(lens, H, G, D, P):
    kv, new = LENS[lens]
    w = cache_util.make(kv, new, H, G, D, P, seed=H + G + D + 1)
    d = cache_util.dev(w)
    for cap, full, max_new in ((0.0, False, 130), (3.0, False, 257), (0.0, True, 129)):
        what = f"larger tiles {lens} H={H} G={G} D={D} P={P} cap={cap} full={full}"
        print(what, flush=True)
        out, lse = fp8bs.cache_attention(d["q"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], max_new, BOUND,
                                         D ** -0.5, softcap=cap, full=full, out_dtype=torch.float32, return_lse=True)
        torch.cuda.synchronize()
        check_attention(w, out, lse, D ** -0.5, cap, full, what)


@pytest.mark.parametrize("D,bound", [(64, 6000), (128, 6000), (128, 1400), (64, 700)])
def test_attention_larger_row_tiles_in_splits(D, bound):
    # 6016 (row, head) pairs: several splits hold tokens, others none
    w = cache_util.make([700, 513, 260, 129], [150, 64, 33, 129], 1, 16, D, 64, seed=bound)
    d = cache_util.dev(w)
    for cap in (0.0, 20.0):
        print(f"larger tiles in splits D={D} bound={bound} cap={cap}", flush=True)
        out, lse = fp8bs.cache_attention(d["q"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], 150, bound,
                                         D ** -0.5, softcap=cap, return_lse=True)
        torch.cuda.synchronize()
        check_attention(w, out, lse, D ** -0.5, cap, False, f"larger tiles in splits D={D} bound={bound}")


@pytest.mark.parametrize("kv,new,G", [([250, 200], [250, 200], 40), ([640, 300], [520, 300], 24)])
def test_attention_many_pairs(kv, new, G):
    # more (row, head) pairs than 16-row tiles take at D = 64, in one split and in three
    w = cache_util.make(kv, new, 2, G, 64, 64, seed=G)
    d = cache_util.dev(w)
    print(f"many pairs G={G}", flush=True)
    out, lse = fp8bs.cache_attention(d["q"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], max(new), max(kv),
                                     0.125, return_lse=True)
    torch.cuda.synchronize()
    check_attention(w, out, lse, 0.125, 0.0, False, f"many pairs G={G}")


def test_attention_long_splits():
    # a bound far above the lengths makes splits of more than 32 steps a wave
    # (pages and scales are looked up 32 steps at a time)
    w = cache_util.make([6000, 4300, 5121], [1, 2, 1], 2, 2, 64, 16, seed=8, table_extra=0)
    d = cache_util.dev(w)
    out, lse = fp8bs.cache_attention(d["q"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], 2, 400000, 0.125,
                                     return_lse=True)
    torch.cuda.synchronize()
    check_attention(w, out, lse, 0.125, 0.0, False, "long splits")


def test_attention_large_scores_and_strided_queries():
    # scores in the hundreds (the running maximum moves late), negative scale,
    # queries as a slice of a wider projection, a bound far above the lengths
    w = cache_util.make([300, 90], [2, 30], 2, 4, 128, 64, seed=9)
    w["q"] = cache_util.bits(bf16.to_f32(w["q"]).astype(np.float64) * 12)
    d = cache_util.dev(w)
    joint = torch.cat([d["q"], torch.zeros_like(d["q"])], dim=1).contiguous()
    for scale in (0.4, -0.4):
        print(f"large scores scale={scale}", flush=True)
        out, lse = fp8bs.cache_attention(joint[:, :8], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], 64, 5000,
                                         scale, return_lse=True)
        torch.cuda.synchronize()
        check_attention(w, out, lse, scale, 0.0, False, f"large scores {scale}")


@pytest.mark.parametrize("D,new", [(128, 140), (64, 140), (128, 20), (64, 1)])
def test_attention_extreme_value_scales(D, new):
    # pages of zeros (scale 0), and scales near both ends of the FP32 range,
    # beside ordinary ones; every sequence has one kind, the last a mix
    w = cache_util.make([200, 333, 150, 400], [new, new, new, new], 1, 2, D, 32, seed=D + new)
    sizes = [0.0, 2.0 ** -120, 2.0 ** 100]
    for b in range(4):
        for j, page in enumerate(w["table"][b][:-(-int(w["kv_lens"][b]) // 32)]):
            size = sizes[b] if b < 3 else sizes[:2][j % 2] if j % 3 else 1.0
            w["vs"][page] = size
            if size == 0.0:
                w["v"][page][w["v"][page] != 0x7F] = 0
    d = cache_util.dev(w)
    for cap in (0.0, 9.0):
        out, lse = fp8bs.cache_attention(d["q"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], new, 400,
                                         D ** -0.5, softcap=cap, return_lse=True)
        torch.cuda.synchronize()
        check_attention(w, out, lse, D ** -0.5, cap, False, f"extreme scales D={D} new={new} cap={cap}")


@pytest.mark.parametrize("D,new", [(128, 140), (64, 140), (128, 40)])
def test_attention_extreme_value_scales_on_larger_row_tiles(D, new):
    # pages of zeros (scale 0), and scales near both ends of the FP32 range,
    # beside ordinary ones; every sequence has one kind, the last a mix
    w = cache_util.make([200, 333, 150, 400], [new, new, new, new], 1, 2, D, 32, seed=D + new)
    sizes = [0.0, 2.0 ** -120, 2.0 ** 100]
    for b in range(4):
        for j, page in enumerate(w["table"][b][:-(-int(w["kv_lens"][b]) // 32)]):
            size = sizes[b] if b < 3 else sizes[:2][j % 2] if j % 3 else 1.0
            w["vs"][page] = size
            if size == 0.0:
                w["v"][page][w["v"][page] != 0x7F] = 0
    d = cache_util.dev(w)
    for cap in (0.0, 9.0):
        out, lse = fp8bs.cache_attention(d["q"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], new, BOUND,
                                         D ** -0.5, softcap=cap, return_lse=True)
        torch.cuda.synchronize()
        check_attention(w, out, lse, D ** -0.5, cap, False, f"extreme scales, larger tiles D={D} new={new} cap={cap}")


def test_attention_absent_pages_and_all_absent_rows():
    # tokens of a table entry outside the pool do not exist; a sequence with
    # only such tokens has empty rows
    w = cache_util.make([100, 40, 200], [1, 2, 20], 1, 4, 64, 16, seed=2)
    w["table"][0, 1] = -1
    w["table"][1, :] = 1 << 20
    w["table"][2, 5:9] = -(1 << 31)
    d = cache_util.dev(w)
    out, lse = fp8bs.cache_attention(d["q"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], 20, 200, 0.1,
                                     return_lse=True)
    torch.cuda.synchronize()
    check_attention(w, out, lse, 0.1, 0.0, False, "absent pages")
    assert torch.isneginf(lse[1:3]).all()


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,G,D,P", SHAPES)
def test_attention_weights(lens, H, G, D, P):
    kv, new = LENS[lens]
    w = cache_util.make(kv, new, H, G, D, P, seed=H + G + D + 1)
    d = cache_util.dev(w)
    scale = D ** -0.5
    slots = w["max_kv"] + 5
    rng = np.random.default_rng(1)
    acc = rng.random((len(kv), H, slots)).astype(np.float32)
    for b in range(len(kv)):
        acc[b, :, max(0, kv[b] - new[b]):] = np.nan          # sums of new and absent slots are not read
    for cap, full in ((0.0, False), (3.0, True)):
        what = f"weights {lens} H={H} G={G} D={D} P={P} cap={cap} full={full}"
        print(what, flush=True)
        args = (w["table"], w["q_offsets"], w["kv_lens"], scale)
        _, lse = oracle.attention(w["q"], cache_util.cache_of(w), *args, cap, full)
        lse = lse.astype(np.float32)
        ref = oracle.weights(w["q"], lse, cache_util.cache_of(w), *args, acc, slots, cap, full)
        out = fp8bs.cache_attention_weights(d["q"], f32_dev(lse), cache_dev(d), d["table"], d["q_offsets"],
                                            d["kv_lens"], w["max_new"], w["max_kv"], scale, f32_dev(acc),
                                            softcap=cap, full=full)
        torch.cuda.synchronize()
        e = 2 * score_error(w, scale, cap) + 2.0 ** -19
        err = np.abs(out_host_f64(out) - ref)
        assert (err <= e * ref + 1e-30).all(), f"{what}: worst {np.max(err / (e * ref + 1e-30)):.3g}"
        # in place, and from nothing
        a = f32_dev(acc)
        got = fp8bs.cache_attention_weights(d["q"], f32_dev(lse), cache_dev(d), d["table"], d["q_offsets"],
                                            d["kv_lens"], w["max_new"], w["max_kv"], scale, a, softcap=cap, full=full,
                                            out=a)
        assert got is a and torch.equal(a, out), what
        fresh = fp8bs.cache_attention_weights(d["q"], f32_dev(lse), cache_dev(d), d["table"], d["q_offsets"],
                                              d["kv_lens"], w["max_new"], w["max_kv"], scale, softcap=cap, full=full,
                                              slots=slots)
        ref0 = oracle.weights(w["q"], lse, cache_util.cache_of(w), *args, None, slots, cap, full)
        assert (np.abs(out_host_f64(fresh) - ref0) <= e * ref0 + 1e-30).all(), what


@pytest.mark.parametrize("G,D", [(1, 128), (4, 64), (6, 128)])
def test_attention_weights_many_rows(G, D):
    # rows split over workgroups, slots that no early row sees, steps whose first
    # rows see only some of a wave's tokens
    w = cache_util.make([1500, 777, 600], [1100, 500, 600], 1, G, D, 64, seed=G + D)
    d = cache_util.dev(w)
    scale = D ** -0.5
    for cap, full in ((0.0, False), (4.0, False), (0.0, True)):
        print(f"weights many rows G={G} D={D} cap={cap} full={full}", flush=True)
        args = (w["table"], w["q_offsets"], w["kv_lens"], scale)
        _, lse = oracle.attention(w["q"], cache_util.cache_of(w), *args, cap, full)
        lse = lse.astype(np.float32)
        ref = oracle.weights(w["q"], lse, cache_util.cache_of(w), *args, None, 1600, cap, full)
        assert fp8bs.cache_attention_weights_workspace_bytes(cache_dev(d), d["table"], G, 1100, 1600) > 0
        out = fp8bs.cache_attention_weights(d["q"], f32_dev(lse), cache_dev(d), d["table"], d["q_offsets"],
                                            d["kv_lens"], 1100, 1500, scale, softcap=cap, full=full, slots=1600)
        torch.cuda.synchronize()
        # FP32 sums of up to 1100 G weights: 2^-24 of the running sum a step
        e = 2 * score_error(w, scale, cap) + 2.0 ** -19 + 2.0 ** -24 * 1100 * G / 2
        err = np.abs(out_host_f64(out) - ref)
        assert (err <= e * ref + 1e-30).all(), f"worst {np.max(err / (e * ref + 1e-30)):.3g}"


@pytest.mark.parametrize("kv,budget,recent", [([5000, 9000], 3000, 100), ([20000, 17000, 40], 6000, 0),
                                              ([16384, 16385, 4096], 4096, 4000)])
def test_evict_long(kv, budget, recent):
    # sums that stay in registers in one or several blocks, and ones that are
    # read again by each pass; many ties
    H, D, P = 1, 64, 128
    w = cache_util.make(kv, [0] * len(kv), H, 1, D, P, seed=1, spare=sum(-(-min(t, budget) // P) for t in kv) + 3)
    used = set(w["table"][w["table"] >= 0].tolist())
    free = [p for p in range(w["k"].shape[0]) if p not in used]
    dst = np.full((len(kv), -(-budget // P)), -1, np.int32)
    for b, t in enumerate(kv):
        n = -(-min(t, budget) // P)
        dst[b, :n], free = free[:n], free[n:]
    rng = np.random.default_rng(7)
    for kind in ("spread", "ties"):
        print(f"evict long {kind} kv={kv}", flush=True)
        acc = np.exp(3 * rng.standard_normal((len(kv), H, max(kv)))).astype(np.float32)
        if kind == "ties":
            acc = np.floor(acc).astype(np.float32)
        wk = {n: (v.copy() if isinstance(v, np.ndarray) else v) for n, v in w.items()}
        d = cache_util.dev(wk)
        kept, lens, out = fp8bs.cache_evict(f32_dev(acc), cache_dev(d), d["table"], torch.from_numpy(dst).cuda(),
                                            d["kv_lens"], max(kv), budget, recent)
        torch.cuda.synchronize()
        rk, rl, ra = oracle.evict(acc, cache_util.cache_of(wk), w["table"], dst, w["kv_lens"], budget, recent)
        assert np.array_equal(kept.cpu().numpy(), rk) and np.array_equal(lens.cpu().numpy(), rl)
        assert np.array_equal(f32_bits_host(out), ra.view(np.uint32))
        same_cache(d, wk, "evict long")


@pytest.mark.parametrize("H,D,P", [(1, 64, 16), (2, 128, 32), (3, 64, 64), (2, 128, 128)])
@pytest.mark.parametrize("kv,budget,recent", [([300, 33, 0, 128], 100, 10), ([70], 64, 64), ([1, 2, 3], 2, 0),
                                              ([2500, 1024, 1025], 1000, 7), ([50, 20], 90, 5), ([40], 16, 400)])
def test_evict(H, D, P, kv, budget, recent):
    w = cache_util.make(kv, [0] * len(kv), H, 1, D, P, seed=H + P, spare=sum(-(-min(t, budget) // P) for t in kv) + 3)
    used = set(w["table"][w["table"] >= 0].tolist())
    free = [p for p in range(w["k"].shape[0]) if p not in used]
    width = -(-min(budget, w["max_kv"]) // P)
    dst = np.full((len(kv), width), -1, np.int32)
    for b, t in enumerate(kv):
        n = -(-min(t, budget) // P)
        dst[b, :n], free = free[:n], free[n:]
    slots = w["max_kv"] + 3
    rng = np.random.default_rng(len(kv))
    for kind in ("spread", "ties", "special"):
        print(f"evict {kind} H={H} D={D} P={P} kv={kv} budget={budget} recent={recent}", flush=True)
        acc = np.exp(3 * rng.standard_normal((len(kv), H, slots))).astype(np.float32)
        if kind == "ties":
            acc = rng.integers(0, 3, acc.shape).astype(np.float32)
        if kind == "special":
            acc[rng.random(acc.shape) < 0.3] = 0.0
            acc[rng.random(acc.shape) < 0.3] *= -1                 # -0 ties with +0
            for x in (np.nan, np.inf, -np.inf, 1e-42):
                acc[rng.random(acc.shape) < 0.1] = x
        wk = {n: (v.copy() if isinstance(v, np.ndarray) else v) for n, v in w.items()}
        d = cache_util.dev(wk)
        kept, lens, out = fp8bs.cache_evict(f32_dev(acc), cache_dev(d), d["table"], torch.from_numpy(dst).cuda(),
                                            d["kv_lens"], w["max_kv"], budget, recent)
        torch.cuda.synchronize()
        rk, rl, ra = oracle.evict(acc, cache_util.cache_of(wk), w["table"], dst, w["kv_lens"], budget, recent)
        assert np.array_equal(kept.cpu().numpy(), rk), "kept slots"
        assert np.array_equal(lens.cpu().numpy(), rl), "lengths"
        assert np.array_equal(f32_bits_host(out), ra.view(np.uint32)), "sums"
        same_cache(d, wk, "evict")


def test_serving_loop_on_a_side_stream_replayed_as_a_graph():
    # append, attend, sum and evict on a stream of their own, captured: every
    # replay equals the eager pass
    w = cache_util.make([90, 200, 17], [1, 1, 1], 2, 4, 128, 32, seed=4, spare=12)
    d = cache_util.dev(w)
    keep = [t.clone() for t in cache_dev(d)]
    used = set(w["table"][w["table"] >= 0].tolist())
    free = [p for p in range(w["k"].shape[0]) if p not in used][:6]
    dst = torch.tensor([free[0:2], free[2:4], free[4:6]], dtype=torch.int32, device="cuda")
    acc = torch.rand(3, 2, 200, device="cuda")

    def step():
        cache = cache_dev(d)
        fp8bs.cache_append(d["k_new"], d["v_new"], cache, d["table"], d["q_offsets"], d["kv_lens"], 1)
        out, lse = fp8bs.cache_attention(d["q"], cache, d["table"], d["q_offsets"], d["kv_lens"], 1, 200, 0.1,
                                         return_lse=True)
        a = fp8bs.cache_attention_weights(d["q"], lse, cache, d["table"], d["q_offsets"], d["kv_lens"], 1, 200, 0.1, acc)
        return (out, lse, a, *fp8bs.cache_evict(a, cache, d["table"], dst, d["kv_lens"], 200, 60, 8), *cache)

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        got = step()
    for rep in range(4):
        for t, k in zip(cache_dev(d), keep):
            t.copy_(k)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            a, b = a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)
            assert torch.equal(a, b), f"replay {rep}, output {i}"
        step()
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    # a pool whose pages start past 2^32 bytes: the last pages are used
    H, D, P = 8, 128, 128
    pages = (1 << 32) // (H * D * P) + 4
    print(f"pool of {pages} pages, {pages * H * D * P} bytes each for keys and values", flush=True)
    w = cache_util.make([200, 300], [1, 5], H, 2, D, P, seed=6, spare=0)
    small = cache_util.dev(w)
    n = w["k"].shape[0]
    k = torch.zeros((pages, H, P, D), dtype=torch.uint8, device="cuda")
    v = torch.zeros((pages, H, P, D), dtype=torch.uint8, device="cuda")
    ks = torch.zeros((pages, H), device="cuda")
    vs = torch.zeros((pages, H), device="cuda")
    at = pages - n
    k[at:], v[at:] = small["k"].view(torch.uint8), small["v"].view(torch.uint8)
    ks[at:], vs[at:] = small["ks"], small["vs"]
    table = torch.where(small["table"] >= 0, small["table"] + at, small["table"])
    big = (k.view(torch.float8_e4m3fn), ks, v.view(torch.float8_e4m3fn), vs)
    args = (small["q_offsets"], small["kv_lens"])
    for pool, tab in ((cache_dev(small), small["table"]), (big, table)):
        fp8bs.cache_append(small["k_new"], small["v_new"], pool, tab, *args, 5)
    a = fp8bs.cache_attention(small["q"], cache_dev(small), small["table"], *args, 5, 300, 0.1, return_lse=True)
    b = fp8bs.cache_attention(small["q"], big, table, *args, 5, 300, 0.1, return_lse=True)
    wa = fp8bs.cache_attention_weights(small["q"], a[1], cache_dev(small), small["table"], *args, 5, 300, 0.1)
    wb = fp8bs.cache_attention_weights(small["q"], b[1], big, table, *args, 5, 300, 0.1)
    torch.cuda.synchronize()
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])
    assert torch.equal(wa, wb)
    assert torch.equal(small["k"].view(torch.uint8), k[at:])


def test_refusals():
    w = cache_util.make([20], [2], 2, 2, 64, 16)
    d = cache_util.dev(w)
    cache, rest = cache_dev(d), (d["table"], d["q_offsets"], d["kv_lens"])
    attend = lambda q=d["q"], c=cache, r=rest, **kw: fp8bs.cache_attention(q, c, *r, 2, 20, 0.1, **kw)  # noqa: E731
    for bad in (dict(q=d["q"].float()), dict(out_dtype=torch.float16), dict(c=(d["k"].float(), *cache[1:]))):
        with pytest.raises(TypeError):
            attend(**bad)
    for bad in (dict(q=d["q"][:, :, :32]), dict(q=d["q"].transpose(1, 2)), dict(q=d["q"].cpu()),
                dict(c=(cache[0][:, :1], *cache[1:])), dict(c=(cache[0], cache[1][:1], *cache[2:])),
                dict(r=(d["table"], d["q_offsets"][:1], d["kv_lens"])), dict(r=(d["table"].cpu(), *rest[1:])),
                dict(r=(d["table"], d["q_offsets"], d["kv_lens"].repeat(2))),
                dict(out=torch.empty(2, 4, 32, device="cuda", dtype=torch.bfloat16)),
                dict(workspace=torch.empty(8, device="cuda"))):
        with pytest.raises(ValueError):
            attend(**bad)
    with pytest.raises(fp8bs.Fp8bsError):
        attend(softcap=-1.0)
    with pytest.raises(fp8bs.Fp8bsError):
        attend(q=d["q"][:, :3].contiguous())                        # 3 query heads on 2 key heads
    odd = torch.zeros(6, 2, 24, 64, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.zeros(6, 2, device="cuda")
    with pytest.raises(fp8bs.Fp8bsError):
        attend(c=(odd, sc, odd, sc))                                # pages of 24 tokens
    with pytest.raises(ValueError):
        fp8bs.cache_append(d["k_new"], d["v_new"][:1], cache, *rest, 2)
    acc = torch.zeros(1, 2, 10, device="cuda")
    with pytest.raises(fp8bs.Fp8bsError):
        fp8bs.cache_evict(acc, cache, d["table"], d["table"], d["kv_lens"], 20, 8, 2)     # fewer sums than slots
    torch.cuda.synchronize()
