"""The cache calls where a sequence is longer than the call's bounds: more cached
tokens than max_kv or the table hold, more rows than max_new.

Row i of n is slot kv_len - n + i whatever the bounds; slots from min(max_kv,
table_width * P) on and rows from max_new on are left out.  Tolerances are those
of tests/test_gpu_cache.py.
"""

import numpy as np
import pytest
import torch

from fp8_block_scaled_04_amd import fp8bs
from oracle import cache as oracle
from tests import cache_util
from tests.gpu_util import f32_bits_host, f32_dev, i32_dev, out_host_f64, require_gpu
from tests.test_gpu_cache import abs_values, cache_dev, same_cache, score_error

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_gpu()


def long_case(kv, new, more, H, G, D, P, seed):
    """Sequences whose lengths pass their tables by more[b] (the table ends with
    the longest one's last page)."""
    w = cache_util.make(kv, new, H, G, D, P, seed=seed, table_extra=0)
    w["kv_lens"] = w["kv_lens"] + np.array(more, np.int32)
    return w


def clamped(w, max_kv):
    """The case as far as scores go: lengths within the bounds."""
    c = dict(w)
    c["kv_lens"] = np.array([oracle.held(cache_util.cache_of(w), w["table"], n, max_kv) for n in w["kv_lens"]], np.int32)
    return c


def owned_rows(w, max_new):
    """Which packed rows the call computes."""
    own = np.zeros(w["q"].shape[0], bool)
    for lo, hi in zip(w["q_offsets"][:-1], w["q_offsets"][1:]):
        own[lo:min(hi, lo + max_new)] = True
    return own


def check(w, max_new, max_kv, scale, cap, full, what):
    """One attention call -> float64 lse of the oracle."""
    d = cache_util.dev(w)
    T, Hq, D = w["q"].shape
    out = torch.full((T, Hq, D), 77.0, dtype=torch.float32, device="cuda")
    print(what, flush=True)
    _, lse = fp8bs.cache_attention(d["q"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], max_new, max_kv,
                                   scale, softcap=cap, full=full, out_dtype=torch.float32, out=out, return_lse=True)
    torch.cuda.synchronize()
    args = (w["table"], w["q_offsets"], w["kv_lens"], scale, cap, full, max_new, max_kv)
    ref, ref_lse = oracle.attention(w["q"], cache_util.cache_of(w), *args)
    size, _ = oracle.attention(w["q"], abs_values(w), *args)
    e = score_error(clamped(w, max_kv), scale, cap)
    own, got = owned_rows(w, max_new), out_host_f64(out)
    assert (got[~own] == 77.0).all(), f"{what}: rows past max_new were written"
    bad = ~(np.abs(got - ref) <= (2 * e + 2.0 ** -8) * size + 1e-30)[own]
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of tolerance"
    z, none = lse.cpu().numpy().astype(np.float64)[own], np.isneginf(ref_lse[own])
    assert np.array_equal(np.isneginf(z), none), f"{what}: lse of empty rows"
    z, want = z[~none], ref_lse[own][~none]
    assert (np.abs(z - want) <= e + 2.0 ** -21 * np.abs(want)).all(), f"{what}: lse"
    return ref_lse


# cached tokens, rows, tokens past the table, heads, group, D, P, max_new, max_kv
CASES = {
    "few rows, short max_kv": ([100, 30, 64, 65], [10, 3, 1, 64], [0] * 4, 2, 2, 64, 16, 64, 64),
    "few rows past the table": ([64, 40, 64], [10, 3, 2], [6, 0, 100], 2, 3, 128, 16, 10, 500),
    "few rows, more than max_new": ([100, 30, 20, 5], [10, 3, 20, 9], [0] * 4, 1, 4, 64, 32, 2, 100),
    "256-row tiles, short max_kv": ([700, 513, 260, 129], [150, 64, 33, 129], [0] * 4, 1, 16, 128, 32, 150, 512),
    "256-row tiles past the table": ([704, 513, 704], [150, 64, 63], [90, 0, 700], 1, 16, 128, 32, 150, 6000),
    "256-row tiles, more than max_new": ([700, 513, 260, 100], [250, 64, 233, 129], [0] * 4, 1, 16, 128, 64, 120, 700),
    "128-row tiles, short max_kv": ([300, 128, 129, 90] * 10, [7] * 40, [0] * 40, 1, 16, 128, 16, 7, 128),
    "128-row tiles of D = 64, short max_kv": ([250, 200], [250, 200], [0, 0], 2, 40, 64, 64, 250, 190),
    "128-row tiles of D = 64 past the table": ([256, 200], [250, 200], [30, 0], 2, 40, 64, 64, 250, 400),
}


@pytest.mark.parametrize("name", CASES)
def test_attention(name):
    kv, new, more, H, G, D, P, max_new, max_kv = CASES[name]
    w = long_case(kv, new, more, H, G, D, P, seed=H + G + D)
    for cap, full in ((0.0, False), (3.0, False), (0.0, True)):
        check(w, max_new, max_kv, D ** -0.5, cap, full, f"{name} cap={cap} full={full}")


@pytest.mark.parametrize("name", CASES)
def test_weights(name):
    kv, new, more, H, G, D, P, max_new, max_kv = CASES[name]
    w = long_case(kv, new, more, H, G, D, P, seed=H + G + D + 1)
    d = cache_util.dev(w)
    slots = max_kv + 3
    acc = np.random.default_rng(2).random((len(kv), H, slots)).astype(np.float32)
    for cap, full in ((0.0, False), (3.0, True)):
        print(f"weights {name} cap={cap} full={full}", flush=True)
        args = (w["table"], w["q_offsets"], w["kv_lens"], D ** -0.5)
        _, lse = oracle.attention(w["q"], cache_util.cache_of(w), *args, cap, full, max_new, max_kv)
        lse = lse.astype(np.float32)
        ref = oracle.weights(w["q"], lse, cache_util.cache_of(w), *args, acc, slots, cap, full, max_new, max_kv)
        out = fp8bs.cache_attention_weights(d["q"], f32_dev(lse), cache_dev(d), d["table"], d["q_offsets"],
                                            d["kv_lens"], max_new, max_kv, D ** -0.5, f32_dev(acc), softcap=cap,
                                            full=full)
        torch.cuda.synchronize()
        e = 2 * score_error(clamped(w, max_kv), D ** -0.5, cap) + 2.0 ** -19 + 2.0 ** -24 * max_new * G / 2
        assert (np.abs(out_host_f64(out) - ref) <= e * ref + 1e-30).all(), name


@pytest.mark.parametrize("max_new,G", [(64, 1), (64, 3), (70, 1)])
def test_weights_where_no_row_sees_a_slot(max_new, G):
    # 200 rows of 5 cached tokens: the first rows, all that max_new lets in, lie
    # before the first slot
    w = cache_util.make([5, 5], [200, 3], 2, G, 64, 16, seed=G)
    d = cache_util.dev(w)
    lse = oracle.attention(w["q"], cache_util.cache_of(w), w["table"], w["q_offsets"], w["kv_lens"], 0.1)[1].astype(np.float32)
    acc = f32_dev(np.ones((2, 2, 8)))
    print(f"weights of hidden rows max_new={max_new} G={G}", flush=True)
    for n in (1, 2):
        args = (w["table"][:n], w["q_offsets"][:n + 1], w["kv_lens"][:n], 0.1, np.ones((n, 2, 8)), 8)
        ref = oracle.weights(w["q"], lse, cache_util.cache_of(w), *args, max_new=max_new)
        out = fp8bs.cache_attention_weights(d["q"], f32_dev(lse), cache_dev(d), d["table"][:n], d["q_offsets"][:n + 1],
                                            d["kv_lens"][:n], max_new, 5, 0.1, acc[:n])
        torch.cuda.synchronize()
        assert (ref[0] == 0).all() and (out[0] == 0).all()
        assert (np.abs(out_host_f64(out) - ref) <= 2.0 ** -12 * ref).all()


@pytest.mark.parametrize("P,D", [(16, 64), (64, 128)])
@pytest.mark.parametrize("kv,new,more,max_new", [
    ([128, 100, 128], [1, 1, 3], [1, 0, 1], 3),          # the last rows have no place
    ([128, 128], [5, 70], [5, 200], 70),                 # none of them has, nor of 70 behind 258
    ([128, 128], [100, 40], [50, 20], 100),              # some of them have not
    ([100, 60, 128], [50, 60, 33], [0, 0, 7], 20),       # rows past max_new
])
def test_append(kv, new, more, max_new, P, D):
    w = long_case(kv, new, more, 2, 1, D, P, seed=P + D)
    d = cache_util.dev(w)
    print(f"append P={P} D={D} kv={kv} new={new} more={more}", flush=True)
    fp8bs.cache_append(d["k_new"], d["v_new"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], max_new)
    torch.cuda.synchronize()
    oracle.append(cache_util.cache_of(w), w["k_new"], w["v_new"], w["table"], w["q_offsets"], w["kv_lens"],
                  max_new=max_new)
    same_cache(d, w, "append")


def test_negative_lengths_hold_nothing():
    w = cache_util.make([0, 40], [2, 3], 1, 2, 64, 16, seed=3)
    w["kv_lens"][0] = -(1 << 31)
    before = {n: w[n].copy() for n in ("k", "ks", "v", "vs")}
    d = cache_util.dev(w)
    fp8bs.cache_append(d["k_new"], d["v_new"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], 3)
    out, lse = fp8bs.cache_attention(d["q"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], 3, 40, 0.1,
                                     return_lse=True)
    torch.cuda.synchronize()
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all() and torch.isfinite(lse[2:]).all()
    w["kv_lens"][0] = 0
    oracle.append(cache_util.cache_of(w), w["k_new"], w["v_new"], w["table"], w["q_offsets"], w["kv_lens"])
    same_cache(d, w, "append")
    mine = [p for p in range(w["k"].shape[0]) if p not in w["table"][1]]
    assert (w["k"][mine] == before["k"][mine]).all()


@pytest.mark.parametrize("max_kv", [90, 128])
def test_evict(max_kv):
    # cached tokens past max_kv, and past the table, are neither kept nor ranked
    H, D, P, budget, recent = 2, 64, 16, 40, 6
    w = cache_util.make([128, 60, 100], [0] * 3, H, 1, D, P, seed=4, spare=12, table_extra=0)
    w["kv_lens"][0] += 9
    free = [p for p in range(w["k"].shape[0]) if p not in set(w["table"].ravel().tolist())][:9]
    dst = np.array(free, np.int32).reshape(3, 3)
    acc = np.exp(np.random.default_rng(5).standard_normal((3, H, 140))).astype(np.float32)
    acc[0, :, max_kv:] = 100.0
    d = cache_util.dev(w)
    kept, lens, out = fp8bs.cache_evict(f32_dev(acc), cache_dev(d), d["table"], i32_dev(dst), d["kv_lens"], max_kv,
                                        budget, recent)
    torch.cuda.synchronize()
    rk, rl, ra = oracle.evict(acc, cache_util.cache_of(w), w["table"], dst, w["kv_lens"], budget, recent, max_kv)
    assert np.array_equal(kept.cpu().numpy(), rk) and np.array_equal(lens.cpu().numpy(), rl)
    assert np.array_equal(f32_bits_host(out), ra.view(np.uint32))
    same_cache(d, w, "evict")
