"""Pins of the cache oracle against torch in float64 and closed forms (CPU)."""

import numpy as np
import torch

from oracle import bf16, cache as oracle, e4m3
from tests import cache_util


def gathered(w, b, h, which):
    """[len][D] values of one head, page by page."""
    n, P = int(w["kv_lens"][b]), w["P"]
    rows = [e4m3.decode(w[which][w["table"][b, t // P], h, t % P]) * np.float64(w[which + "s"][w["table"][b, t // P], h])
            for t in range(n)]
    return torch.tensor(np.array(rows).reshape(n, w["D"]))


def test_attention_and_weights_match_torch_float64():
    w = cache_util.make([40, 3, 70], [5, 3, 1], 2, 3, 64, 16, seed=1)
    q = torch.tensor(bf16.to_f32(w["q"]).astype(np.float64))
    for cap, full in ((0.0, False), (2.0, False), (0.0, True)):
        args = (w["table"], w["q_offsets"], w["kv_lens"], 0.2, cap, full)
        out, lse = oracle.attention(w["q"], cache_util.cache_of(w), *args)
        acc = np.ones((3, 2, 75), np.float32)
        total = oracle.weights(w["q"], lse, cache_util.cache_of(w), w["table"], w["q_offsets"], w["kv_lens"], 0.2, acc, 75,
                               cap, full)
        for b, (lo, hi) in enumerate([(0, 5), (5, 8), (8, 9)]):
            n = int(w["kv_lens"][b])
            want = np.zeros((2, n))
            for hq in range(6):
                x = q[lo:hi, hq] @ gathered(w, b, hq // 3, "k").T * 0.2
                if cap:
                    x = cap * torch.tanh(x / cap)
                if not full:
                    x = x.masked_fill(torch.ones_like(x).triu(n - (hi - lo) + 1).bool(), -torch.inf)
                p = torch.softmax(x, -1)
                assert np.allclose(out[lo:hi, hq], (p @ gathered(w, b, hq // 3, "v")).numpy(), rtol=1e-12, atol=1e-13)
                assert np.allclose(lse[lo:hi, hq], torch.logsumexp(x, -1).numpy(), rtol=1e-13)
                want[hq // 3] += p.sum(0).numpy()
            want[:, : n - (hi - lo)] += 1
            assert np.allclose(total[b, :, :n], want, rtol=1e-12) and (total[b, :, n:] == 0).all()


def test_empty_rows():
    w = cache_util.make([2, 0], [4, 1], 1, 1, 64, 16)
    out, lse = oracle.attention(w["q"], cache_util.cache_of(w), w["table"], w["q_offsets"], w["kv_lens"], 1.0)
    assert (out[[0, 1, 4]] == 0).all() and np.isneginf(lse[[0, 1, 4]]).all() and np.isfinite(lse[2:4]).all()


def test_append_quantizes_a_fresh_page_like_one_block():
    w = cache_util.make([32], [32], 2, 1, 64, 16, seed=2)
    oracle.append(cache_util.cache_of(w), w["k_new"], w["v_new"], w["table"], w["q_offsets"], w["kv_lens"])
    x = bf16.to_f32(w["k_new"])
    for j in range(2):
        for h in range(2):
            y = torch.tensor(x[16 * j:16 * j + 16, h])
            s = y.abs().max() / 448
            want = (y / s).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            page = w["table"][0, j]
            assert w["ks"][page, h] == s.numpy() and np.array_equal(w["k"][page, h], want)


def test_append_scale_only_grows_and_older_codes_follow():
    w = cache_util.make([2], [1], 1, 1, 64, 16, seed=3)
    page = w["table"][0, 0]
    w["ks"][page, 0], w["k"][page, 0, 0] = 1.0, e4m3.encode(np.full(64, 96.0, np.float32))
    for size, scale, older in ((448.0, 1.0, 96.0), (896.0, 2.0, 48.0), (10.0, 2.0, 48.0)):
        w["k_new"] = cache_util.bits(np.full((1, 1, 64), size))
        oracle.append(cache_util.cache_of(w), w["k_new"], w["v_new"], w["table"], w["q_offsets"], w["kv_lens"])
        assert w["ks"][page, 0] == scale and (e4m3.decode(w["k"][page, 0, 0]) == older).all()
        assert (e4m3.decode(w["k"][page, 0, 1]) == min(size, 448 * scale) / scale).all()
    assert oracle.scale_of(0) == 0 and oracle.scale_of(448 * 3, True) == 4 and oracle.scale_of(448 * 4, True) == 4


def test_evict_keeps_recent_and_heaviest_in_order():
    w = cache_util.make([40], [0], 1, 1, 64, 16, seed=4)
    free = [p for p in range(w["k"].shape[0]) if p not in w["table"]]
    acc = np.zeros((1, 1, 40), np.float32)
    acc[0, 0, [3, 30, 17]] = [5, 9, 5]
    acc[0, 0, 8] = np.nan
    before = gathered(w, 0, 0, "v").numpy()
    kept, lens, out = oracle.evict(acc, cache_util.cache_of(w), w["table"], np.array([free[:1]], np.int32), [40], 8, 2)
    assert kept[0, 0].tolist() == [0, 1, 2, 3, 17, 30, 38, 39] and lens.tolist() == [8]
    assert out[0, 0, :8].tolist() == [0, 0, 0, 5, 5, 9, 0, 0] and (out[0, 0, 8:] == 0).all()
    s = w["vs"][free[0], 0]
    moved = e4m3.decode(w["v"][free[0], 0]) * np.float64(s)
    # half a code step of the new scale for values that were encoded again
    step = np.maximum(2.0 ** -4 * np.abs(before[kept[0, 0]]), 2.0 ** -10 * s)
    assert (np.abs(moved[:8] - before[kept[0, 0]]) <= step).all() and (moved[8:] == 0).all()
    assert s == max(w["vs"][w["table"][0, t // 16], 0] for t in kept[0, 0])
