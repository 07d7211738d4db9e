"""Calls of the paged FP8 cache at the edges of what the header allows."""

import numpy as np
import pytest
import torch

from fp8_block_scaled_04_amd import fp8bs
from oracle import cache as oracle
from tests import cache_util
from tests.gpu_util import f32_dev, i32_dev, out_host_f64, require_gpu
from tests.test_gpu_cache import BOUND, abs_values, cache_dev, score_error

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_gpu()


@pytest.mark.parametrize("H,P", [(1, 128), (64, 16)])
def test_evict_updates_lengths_in_place(H, P):
    # new_lens is the cache's kv_lens: every head still sees the old lengths
    kv, budget, recent = [3000, 700, 1, 0, 2500, 1999], 600, 50
    w = cache_util.make(kv, [0] * 6, H, 1, 64, P, seed=H, spare=6 * -(-budget // P))
    free = [p for p in range(w["k"].shape[0]) if p not in set(w["table"].ravel().tolist())]
    width = -(-budget // P)
    dst = i32_dev(np.array(free[:6 * width]).reshape(6, width))
    acc = f32_dev(np.random.default_rng(H).random((6, H, 3000)))
    d, e = cache_util.dev(w), cache_util.dev(w)
    print(f"evict in place H={H} P={P}", flush=True)
    want = fp8bs.cache_evict(acc, cache_dev(d), d["table"], dst, d["kv_lens"], 3000, budget, recent)
    kept, out = torch.empty_like(want[0]), torch.empty_like(want[2])
    c, dev = fp8bs._cache_args(cache_dev(e), e["table"], e["kv_lens"])
    assert fp8bs._cevict(c, acc.data_ptr(), 3000, dst.data_ptr(), width, 3000, budget, recent, kept.data_ptr(),
                         e["kv_lens"].data_ptr(), out.data_ptr(), fp8bs._stream_of(dev)) == 0
    torch.cuda.synchronize()
    assert e["kv_lens"].tolist() == [600, 600, 1, 0, 600, 600] == want[1].tolist()
    assert torch.equal(kept, want[0]) and torch.equal(out, want[2])
    for n in ("k", "v"):
        assert torch.equal(e[n].view(torch.uint8), d[n].view(torch.uint8))
        assert torch.equal(e[n + "s"].view(torch.int32), d[n + "s"].view(torch.int32))


def test_evict_of_empty_sequences():
    w = cache_util.make([0, 0], [0, 0], 2, 1, 64, 16)
    d = cache_util.dev(w)
    before = d["k"].view(torch.uint8).clone()
    for max_kv in (0, 20):
        print(f"evict of empty sequences max_kv={max_kv}", flush=True)
        kept, lens, out = fp8bs.cache_evict(torch.ones(2, 2, max_kv, device="cuda"), cache_dev(d), d["table"], d["table"],
                                            d["kv_lens"], max_kv, 5, 2)
        torch.cuda.synchronize()
        assert (kept == -1).all() and lens.tolist() == [0, 0] and (out == 0).all()
        assert torch.equal(d["k"].view(torch.uint8), before)


# A launch holds fewer than 2^32 work-items; these calls need more.


def pool(pages, H, D, P):
    return (torch.zeros((pages, H, P, D), dtype=torch.float8_e4m3fn, device="cuda"),
            torch.zeros((pages, H), device="cuda"),
            torch.zeros((pages, H, P, D), dtype=torch.float8_e4m3fn, device="cuda"),
            torch.zeros((pages, H), device="cuda"))


def offsets(new):
    return i32_dev(np.concatenate([[0], np.cumsum(new)]))


def bits_of(t):
    return t.contiguous().view(torch.uint8)


def test_append_of_a_long_prompt_among_many_sequences():
    # 256 sequences of 16 heads, pages of 16: 2^26 workgroups of 256 by max_new
    B, H, D, P, long = 256, 16, 64, 16, 131072
    new = [1 + b % 3 for b in range(B)]
    new[200] = long
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(sum(new), H, D, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.full((B, long // P), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = torch.arange(B, dtype=torch.int32)
    table[200] = B + torch.arange(long // P, dtype=torch.int32)
    lens, off = i32_dev(new), offsets(new)
    got, want = pool(B + long // P, H, D, P), pool(B + long // P, H, D, P)
    print("append, one call", flush=True)
    fp8bs.cache_append(x, -x, got, table, off, lens, long)
    print("append, three calls", flush=True)
    for lo, hi, most in ((0, 200, 3), (200, 201, long), (201, 256, 3)):
        fp8bs.cache_append(x, -x, want, table[lo:hi], off[lo:hi + 1], lens[lo:hi], most)
    torch.cuda.synchronize()
    assert float(got[1].min(1)[0][table[table >= 0].long()].min()) > 0
    for a, b in zip(got, want):
        assert torch.equal(bits_of(a), bits_of(b))


@pytest.mark.parametrize("D,H,G", [(128, 2, 8), (64, 2, 8)])
def test_attention_and_weights_of_very_many_row_tiles(D, H, G):
    # 4096 sequences of 32 tokens, max_new the rows of the whole call
    B, n, P = 4096, 32, 32
    g = torch.Generator(device="cuda").manual_seed(D)
    k = torch.randn(B * n, H, D, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(B * n, H * G, D, generator=g, device="cuda").to(torch.bfloat16)
    cache = pool(B, H, D, P)
    table, lens, off = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous(), i32_dev([n] * B), offsets([n] * B)
    fp8bs.cache_append(k, -k, cache, table, off, lens, n)
    print(f"attention D={D}, one call", flush=True)
    out, lse = fp8bs.cache_attention(q, cache, table, off, lens, B * n, n, 0.1, return_lse=True)
    print(f"weights D={D}, one call", flush=True)
    acc = fp8bs.cache_attention_weights(q, lse, cache, table, off, lens, B * n, n, 0.1)
    torch.cuda.synchronize()
    for b in (0, 1, 1023, 1024, 2047, 2048, 2049, 4094):
        print(f"sequences {b}, {b + 1}", flush=True)
        rows = slice(b * n, (b + 2) * n)
        # the same kernels: a bound far above the rows, and of the cached tokens as above
        o, z = fp8bs.cache_attention(q[rows], cache, table[b:b + 2], off[:3], lens[:2], 4 * n, n, 0.1, return_lse=True)
        a = fp8bs.cache_attention_weights(q[rows], z, cache, table[b:b + 2], off[:3], lens[:2], 4 * n, n, 0.1)
        torch.cuda.synchronize()
        e = (out[rows].float() - o.float()).abs().max() / o.float().abs().max()
        assert float(e) < 2.0 ** -6 and torch.allclose(lse[rows], z, rtol=0, atol=2.0 ** -12)
        assert torch.allclose(acc[b:b + 2], a, rtol=2.0 ** -10, atol=1e-6)


def test_weights_over_very_many_slots():
    # 2048 sequences, 4 heads, 2^19 + 256 slots of sums: 2^32 of them and more
    B, H, D, P, slots = 2048, 4, 64, 16, (1 << 19) + 256
    n = 20
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn(B * n, H, D, generator=g, device="cuda").to(torch.bfloat16)
    cache = pool(2 * B, H, D, P)
    table, lens, off = torch.arange(2 * B, dtype=torch.int32, device="cuda").view(B, 2), i32_dev([n] * B), offsets([n] * B)
    fp8bs.cache_append(k, k, cache, table, off, lens, n)
    ones = offsets([1] * B)
    q = torch.randn(B, H, D, generator=g, device="cuda").to(torch.bfloat16)
    _, lse = fp8bs.cache_attention(q, cache, table, ones, lens, 1, n, 0.1, return_lse=True)
    small = fp8bs.cache_attention_weights(q, lse, cache, table, ones, lens, 1, n, 0.1)
    out = torch.full((B, H, slots), 5.0, device="cuda")
    print("weights, one call", flush=True)
    fp8bs.cache_attention_weights(q, lse, cache, table, ones, lens, 1, n, 0.1, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out[:, :, :n], small)
    assert all(int(torch.count_nonzero(out[b:b + 64, :, n:])) == 0 for b in range(0, B, 64))


def test_evict_to_very_many_pages():
    # 1024 sequences, 8 heads, a budget of 16400 tokens in pages of 16
    B, H, D, P, budget, kv = 1024, 8, 64, 16, 16400, 40
    width = -(-budget // P)
    g = torch.Generator(device="cuda").manual_seed(4)
    k = torch.randn(B * kv, H, D, generator=g, device="cuda").to(torch.bfloat16)
    cache = pool(6 * B, H, D, P)
    table, lens = torch.arange(3 * B, dtype=torch.int32, device="cuda").view(B, 3), i32_dev([kv] * B)
    fp8bs.cache_append(k, -k, cache, table, offsets([kv] * B), lens, kv)
    dst = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    dst[:, :3] = 3 * B + table
    acc = torch.rand(B, H, budget, generator=g, device="cuda")
    print("evict, one call", flush=True)
    kept, new, out = fp8bs.cache_evict(acc, cache, table, dst, lens, budget, budget, 5)
    torch.cuda.synchronize()
    assert (new == kv).all() and torch.equal(out[:, :, :kv], acc[:, :, :kv]) and (out[:, :, kv:] == 0).all()
    assert (kept[:, :, :kv] == torch.arange(kv, dtype=torch.int32, device="cuda")).all() and (kept[:, :, kv:] == -1).all()
    for a in (cache[1], cache[3]):
        assert torch.equal(a[3 * B:], a[:3 * B])
    used = (torch.arange(3 * P, device="cuda") < kv).view(3, 1, P, 1)
    for a in (cache[0], cache[2]):
        x = bits_of(a).view(2, B, 3, H, P, D)
        assert torch.equal(x[1], torch.where(used, x[0], torch.zeros_like(x[0])))


# FP32 outputs: the weights meet the codes as two BF16 parts on every kernel.  A
# part is rounded to nearest, so 2^-18 of a weight is lost (2^-17 taken, doubled
# for the sum it is divided by); scores as in tests/test_gpu_cache.py.
FP32_SHAPES = [  # cached tokens, rows, heads, group, D, P, max_new, max_kv
    ([30] * 12, [30] * 12, 2, 8, 128, 32, 30, BOUND),                          # 256-row tiles
    ([30] * 12, [30] * 12, 2, 4, 128, 32, 30, BOUND),                          # 128-row tiles
    ([30] * 12, [30] * 12, 2, 8, 64, 16, 30, BOUND),                           # 128-row tiles of D = 64
    ([700, 513, 260, 129], [150, 64, 33, 129], 1, 16, 128, 64, 150, 1400),     # splits
    ([700, 513, 260, 129], [150, 64, 33, 129], 1, 16, 64, 64, 150, 6000),
    ([300, 128, 129, 90] * 10, [7] * 40, 1, 16, 128, 16, 7, 300),
    ([250, 200], [250, 200], 2, 40, 64, 64, 250, 250),
    ([1, 15, 40], [1, 1, 2], 2, 3, 128, 16, 2, 40),                            # 16-row tiles
]


@pytest.mark.parametrize("kv,new,H,G,D,P,max_new,max_kv", FP32_SHAPES)
def test_fp32_outputs_keep_two_part_weights(kv, new, H, G, D, P, max_new, max_kv):
    w = cache_util.make(kv, new, H, G, D, P, seed=H + G + D)
    d = cache_util.dev(w)
    for cap, full in ((0.0, False), (3.0, False), (0.0, True)):
        print(f"FP32 outputs H={H} G={G} D={D} P={P} cap={cap} full={full}", flush=True)
        out = fp8bs.cache_attention(d["q"], cache_dev(d), d["table"], d["q_offsets"], d["kv_lens"], max_new, max_kv,
                                    D ** -0.5, softcap=cap, full=full, out_dtype=torch.float32)
        torch.cuda.synchronize()
        args = (w["table"], w["q_offsets"], w["kv_lens"], D ** -0.5, cap, full)
        ref, _ = oracle.attention(w["q"], cache_util.cache_of(w), *args)
        size, _ = oracle.attention(w["q"], abs_values(w), *args)
        tol = (2 * score_error(w, D ** -0.5, cap) + 2.0 ** -16) * size + 1e-30
        bad = np.abs(out_host_f64(out) - ref) > tol
        assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.max(np.abs(out_host_f64(out) - ref) / tol):.3g}"
