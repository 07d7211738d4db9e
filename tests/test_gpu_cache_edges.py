"""Calls of the paged FP8 cache at the edges of what the header allows."""

import numpy as np
import pytest
import torch

from fp8_block_scaled_04_amd import fp8bs
from tests import cache_util
from tests.gpu_util import f32_dev, i32_dev, require_gpu
from tests.test_gpu_cache import cache_dev

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
