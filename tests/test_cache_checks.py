"""Checks of the cache calls and their binding that need no GPU."""

import ctypes
import importlib.util

import pytest
import torch

from tests.test_cache_abi import DEVICE, F32, FAKE, FLAGS, I32, I64, NO_DEVICE, OK, P, SHAPE, U32, cache, fn


@pytest.fixture(scope="module")
def lib(lib_path):
    return ctypes.CDLL(lib_path)


# A launch holds fewer than 2^32 work-items; a call is launched in runs of
# sequences, so only one sequence's own work is bounded by that.


def test_work_of_one_sequence_append(lib):
    f = fn(lib, "fp8bs_cache_append", [P, P, P, I64, P, I64, I32, U32, P])

    def call(rows, new, **kw):
        return f(cache(page=16, heads=16, table_width=1 << 26, **kw), FAKE, FAKE, 2048, FAKE, rows, new, 0, None)
    assert call(1 << 24, 1 << 24) == SHAPE
    if NO_DEVICE:
        assert call(1 << 22, 1 << 22) == DEVICE
        assert call(1 << 22, 1 << 22, batch=4096) == DEVICE                # more than one launch
        assert call(5, 1 << 24) == DEVICE                                  # max_new far above the rows


def test_work_of_one_sequence_attention(lib):
    f = fn(lib, "fp8bs_cache_attention", [P, P, I64, I32, P, I64, I32, I32, F32, F32, P, I32, P, U32, P, I64, P])

    def call(rows, new, **kw):
        return f(cache(dim=64, **kw), FAKE, 512, 8, FAKE, rows, new, 512, 0.1, 0.0, FAKE, 0, None, 0, FAKE, 1 << 50, None)
    if NO_DEVICE:
        assert call(1 << 27, 1 << 27) == DEVICE
        assert call(1 << 27, 1 << 27, batch=4096) == DEVICE
        assert call(5, 1 << 27) == DEVICE


def test_work_of_one_sequence_weights(lib):
    f = fn(lib, "fp8bs_cache_attention_weights",
           [P, P, I64, I32, P, I64, I32, I32, F32, F32, P, P, P, I64, U32, P, I64, P])

    def call(slots, **kw):
        return f(cache(**kw), FAKE, 4096, 32, FAKE, 5, 1, 512, 0.1, 0.0, FAKE, FAKE, FAKE, slots, 0, None, 0, None)
    assert call(1 << 28, heads=32) == SHAPE
    if NO_DEVICE:
        assert call(1 << 25, heads=32) == DEVICE
        assert call(1 << 25, heads=32, batch=4096) == DEVICE


def test_work_of_one_sequence_evict(lib):
    f = fn(lib, "fp8bs_cache_evict", [P, P, I64, P, I32, I32, I32, I32, P, P, P, P])

    def call(budget, **kw):
        c = cache(page=16, table_width=1 << 26, **kw)
        return f(c, FAKE, 1 << 30, FAKE, 1 << 26, 1 << 30, budget, 0, FAKE, FAKE, 0x20000, None)
    assert call(1 << 26, heads=16) == SHAPE
    assert call(1 << 26, heads=16, batch=0) == SHAPE
    assert call(1 << 20, heads=16, batch=0) == OK
    if NO_DEVICE:
        assert call(1 << 22, heads=16) == DEVICE
        assert call(1 << 22, heads=16, batch=4096) == DEVICE


def test_binding_imports_without_gpu_support_in_torch(lib_path, monkeypatch):
    # host-only calls (tiles, workspace sizes) need no stream
    from fp8_block_scaled_04_amd import fp8bs
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    spec = importlib.util.spec_from_file_location("fp8_block_scaled_04_amd.fp8bs_again", fp8bs.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    pool = (torch.zeros(4, 2, 16, 64, dtype=torch.uint8), None, None, None)
    assert again.cache_attention_workspace_bytes(pool, torch.zeros(1, 2, dtype=torch.int32), 4, 1, 1, 5) == 0


def test_binding_refuses_counts_past_32_bits(lib_path):
    # (2^32 would arrive as 0: every cached token left out)
    from fp8_block_scaled_04_amd import fp8bs
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    codes, scales = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2)
    pool = (codes, scales, codes, scales)
    q, lse, acc = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 4), torch.zeros(1, 2, 8)
    big = 1 << 32
    calls = [lambda: fp8bs.cache_append(q[:, :2], q[:, :2], pool, i32(1, 2), i32(2), i32(1), big),
             lambda: fp8bs.cache_attention_workspace_bytes(pool, i32(1, 2), 4, 1, 1, big),
             lambda: fp8bs.cache_attention_workspace_bytes(pool, i32(1, 2), 4, 1, big + 1, 5),
             lambda: fp8bs.cache_attention(q, pool, i32(1, 2), i32(2), i32(1), 1, big, 0.1),
             lambda: fp8bs.cache_attention_weights_workspace_bytes(pool, i32(1, 2), 4, big + 1, 8),
             lambda: fp8bs.cache_attention_weights(q, lse, pool, i32(1, 2), i32(2), i32(1), 1, big, 0.1),
             lambda: fp8bs.cache_evict(acc, pool, i32(1, 2), i32(1, 2), i32(1), 8, 4, big)]
    for call in calls:
        with pytest.raises(ValueError, match="below 2"):
            call()


def test_caps_whose_reciprocal_or_double_overflows_are_refused(lib):
    # a score of 0 times the reciprocal of a subnormal cap is NaN
    f = fn(lib, "fp8bs_cache_attention", [P, P, I64, I32, P, I64, I32, I32, F32, F32, P, I32, P, U32, P, I64, P])
    g = fn(lib, "fp8bs_cache_attention_weights",
           [P, P, I64, I32, P, I64, I32, I32, F32, F32, P, P, P, I64, U32, P, I64, P])

    def both(cap):
        return (f(cache(), FAKE, 1024, 8, FAKE, 2, 1, 100, 0.1, cap, FAKE, 0, None, 0, None, 0, None),
                g(cache(), FAKE, 1024, 8, FAKE, 2, 1, 512, 0.1, cap, FAKE, FAKE, FAKE, 512, 0, None, 0, None))
    for cap in (1e-40, 2.0 ** -149, 2.0 ** 126.5, 3e38, float("inf"), float("nan"), -1.0):
        assert both(cap) == (FLAGS, FLAGS), cap
    if NO_DEVICE:
        for cap in (0.0, -0.0, 2.0 ** -126, 30.0, 2.0 ** 126):
            assert both(cap) == (DEVICE, DEVICE), cap


def test_attention_tile(lib):
    f = lib.fp8bs_cache_attention_tile
    f.argtypes, f.restype = [P, I32, I64, I32, I32], I32

    def tile(q_heads, rows, new, kv, **kw):
        return f(cache(**kw), q_heads, rows, new, kv)
    assert f(None, 8, 1, 1, 100) == 0
    assert tile(6, 1, 1, 100) == tile(0, 1, 1, 100) == tile(8, -1, 1, 100) == tile(8, 1, 1, -1) == tile(8, 1, 1, 1, page=48) == 0
    # single tokens; few (row, head) pairs; few rows of a sequence
    assert tile(32, 2, 1, 131072) == tile(32, 128, 64, 128) == tile(32, 40000, 8, 131072, heads=8) == 16
    assert tile(32, 8000, 8, 131072, dim=64) == tile(8, 4096, 4096, 1024, dim=64) == 16
    # (eight query heads per key head: 64, 72, 128 and 136 rows)
    assert tile(32, 8000, 8, 4096, dim=64) == 16 and tile(32, 8000, 9, 4096, dim=64) == 128
    assert tile(32, 8000, 8, 4096) == 16 and tile(32, 8000, 8, 4096, batch=16) == 128
    assert tile(32, 8000, 16, 4096) == 128 and tile(32, 8000, 17, 4096) == 256
    assert tile(32, 8000, 4000, 4096) == 256
    from fp8_block_scaled_04_amd import fp8bs
    pool, table = (torch.zeros(4, 8, 16, 128, dtype=torch.uint8),), torch.zeros(2, 6000, dtype=torch.int32)
    assert fp8bs.cache_attention_tile(pool, table, 32, 8000, 4000, 4096) == 256
    with pytest.raises(ValueError):
        fp8bs.cache_attention_tile(pool, table, 30, 8000, 4000, 4096)


def test_attention_workspace_bytes_do_not_overflow(lib):
    # 64 splits of 2^50 (row, query head) pairs: 2^65 bytes
    ws = fn(lib, "fp8bs_cache_attention_workspace", [P, I32, I64, I32, I32, P])
    f = fn(lib, "fp8bs_cache_attention", [P, P, I64, I32, P, I64, I32, I32, F32, F32, P, I32, P, U32, P, I64, P])
    n = I64(-1)
    for lg in range(8, 31):
        status = ws(cache(batch=1, heads=1), 1 << lg, 1 << 30, 1, 1 << 30, ctypes.byref(n))
        if lg <= 10:
            one = (1 << 30 + lg) * 130 * 4
            assert status == OK and n.value % one == 0 and 1 < n.value // one <= 64
        else:
            assert status == SHAPE
            assert f(cache(batch=1, heads=1), FAKE, 128 << lg, 1 << lg, FAKE, 1 << 30, 1, 1 << 30, 0.1, 0.0, FAKE, 0, None,
                     0, FAKE, 1 << 62, None) == SHAPE
