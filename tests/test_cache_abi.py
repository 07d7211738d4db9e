"""Argument checks of the cache calls (include/fp8bs_cache.h) without a GPU:
the documented status comes back before the HIP runtime is touched."""

import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8bs_cache.h")
OK, NULL, SHAPE, ALIGN, FLAGS, DEVICE, LAUNCH = range(7)
P = ctypes.c_void_p
I64, I32, U32, F32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_float
FAKE, MIS, ODD = 0x10000, 0x10008, 0x10002


class Cache(ctypes.Structure):
    _fields_ = [("k", P), ("ks", P), ("v", P), ("vs", P), ("table", P), ("kv_lens", P), ("pages", I64), ("batch", I32),
                ("table_width", I32), ("heads", I32), ("page", I32), ("dim", I32)]


def cache(**kw):
    d = dict(k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, table=FAKE, kv_lens=FAKE, pages=10, batch=2, table_width=8, heads=4,
             page=64, dim=128)
    d.update(kw)
    return ctypes.byref(Cache(**d))


def _no_device():
    import torch
    return torch.cuda.device_count() == 0


NO_DEVICE = _no_device()
BAD_CACHES = [dict(pages=0), dict(batch=-1), dict(table_width=0), dict(heads=0), dict(page=48), dict(page=256),
              dict(dim=96), dict(dim=256), dict(table_width=1 << 25)]


@pytest.fixture(scope="module")
def lib(lib_path):
    return ctypes.CDLL(lib_path)


def fn(lib, name, args):
    f = getattr(lib, name)
    f.argtypes = args
    f.restype = ctypes.c_int
    return f


def test_every_declared_symbol_is_exported(lib):
    names = sorted(set(re.findall(r"^fp8bs_status (fp8bs_\w+)\s*\(", open(HEADER).read(), re.M)))
    assert len(names) == 6, names
    for n in names:
        assert hasattr(lib, n), n


def test_append(lib):
    f = fn(lib, "fp8bs_cache_append", [P, P, P, I64, P, I64, I32, U32, P])
    good = dict(k=FAKE, v=FAKE, ld=512, off=FAKE, rows=5, new=3, flags=0)

    def call(c=None, **kw):
        d = dict(good, **kw)
        return f(c if c is not None else cache(), d["k"], d["v"], d["ld"], d["off"], d["rows"], d["new"], d["flags"], None)
    for bad in BAD_CACHES:
        assert call(cache(**bad)) == SHAPE, bad
    assert f(None, FAKE, FAKE, 512, FAKE, 5, 3, 0, None) == NULL
    assert call(ld=504) == SHAPE and call(ld=516) == SHAPE and call(rows=-1) == SHAPE and call(new=-1) == SHAPE
    assert call(flags=2) == FLAGS
    assert call(rows=0, k=None) == OK and call(new=0) == OK and call(cache(batch=0, table=None)) == OK
    assert call(k=None) == NULL and call(off=None) == NULL and call(cache(vs=None)) == NULL
    assert call(v=MIS) == ALIGN and call(off=ODD) == ALIGN and call(cache(k=MIS)) == ALIGN and call(cache(table=ODD)) == ALIGN
    if NO_DEVICE:
        assert call() == DEVICE and call(ld=520, flags=1) == DEVICE


def test_attention(lib):
    f = fn(lib, "fp8bs_cache_attention", [P, P, I64, I32, P, I64, I32, I32, F32, F32, P, I32, P, U32, P, I64, P])
    ws = fn(lib, "fp8bs_cache_attention_workspace", [P, I32, I64, I32, I32, P])
    need = I64(-1)
    assert ws(cache(), 8, 2, 1, 512, ctypes.byref(need)) == OK
    splits = need.value // (2 * 8 * 130 * 4)
    assert need.value == splits * 2 * 8 * 130 * 4 and splits > 1
    good = dict(q=FAKE, ld=1024, hq=8, off=FAKE, rows=2, new=1, kv=512, scale=0.1, cap=0.0, out=FAKE, dt=0, lse=FAKE,
                flags=0, ws=FAKE, n=need.value)

    def call(c=None, **kw):
        d = dict(good, **kw)
        return f(c if c is not None else cache(), *[d[x] for x in ("q", "ld", "hq", "off", "rows", "new", "kv", "scale", "cap", "out", "dt", "lse",
                                                                  "flags", "ws", "n")], None)
    for bad in BAD_CACHES:
        assert call(cache(**bad)) == SHAPE, bad
    for bad in (dict(hq=6, ld=1024), dict(hq=0), dict(ld=1016), dict(ld=1028), dict(kv=-1), dict(rows=-1), dict(new=-2),
                dict(n=need.value - 1), dict(new=1 << 28)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(dt=2), dict(flags=1), dict(flags=4), dict(scale=float("inf")), dict(scale=float("nan")),
                dict(cap=-1.0), dict(cap=float("nan"))):
        assert call(**bad) == FLAGS, bad
    assert call(rows=0, n=0) == OK and call(cache(batch=0), n=0) == OK
    assert call(q=None) == NULL and call(out=None) == NULL and call(ws=None) == NULL and call(cache(kv_lens=None)) == NULL
    assert call(q=MIS) == ALIGN and call(out=MIS) == ALIGN and call(lse=ODD) == ALIGN and call(ws=MIS) == ALIGN
    assert ws(cache(), 8, 2, 1, 512, None) == NULL and ws(cache(), 6, 2, 1, 512, ctypes.byref(need)) == SHAPE
    assert ws(None, 8, 2, 1, 512, ctypes.byref(need)) == NULL
    if NO_DEVICE:
        assert call() == DEVICE and call(lse=None, dt=1, flags=2, cap=30.0) == DEVICE
        assert call(kv=100, n=0, ws=None) == DEVICE                 # one split: no workspace


def test_attention_workspace_covers_every_size(lib):
    # the workspace is a whole number of partial results, at most 64 splits,
    # and none where the cached tokens are not split
    ws = fn(lib, "fp8bs_cache_attention_workspace", [P, I32, I64, I32, I32, P])
    for dim in (64, 128):
        for hq in (4, 12, 64):
            for new in (1, 5, 33, 400, 5000):
                for kv in (0, 1, 127, 129, 5000, 1 << 20):
                    n = I64(-1)
                    assert ws(cache(dim=dim, table_width=1 << 14), hq, 2 * new, new, kv, ctypes.byref(n)) == OK
                    one = 2 * new * hq * (dim + 2) * 4
                    assert n.value % one == 0 and n.value // one <= 64 and n.value // one != 1


def test_attention_weights(lib):
    f = fn(lib, "fp8bs_cache_attention_weights",
           [P, P, I64, I32, P, I64, I32, I32, F32, F32, P, P, P, I64, U32, P, I64, P])
    ws = fn(lib, "fp8bs_cache_attention_weights_workspace", [P, I32, I32, I64, P])
    good = dict(q=FAKE, ld=1024, hq=8, off=FAKE, rows=2, new=1, kv=512, scale=0.1, cap=0.0, lse=FAKE, inp=FAKE, out=FAKE,
                slots=512, flags=0, ws=None, n=0)

    def call(c=None, **kw):
        d = dict(good, **kw)
        return f(c if c is not None else cache(), *[d[x] for x in ("q", "ld", "hq", "off", "rows", "new", "kv", "scale", "cap", "lse", "inp", "out",
                                                                  "slots", "flags", "ws", "n")], None)
    for bad in BAD_CACHES:
        assert call(cache(**bad)) == SHAPE, bad
    assert call(slots=511) == SHAPE and call(hq=7, ld=1024) == SHAPE and call(ld=8) == SHAPE
    assert call(flags=1) == FLAGS and call(cap=-2.0) == FLAGS and call(scale=float("nan")) == FLAGS
    assert call(kv=0, slots=0) == OK and call(cache(batch=0)) == OK
    assert call(lse=None) == NULL and call(out=None) == NULL and call(off=None) == NULL and call(cache(k=None)) == NULL
    assert call(q=MIS) == ALIGN and call(inp=ODD) == ALIGN
    need = I64(-1)
    assert ws(cache(), 8, 1, 512, ctypes.byref(need)) == OK and need.value == 0
    assert ws(cache(), 8, 4000, 4096, ctypes.byref(need)) == OK and need.value > 0
    assert call(new=4000, slots=4096, n=need.value - 1, ws=FAKE) == SHAPE
    assert call(new=4000, slots=4096, n=need.value) == NULL
    assert call(new=4000, slots=4096, n=need.value, ws=MIS) == ALIGN
    assert ws(cache(), 8, 1, 512, None) == NULL and ws(cache(), 8, 1, -1, ctypes.byref(need)) == SHAPE
    if NO_DEVICE:
        assert call() == DEVICE and call(inp=None) == DEVICE and call(cache(v=None, vs=None)) == DEVICE
        assert call(rows=0, q=None, lse=None) == DEVICE             # the sums are still written


def test_evict(lib):
    f = fn(lib, "fp8bs_cache_evict", [P, P, I64, P, I32, I32, I32, I32, P, P, P, P])
    good = dict(acc=FAKE, slots=512, dst=FAKE, width=4, kv=512, budget=256, recent=16, kept=FAKE, lens=FAKE, out=0x20000)

    def call(c=None, **kw):
        d = dict(good, **kw)
        return f(c if c is not None else cache(), *[d[x] for x in ("acc", "slots", "dst", "width", "kv", "budget", "recent", "kept", "lens", "out")],
                 None)
    for bad in BAD_CACHES:
        assert call(cache(**bad)) == SHAPE, bad
    for bad in (dict(slots=511), dict(width=3), dict(budget=0), dict(budget=-3), dict(recent=-1), dict(width=-1),
                dict(out=FAKE), dict(kv=-1)):
        assert call(**bad) == SHAPE, bad
    assert call(cache(batch=0)) == OK
    for n in ("acc", "dst", "kept", "lens", "out"):
        assert call(**{n: None}) == NULL, n
    assert call(kept=ODD) == ALIGN and call(cache(ks=ODD)) == ALIGN
    if NO_DEVICE:
        assert call() == DEVICE and call(budget=1000, width=8, recent=5000) == DEVICE
