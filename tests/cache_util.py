"""Cases of the paged FP8 cache: NumPy arrays for the oracle, copied to the
GPU by dev()."""

import numpy as np

from oracle import bf16, e4m3


def bits(x):
    return bf16.from_f64_rne(x)


def make(kv, new, H=2, G=2, D=64, P=16, seed=0, spare=2, table_extra=2):
    """Sequences with kv[b] cached tokens, the last new[b] of them rows of this
    call.  Rows of the pages past the cached tokens hold the NaN code, unused
    pages a NaN scale, table entries past the end -7."""
    rng = np.random.default_rng(seed)
    B = len(kv)
    need = [-(-t // P) for t in kv]
    pages = max(1, sum(need) + spare)
    order = rng.permutation(pages)[:sum(need)]
    width = max(need + [0]) + table_extra
    table = np.full((B, width), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    w = {"P": P, "D": D, "H": H, "G": G, "table": table, "kv_lens": np.array(kv, np.int32),
         "q_offsets": np.concatenate([[0], np.cumsum(new)]).astype(np.int32), "max_new": max(list(new) + [0]),
         "max_kv": max(list(kv) + [0])}
    for name, spread in (("k", 0.5), ("v", 0.2)):
        x = rng.standard_normal((pages, H, P, D)) * np.exp(spread * rng.standard_normal((1, H, 1, D)))
        s = (np.abs(x).max(axis=(2, 3)) / 448).astype(np.float32)
        c = e4m3.encode((x / s[:, :, None, None]).astype(np.float32))
        scale = np.full((pages, H), np.nan, np.float32)
        codes = np.full(c.shape, 0x7F, np.uint8)
        for b in range(B):
            for j in range(need[b]):
                p, n = table[b, j], min(P, kv[b] - j * P)
                scale[p] = s[p]
                codes[p, :, :n] = c[p, :, :n]
        w[name], w[name + "s"] = codes, scale
    T = int(sum(new))
    w["q"] = bits(rng.standard_normal((T, H * G, D)))
    size = np.exp(0.8 * rng.standard_normal((T, 1, 1)))
    w["k_new"] = bits(rng.standard_normal((T, H, D)) * size)
    w["v_new"] = bits(rng.standard_normal((T, H, D)) * size)
    return w


def cache_of(w):
    return w["k"], w["ks"], w["v"], w["vs"]


def dev(w):
    """The same case as GPU tensors."""
    import torch
    from tests.gpu_util import bf16_dev, codes_dev, f32_dev, i32_dev
    d = dict(w)
    for n in ("k", "v"):
        d[n] = codes_dev(w[n])
        d[n + "s"] = f32_dev(w[n + "s"])
        d[n + "_new"] = bf16_dev(w[n + "_new"])
    d["q"] = bf16_dev(w["q"])
    for n in ("table", "kv_lens", "q_offsets"):
        d[n] = i32_dev(w[n])
    torch.cuda.synchronize()
    return d
