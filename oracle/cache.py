"""Float64 oracle of the paged FP8 key/value cache (tests only).

Follows the definitions of include/fp8bs_cache.h, one sequence, head and token
at a time.  Codes and scales are exact functions of their inputs; attention,
weights and lse are computed in float64.

max_new and max_kv (None: no bound) leave out a sequence's rows and cached tokens
past them, as the end of its table does; results of rows that are left out stay
0 (lse -inf).
"""

import numpy as np

from . import bf16, e4m3

F32 = np.float32


def scale_of(amax, pow2=False):
    """FP32 scale of the largest |x|; 0 for 0."""
    amax = F32(amax)
    if amax == 0:
        return F32(0)
    s = max(F32(amax / F32(448)), F32(2.0 ** -149))
    if pow2:
        m, e = np.frexp(np.float64(s))
        s = F32(np.ldexp(1.0, int(e) - 1 if m == 0.5 else int(e)))
    return s


def encode(x, s):
    """E4M3 codes of FP32 x over an FP32 scale; 0 where the scale is 0."""
    x = np.asarray(x, F32)
    if s == 0:
        return np.zeros(x.shape, np.uint8)
    with np.errstate(under="ignore", over="ignore"):
        return e4m3.encode((x / F32(s)).astype(F32))


def reencode(codes, old, new):
    with np.errstate(under="ignore"):
        return encode((e4m3.decode(codes).astype(F32) * F32(old)).astype(F32), new)


def held(cache, table, kv_len, max_kv=None):
    """Cached tokens of a sequence that a call takes into account."""
    room = table.shape[1] * cache[0].shape[2]
    return max(0, min(int(kv_len), room, room if max_kv is None else max_kv))


def append(cache, k_bits, v_bits, table, q_offsets, kv_lens, pow2=False, max_new=None):
    """cache = (k, ks, v, vs) arrays (uint8 codes, FP32 scales), changed in
    place; k_bits, v_bits: BF16 bits [T][heads][D]."""
    P = cache[0].shape[2]
    for bits, codes, scales in ((k_bits, cache[0], cache[1]), (v_bits, cache[2], cache[3])):
        x = bf16.to_f32(bits)
        for b in range(len(kv_lens)):
            lo, hi = int(q_offsets[b]), int(q_offsets[b + 1])
            base = int(kv_lens[b]) - (hi - lo)
            end = base + (hi - lo if max_new is None else min(hi - lo, max_new))
            slots = np.arange(max(base, 0), min(end, held(cache, table, kv_lens[b])))
            for blk in np.unique(slots // P):
                page = int(table[b][blk])
                if not 0 <= page < codes.shape[0]:
                    continue
                mine = slots[slots // P == blk]
                rows, first = mine % P, int(mine[0] % P)
                for h in range(codes.shape[1]):
                    y = x[lo + mine - base, h]
                    old = scales[page, h] if first else F32(0)
                    new = max(F32(old), scale_of(np.abs(y).max(), pow2))
                    if first and new != old:
                        codes[page, h, :first] = reencode(codes[page, h, :first], old, new)
                    codes[page, h, rows] = encode(y, new)
                    scales[page, h] = new


def values(codes, scales, table, length, h):
    """[length][D] float64 values of one head, and which tokens are present."""
    P, D = codes.shape[2], codes.shape[3]
    out = np.zeros((length, D))
    there = np.zeros(length, bool)
    for t in range(0, length, P):
        page = int(table[t // P])
        n = min(P, length - t)
        if 0 <= page < codes.shape[0]:
            out[t:t + n] = e4m3.decode(codes[page, h, :n]) * np.float64(scales[page, h])
            there[t:t + n] = True
    return out, there


def scores(q, k, there, scale, softcap, base, full):
    """[n][len] scores of one query head (masked: -inf)."""
    x = (q @ k.T) * scale
    if softcap:
        x = softcap * np.tanh(x / softcap)
    seen = np.arange(k.shape[0])[None, :] <= (base + np.arange(q.shape[0]))[:, None]
    if full:
        seen = np.ones_like(seen)
    return np.where(seen & there[None, :], x, -np.inf)


def attention(q_bits, cache, table, q_offsets, kv_lens, scale, softcap=0.0, full=False, max_new=None, max_kv=None):
    """-> out [T][q_heads][D], lse [T][q_heads] in float64."""
    q = bf16.to_f32(q_bits).astype(np.float64)
    T, Hq, D = q.shape
    G = Hq // cache[0].shape[1]
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    for b in range(len(kv_lens)):
        lo, hi, length = int(q_offsets[b]), int(q_offsets[b + 1]), held(cache, table, kv_lens[b], max_kv)
        base = int(kv_lens[b]) - (hi - lo)
        hi = hi if max_new is None else min(hi, lo + max_new)
        for hq in range(Hq):
            k, there = values(cache[0], cache[1], table[b], length, hq // G)
            v, _ = values(cache[2], cache[3], table[b], length, hq // G)
            x = scores(q[lo:hi, hq], k, there, scale, softcap, base, full)
            if x.size == 0:
                continue
            top = x.max(axis=1, keepdims=True)
            top = np.where(np.isinf(top), 0.0, top)
            p = np.exp(x - top)
            total = p.sum(axis=1, keepdims=True)
            out[lo:hi, hq] = (p @ v) / np.where(total > 0, total, 1.0)
            with np.errstate(divide="ignore"):
                lse[lo:hi, hq] = (top + np.log(total))[:, 0]
    return out, lse


def weights(q_bits, lse, cache, table, q_offsets, kv_lens, scale, acc, slots, softcap=0.0, full=False, max_new=None,
            max_kv=None):
    """-> [batch][heads][slots] float64; acc may be None."""
    q = bf16.to_f32(q_bits).astype(np.float64)
    H = cache[0].shape[1]
    G = q.shape[1] // H
    out = np.zeros((len(kv_lens), H, slots))
    for b in range(len(kv_lens)):
        lo, hi, length = int(q_offsets[b]), int(q_offsets[b + 1]), held(cache, table, kv_lens[b], max_kv)
        base = int(kv_lens[b]) - (hi - lo)
        hi = hi if max_new is None else min(hi, lo + max_new)
        old = max(0, min(base, length))
        for h in range(H):
            if acc is not None:
                out[b, h, :old] = acc[b, h, :old]
            k, there = values(cache[0], cache[1], table[b], length, h)
            for hq in range(h * G, (h + 1) * G):
                x = scores(q[lo:hi, hq], k, there, scale, softcap, base, full)
                z = np.asarray(lse[lo:hi, hq], np.float64)[:, None]
                out[b, h, :length] += np.where(np.isneginf(x) | np.isneginf(z), 0.0,
                                               np.exp(x - np.where(np.isinf(z), 0.0, z))).sum(axis=0)
    return out


def evict(acc, cache, table, dst_table, kv_lens, budget, recent, max_kv=None):
    """Changes the cache's destination pages in place; -> kept, new_lens, acc_out."""
    B, H, S = acc.shape
    P = cache[0].shape[2]
    kept = np.full((B, H, budget), -1, np.int32)
    acc_out = np.zeros_like(acc)
    there = [held(cache, table, n, max_kv) for n in kv_lens]
    lens = np.minimum(there, budget).astype(np.int32)
    for b in range(B):
        length, count = there[b], int(lens[b])
        near = min(count, recent)
        for h in range(H):
            a = acc[b, h, :length - near]
            rank = sorted(range(a.size), key=lambda i: (np.isnan(a[i]), -a[i] if not np.isnan(a[i]) else 0.0, i))
            keep = sorted(rank[:count - near]) + list(range(length - near, length))
            kept[b, h, :count] = keep
            acc_out[b, h, :count] = acc[b, h, keep]
            for codes, scales in ((cache[0], cache[1]), (cache[2], cache[3])):
                for j in range(-(-count // P)):
                    to = int(dst_table[b][j])
                    if not 0 <= to < codes.shape[0]:
                        continue
                    src = [(int(table[b][t // P]), t % P) for t in keep[j * P:(j + 1) * P]]
                    src = [(p, r) if 0 <= p < codes.shape[0] else None for p, r in src]
                    new = max([F32(0)] + [scales[s[0], h] for s in src if s])
                    page = np.zeros((P, codes.shape[3]), np.uint8)
                    for i, s in enumerate(src):
                        if s is None:
                            continue
                        c, old = codes[s[0], h, s[1]], scales[s[0], h]
                        page[i] = c if old == new else reencode(c, old, new)
                    codes[to, h] = page
                    scales[to, h] = new
    return kept, lens, acc_out
