"""Float64 oracle of the norm, the router and the experts of few tokens (tests
only).

Follows the definitions of include/fp8bs_layer.h, one row, token or expert at a
time.  BF16 data are uint16 bit patterns, E4M3 data code bytes.  Nothing is
rounded but the stored sum of the norm (BF16, by definition) and, where a test
asks for them, the codes.
"""

import numpy as np

from . import bf16, e4m3


def norm(x_bits, residual_bits, weight, eps):
    """-> (h bits [M][K], rstd [M], y [M][K]) of the RMS norm; rstd and y float64."""
    h_bits = np.asarray(x_bits, np.uint16)
    if residual_bits is not None:
        h_bits = bf16.from_f64_rne(bf16.to_f32(x_bits).astype(np.float64) + bf16.to_f32(residual_bits).astype(np.float64))
    h = bf16.to_f32(h_bits).astype(np.float64)
    rstd = np.array([1.0 / np.sqrt(np.dot(r, r) / r.size + float(np.float32(eps))) for r in h])
    return h_bits, rstd, h * rstd[:, None] * np.asarray(weight, np.float64)


def tile_scales(y):
    """Unrounded scale of each 1x128 tile, [K/128][M]; 1 for a tile of zeros."""
    m, k = y.shape
    amax = np.abs(y).reshape(m, k // 128, 128).max(2)
    return np.where(amax > 0, np.maximum(amax / 448.0, 2.0 ** -149), 1.0).T


def norm_backward(dy_bits, h_bits, rstd, weight, dh_bits=None):
    """-> (dx [M][K], dweight [K]), float64, rstd taken as given."""
    dy, h = (bf16.to_f32(b).astype(np.float64) for b in (dy_bits, h_bits))
    dx, dw = np.zeros(h.shape), np.zeros(h.shape[1])
    for m in range(h.shape[0]):
        n = h[m] * float(rstd[m])
        g = dy[m] * np.asarray(weight, np.float64)
        dx[m] = float(rstd[m]) * (g - n * np.mean(g * n))
        dw += dy[m] * n
    if dh_bits is not None:
        dx += bf16.to_f32(dh_bits)
    return dx, dw


def _softmax(x):
    """Softmax of the values above -inf; the others get 0 (all: 0)."""
    x = np.asarray(x, np.float64)
    live = x > -np.inf
    p = np.zeros(x.shape)
    if live.any():
        top = x[live].max()
        p[live] = (x[live] == top) if np.isinf(top) else np.exp(x[live] - top)
        p /= p.sum()
    return p


def route(logits, topk, renorm):
    """-> (ids int32 [T][topk], weights float64): a token's largest logits."""
    logits = np.asarray(logits, np.float64)
    ids = np.full((logits.shape[0], topk), -1, np.int32)
    weights = np.zeros(ids.shape)
    for t, x in enumerate(logits):
        order = sorted((e for e in range(x.size) if x[e] > -np.inf), key=lambda e: (-x[e], e))[:topk]
        ids[t, :len(order)] = order
        weights[t, :len(order)] = _softmax(x[order]) if renorm else _softmax(np.where(np.isnan(x), -np.inf, x))[order]
    return ids, weights


def route_backward(logits, ids, dweights, renorm):
    """dlogits float64 [T][E]."""
    logits = np.asarray(logits, np.float64)
    out = np.zeros(logits.shape)
    for t, x in enumerate(logits):
        x = np.where(np.isnan(x), -np.inf, x)
        places = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < x.size and x[ids[t, j]] > -np.inf]
        at, g = ids[t, places], np.asarray(dweights, np.float64)[t, places]
        if renorm:
            w = _softmax(x[at])
            np.add.at(out[t], at, w * (g - np.dot(w, g)))
        else:
            p = _softmax(x)
            total = np.zeros(x.size)
            np.add.at(total, at, g)
            out[t] = p * (total - np.dot(p, total))
    return out


def dequantize_rows(q, s):
    """Codes [M][K] with 1x128 scales [K/128][M] -> float64."""
    return e4m3.decode(q) * np.repeat(np.asarray(s, np.float64).T, 128, 1)


def dequantize_blocks(q, s):
    """Codes [N][K] with 128x128 scales -> float64."""
    return e4m3.decode(q) * np.repeat(np.repeat(np.asarray(s, np.float64), 128, 0), 128, 1)


def experts(x, sx, ids, weights, w13, s13, w2, s2):
    """-> (out [T][H], size [T][H]): the layer's output in float64, and the sum
    of the absolute values of its terms (for error bounds)."""
    xs = dequantize_rows(x, sx)
    T, H = xs.shape
    out, size = np.zeros((T, H)), np.zeros((T, H))
    for e in range(w13.shape[0]):
        tok = sorted({int(t) for t in np.argwhere(ids == e)[:, 0]})
        if not tok:
            continue
        up = xs[tok] @ dequantize_blocks(w13[e], s13[e]).T
        g, u = np.split(up, 2, axis=1)
        share = np.array([np.asarray(weights, np.float64)[t][ids[t] == e].sum() for t in tok])
        with np.errstate(over="ignore"):
            act = share[:, None] * (g / (1 + np.exp(-g))) * u
        wide = dequantize_blocks(w2[e], s2[e])
        out[tok] += act @ wide.T
        size[tok] += np.abs(act) @ np.abs(wide).T
    return out, size
