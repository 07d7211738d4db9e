"""Inputs of the norm, router and expert tests: NumPy arrays for the oracle,
copied to the GPU by the helpers of gpu_util."""

import numpy as np

from oracle import bf16, e4m3


def rows_bits(rng, m, k, spread=1.0):
    """BF16 activations, some channels much larger than the rest."""
    x = rng.standard_normal((m, k)) * spread
    x[:, rng.permutation(k)[:max(1, k // 100)]] *= 50
    return bf16.from_f64_rne(x)


def weight_of(rng, k, kind):
    """(values float64, array to give to the GPU): norm weights, BF16 or FP32."""
    w = 1 + 0.3 * rng.standard_normal(k)
    if kind == "fp32":
        w = w.astype(np.float32)
        return w.astype(np.float64), w
    b = bf16.from_f64_rne(w)
    return bf16.to_f32(b).astype(np.float64), b


def expert_case(T, H, I, E, topk, seed=0, pad=0, ids=None):
    """Quantized activations and weights, routing with different experts per
    token; the last `pad` tokens have none."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H))
    x[:, rng.permutation(H)[:max(1, H // 100)]] *= 50
    sx = (np.abs(x).reshape(T, H // 128, 128).max(2) / 448).astype(np.float32).T.copy()
    w = {"x": e4m3.encode((x / np.repeat(sx.T, 128, 1)).astype(np.float32)), "sx": sx}
    for name, n, k in (("w13", 2 * I, H), ("w2", H, I)):
        v = 0.02 * rng.standard_normal((E, n, k)) * np.exp(0.3 * rng.standard_normal((E, n // 128, 1, k // 128, 1))).repeat(
            128, 2).repeat(128, 4).reshape(E, n, k)
        s = (np.abs(v).reshape(E, n // 128, 128, k // 128, 128).max((2, 4)) / 448).astype(np.float32)
        w[name] = e4m3.encode((v / s.repeat(128, 1).repeat(128, 2)).astype(np.float32))
        w["s" + name[1:]] = s
    if ids is None:
        ids = np.stack([rng.permutation(E)[:topk] for _ in range(T)]) if T else np.zeros((0, topk))
    w["ids"] = np.asarray(ids, np.int32).reshape(T, topk).copy()
    w["weights"] = rng.dirichlet(np.ones(topk), T).astype(np.float32).reshape(T, topk)
    if pad:
        w["ids"][T - pad:] = -1
    return w


EXPERT_ARGS = ("x", "sx", "ids", "weights", "w13", "s13", "w2", "s2")


def expert_dev(w):
    from tests.gpu_util import codes_dev, f32_dev, i32_dev
    put = {"x": codes_dev, "w13": codes_dev, "w2": codes_dev, "ids": i32_dev}
    return [put.get(n, f32_dev)(w[n]) for n in EXPERT_ARGS]
