"""Performance cases of the norm, the router and the experts of a mixture-of-
experts block.

Five operators of the block between attention and the next layer:

  norm        add the residual, RMS norm, quantize 1x128 (rms_norm_quantize)
  norm_back   its gradients (rms_norm_backward)
  route       the largest router logits of each token and their softmax weights
              (moe_route)
  route_back  its gradient (moe_route_backward)
  experts     gate, up and down products of each token's experts, weighted and
              summed, for few tokens (moe_experts)

Activations are BF16, or E4M3 codes q [M][K] with one FP32 scale per 1x128 tile,
s [K/128][M].  Expert weights are E4M3 codes with one FP32 scale per 128x128
block: w13 [E][2 I][H] (gate rows, then up rows), w2 [E][H][I].

With `own` false, run() computes an operator from elementary torch operations
in FP32; with `own` true it calls this repository's library.
"""

import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


def listed():
    return [
        # One token of one sequence between attention and the experts: latency.
        {"name": "norm_token", "op": "norm", "m": 1, "k": 7168, "residual": True, "y": True, "wt": "bf16"},
        # The rows of a training step; the sum stays for the backward pass.
        {"name": "norm_train", "op": "norm", "m": 8192, "k": 7168, "residual": True, "y": False, "wt": "bf16"},
        # A short ragged batch, a small width, FP32 norm weights.
        {"name": "norm_back_short", "op": "norm_back", "m": 333, "k": 1536, "residual": True, "wt": "fp32"},
        # The backward pass of norm_train.
        {"name": "norm_back_train", "op": "norm_back", "m": 8192, "k": 7168, "residual": True, "wt": "bf16"},
        # A decoding step's tokens.
        {"name": "route_step", "op": "route", "t": 64, "e": 256, "topk": 8, "type": "fp32", "renorm": True},
        # The tokens of a training step, logits in BF16 (many ties).
        {"name": "route_train", "op": "route", "t": 16384, "e": 256, "topk": 8, "type": "bf16", "renorm": True},
        # Gradients of a small router without renormalized weights.
        {"name": "route_back_small", "op": "route_back", "t": 1000, "e": 64, "topk": 6, "type": "fp32", "renorm": False},
        {"name": "route_back_train", "op": "route_back", "t": 16384, "e": 256, "topk": 8, "type": "fp32", "renorm": True},
        # The smallest call: one token, two of eight small experts.
        {"name": "experts_small", "op": "experts", "t": 1, "pad": 0, "e": 8, "topk": 2, "h": 1024, "i": 512},
        # One token, full-size experts.
        {"name": "experts_token", "op": "experts", "t": 1, "pad": 0, "e": 32, "topk": 8, "h": 7168, "i": 2048},
        # A few tokens of a padded batch, many middle-size experts.
        {"name": "experts_few", "op": "experts", "t": 16, "pad": 3, "e": 64, "topk": 6, "h": 2048, "i": 1408},
        # A full decoding batch: every expert has work.
        {"name": "experts_batch", "op": "experts", "t": 64, "pad": 0, "e": 32, "topk": 8, "h": 7168, "i": 2048},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    top = [work(c) for c in listed()]
    max_bytes, max_flops = max(w["bytes"] for w in top), max(w["flops"] for w in top)
    while True:
        op = rng.choice(["norm", "norm_back", "route", "route_back", "experts", "experts"])
        case = {"op": op}
        if op in ("norm", "norm_back"):
            case.update(m=_log_int(rng, 1, 16384), k=128 * _log_int(rng, 2, 64), residual=rng.random() < 0.7,
                        wt=rng.choice(["bf16", "bf16", "fp32"]))
            if op == "norm":
                case["y"] = rng.random() < 0.3
        elif op in ("route", "route_back"):
            case.update(t=_log_int(rng, 1, 16384), e=rng.choice([4, 8, 16, 24, 32, 60, 64, 96, 128, 160, 200, 256]),
                        type=rng.choice(["fp32", "bf16"]), renorm=rng.random() < 0.5)
            case["topk"] = rng.randint(1, min(16, case["e"]))
        else:
            case.update(t=_log_int(rng, 1, 64), e=rng.choice([2, 4, 8, 16, 32, 48, 64, 128]),
                        h=128 * _log_int(rng, 2, 56), i=128 * _log_int(rng, 1, 16))
            case["topk"] = rng.randint(1, min(8, case["e"]))
            case["pad"] = rng.choice([0, 0, rng.randint(0, case["t"] - 1)])
            if case["e"] * case["h"] * case["i"] > 32 * 7168 * 2048:
                continue
        w = work(case)
        if w["bytes"] <= max_bytes and w["flops"] <= max_flops:
            return case


def work(case):
    op = case["op"]
    if op in ("norm", "norm_back"):
        m, k, add = case["m"], case["k"], case["residual"]
        wt = k * (4 if case["wt"] == "fp32" else 2)
        if op == "norm":
            # x (and the residual) in; codes (the sum, the normalized rows) out; scales, 1 / rms
            per = 2 + 1 + (4 if add else 0) + (2 if case["y"] else 0)
            return {"bytes": per * m * k + 4 * m * k // 128 + 4 * m + wt, "flops": 8 * m * k}
        return {"bytes": (6 + (2 if add else 0)) * m * k + 4 * m + wt + 4 * k, "flops": 10 * m * k}
    t, e, topk = case["t"], case["e"], case["topk"]
    if op == "route":
        size = 4 if case["type"] == "fp32" else 2
        return {"bytes": t * e * size + t * topk * 8, "flops": 4 * t * e}
    if op == "route_back":
        size = 4 if case["type"] == "fp32" else 2
        # with renormalized weights only the chosen experts' logits are needed
        read = t * topk if case["renorm"] else t * e
        return {"bytes": read * size + t * e * size + t * topk * 8, "flops": 6 * t * e}
    h, i, real = case["h"], case["i"], case["t"] - case["pad"]
    # experts that get at least one token, where every token's are drawn evenly
    active = e * (1 - (1 - topk / e) ** real)
    per = 3 * h * i * (1 + 4 / 128 ** 2)
    return {"bytes": active * per + real * h * (1 + 4 / 128) + t * topk * 8 + t * h * 2, "flops": 6 * h * i * real * topk}


# ---- inputs ----


def _bf16(x):
    return x.to(torch.bfloat16)


def _rows(gen, m, k):
    """Activations: normal values, one channel in a hundred fifty times larger."""
    x = torch.randn(m, k, generator=gen, device=DEV)
    big = torch.randperm(k, generator=gen, device=DEV)[: max(1, round(0.01 * k))]
    x[:, big] *= 50.0
    return x


def _weights(gen, e, n, k):
    """Expert weights, quantized by 128x128 blocks."""
    q = torch.empty(e, n, k, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty(e, n // 128, k // 128, device=DEV)
    for j in range(e):
        w = 0.02 * torch.randn(n // 128, 128, k // 128, 128, generator=gen, device=DEV)
        s[j] = w.abs().amax((1, 3)) / E4M3_MAX
        q[j] = (w / s[j][:, None, :, None]).view(n, k).to(torch.float8_e4m3fn)
    return q, s


def _logits(gen, case):
    t, e = case["t"], case["e"]
    x = 1.5 * torch.randn(t, e, generator=gen, device=DEV) + 0.3 * torch.randn(e, generator=gen, device=DEV)
    return _bf16(x) if case.get("type") == "bf16" else x


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st, op = {"case": case}, case["op"]
    if op in ("norm", "norm_back"):
        m, k = case["m"], case["k"]
        w = 1.0 + 0.2 * torch.randn(k, generator=gen, device=DEV)
        st["weight"] = w if case["wt"] == "fp32" else _bf16(w)
        st["eps"] = 1e-6
        st["x"] = _bf16(_rows(gen, m, k))
        if op == "norm":
            st["residual"] = _bf16(3.0 * torch.randn(m, k, generator=gen, device=DEV)) if case["residual"] else None
            return st
        st["rstd"] = torch.rsqrt(st["x"].float().square().mean(1) + st["eps"])
        st["dy"] = _bf16(1e-3 * torch.randn(m, k, generator=gen, device=DEV))
        st["dh"] = _bf16(1e-3 * torch.randn(m, k, generator=gen, device=DEV)) if case["residual"] else None
        return st
    if op in ("route", "route_back"):
        st["logits"] = _logits(gen, case)
        if op == "route_back":
            st["ids"] = torch.sort(st["logits"].float(), dim=1, descending=True, stable=True).indices[:, : case["topk"]]
            st["ids"] = st["ids"].to(torch.int32).contiguous()
            st["dweights"] = torch.randn(case["t"], case["topk"], generator=gen, device=DEV)
        return st
    t, e, topk, h, i = case["t"], case["e"], case["topk"], case["h"], case["i"]
    x = _rows(gen, t, h).view(t, h // 128, 128)
    s = x.abs().amax(2) / E4M3_MAX
    st["x"] = (x / s[..., None]).view(t, h).to(torch.float8_e4m3fn)
    st["sx"] = s.t().contiguous()
    logits = torch.randn(t, e, generator=gen, device=DEV)
    top = torch.topk(logits, topk, dim=1)
    st["ids"], st["weights"] = top.indices.to(torch.int32).contiguous(), torch.softmax(top.values, 1).contiguous()
    if case["pad"]:
        # rows that only fill the batch up to the size of a captured graph
        st["ids"][t - case["pad"]:] = -1
        st["weights"][t - case["pad"]:] = 0.0
    st["w13"], st["s13"] = _weights(gen, e, 2 * i, h)
    st["w2"], st["s2"] = _weights(gen, e, h, i)
    return st


# ---- plain forms (FP32) ----


def _plain_norm(st):
    x, eps = st["x"], st["eps"]
    if st["residual"] is not None:
        x = _bf16(x.float() + st["residual"].float())
    v = x.float()
    rstd = 1.0 / torch.sqrt(v.square().mean(1) + eps)
    y = v * rstd[:, None] * st["weight"].float()
    tiles = y.view(y.shape[0], -1, 128)
    amax = tiles.abs().amax(2)
    s = torch.where(amax > 0, (amax / E4M3_MAX).clamp_min(2.0 ** -149), torch.ones_like(amax))
    q = (tiles / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(y.shape)
    out = {"q": q, "s": s.t().contiguous(), "rstd": rstd}
    if st["residual"] is not None:
        out["h"] = x
    if st["case"]["y"]:
        out["y"] = _bf16(y)
    return out


def _plain_norm_back(st):
    dy, h, rstd = st["dy"].float(), st["x"].float(), st["rstd"][:, None]
    n = h * rstd
    g = dy * st["weight"].float()
    dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
    if st["dh"] is not None:
        dx = dx + st["dh"].float()
    return _bf16(dx), (dy * n).sum(0)


def _plain_route(st):
    x, topk = st["logits"].float(), st["case"]["topk"]
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :topk]
    p = torch.exp(x - x.amax(1, keepdim=True))
    w = p.gather(1, ids)
    w = w / (w if st["case"]["renorm"] else p).sum(1, keepdim=True)
    return ids.to(torch.int32), w


def _plain_route_back(st):
    x, ids, g = st["logits"].float(), st["ids"].long(), st["dweights"]
    p = torch.exp(x - x.amax(1, keepdim=True))
    if st["case"]["renorm"]:
        p = torch.zeros_like(p).scatter_(1, ids, p.gather(1, ids))
    p = p / p.sum(1, keepdim=True)
    full = torch.zeros_like(p).scatter_(1, ids, g)
    return (p * (full - (p * full).sum(1, keepdim=True))).to(st["logits"].dtype)


def _blocks(q, s):
    """FP32 values of block-scaled weights [E][N][K]."""
    e, n, k = q.shape
    return (q.view(e, n // 128, 128, k // 128, 128).float() * s[:, :, None, :, None]).view(e, n, k)


def _plain_experts(st):
    t, h = st["x"].shape
    e, i, topk = st["w13"].shape[0], st["w13"].shape[1] // 2, st["ids"].shape[1]
    ids = st["ids"].long()
    there = (ids >= 0) & (ids < e)
    weight = torch.where(there, st["weights"], torch.zeros_like(st["weights"]))
    ids = torch.where(there, ids, torch.zeros_like(ids))
    w13, s13, w2, s2 = st["w13"], st["s13"], st["w2"], st["s2"]
    if t * topk < e:
        # the chosen experts alone, one entry for each choice
        at = ids.reshape(-1)
        w13, s13, w2, s2 = w13[at], s13[at], w2[at], s2[at]
        c = torch.zeros(t, t, topk, device=DEV)
        c[torch.arange(t, device=DEV), torch.arange(t, device=DEV)] = weight
        c = c.view(t, t * topk)
    else:
        c = torch.zeros(t, e, device=DEV).scatter_add_(1, ids, weight)
    x = (st["x"].float().view(t, h // 128, 128) * st["sx"].t()[..., None]).reshape(t, h)
    n = w13.shape[0]
    gu = torch.matmul(_blocks(w13, s13).view(n * 2 * i, h), x.t()).view(n, 2, i, t)
    g, u = gu[:, 0], gu[:, 1]
    a = (g * torch.sigmoid(g) * u * c.t()[:, None, :]).transpose(1, 2).contiguous()
    return _bf16(torch.bmm(a, _blocks(w2, s2).transpose(1, 2)).sum(0))


# ---- one pass ----


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"norm": _plain_norm, "norm_back": _plain_norm_back, "route": _plain_route,
                "route_back": _plain_route_back, "experts": _plain_experts}[op](st)
    import fp8_block_scaled_04_amd as fb

    if op == "norm":
        got = fb.rms_norm_quantize(st["x"], st["weight"], st["eps"], residual=st["residual"], return_y=case["y"])
        out = {"q": got[0], "s": got[1], "rstd": got[3]}
        if case["residual"]:
            out["h"] = got[2]
        if case["y"]:
            out["y"] = got[4]
        return out
    if op == "norm_back":
        return fb.rms_norm_backward(st["dy"], st["x"], st["rstd"], st["weight"], dh=st["dh"])
    if op == "route":
        return fb.moe_route(st["logits"], case["topk"], renormalize=case["renorm"])
    if op == "route_back":
        return fb.moe_route_backward(st["logits"], st["ids"], st["dweights"], renormalize=case["renorm"])
    return fb.moe_experts(st["x"], st["sx"], st["ids"], st["weights"], st["w13"], st["s13"], st["w2"], st["s2"])


# ---- the definitions in 64 bits ----


def _e4m3_64(x):
    """Nearest E4M3 value of float64 numbers up to 448 (ties to even)."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return torch.round(x / step).mul_(step).clamp_(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        m, k = st["x"].shape
        q = torch.empty(m, k, dtype=torch.float64, device=DEV)
        s = torch.empty(k // 128, m, dtype=torch.float64, device=DEV)
        rstd = torch.empty(m, dtype=torch.float64, device=DEV)
        h = torch.empty(m, k, dtype=torch.float64, device=DEV)
        y = torch.empty(m, k, dtype=torch.float64, device=DEV)
        for at in range(0, m, 1024):
            r = slice(at, min(m, at + 1024))
            v = st["x"][r].double()
            if st["residual"] is not None:
                # the stored sum is BF16, and the norm is that of the stored sum
                v = (v + st["residual"][r].double()).to(torch.bfloat16).double()
            rstd[r] = (v.pow(2).sum(1) / k + st["eps"]).pow(-0.5)
            h[r], y[r] = v, torch.einsum("mk,m,k->mk", v, rstd[r], st["weight"].double())
            for j in range(k // 128):
                part = y[r, 128 * j:128 * j + 128]
                s[j, r] = part.abs().max(1).values / E4M3_MAX
                q[r, 128 * j:128 * j + 128] = _e4m3_64(part / s[j, r][:, None])
        out = {"q": q, "s": s, "rstd": rstd}
        if case["residual"]:
            out["h"] = h
        if case["y"]:
            out["y"] = y
        return out
    if op == "norm_back":
        m, k = st["x"].shape
        w = st["weight"].double()
        dx = torch.empty(m, k, dtype=torch.float64, device=DEV)
        dw = torch.zeros(k, dtype=torch.float64, device=DEV)
        for at in range(0, m, 1024):
            r = slice(at, min(m, at + 1024))
            v, d, inv = st["x"][r].double(), st["dy"][r].double(), st["rstd"][r].double()
            dot = (v * d) @ w
            dx[r] = inv[:, None] * d * w - v * (inv.pow(3) * dot / k)[:, None]
            if st["dh"] is not None:
                dx[r] += st["dh"][r].double()
            dw += (v * d).t() @ inv
        return dx, dw
    if op in ("route", "route_back"):
        x = st["logits"].double()
        if op == "route":
            chosen = torch.sort(-x, dim=1, stable=True).indices[:, : case["topk"]]
            lse = torch.logsumexp(x.gather(1, chosen) if case["renorm"] else x, 1, keepdim=True)
            return None, torch.exp(x.gather(1, chosen) - lse)
        ids, g = st["ids"].long(), st["dweights"].double()
        seen = x.gather(1, ids)
        w = torch.exp(seen - torch.logsumexp(seen if case["renorm"] else x, 1, keepdim=True))
        mean = (w * g).sum(1, keepdim=True)
        # d weight_i / d logit_j = weight_i ((i is j) - p_j); p is the softmax over what is normalized
        if case["renorm"]:
            out = torch.zeros_like(x)
        else:
            out = -mean * torch.softmax(x, 1)
        return out.scatter_add(1, ids, w * (g - mean) if case["renorm"] else w * g)
    t, h = st["x"].shape
    e, i = st["w13"].shape[0], case["i"]
    wide = lambda q, s: q.double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)  # noqa: E731
    x = st["x"].double() * st["sx"].t().double().repeat_interleave(128, 1)
    out = torch.zeros(t, h, dtype=torch.float64, device=DEV)
    chosen = st["ids"].cpu()
    for j in range(e):
        tok, place = (chosen == j).nonzero(as_tuple=True)
        if not len(tok):
            continue
        tok, place = tok.to(DEV), place.to(DEV)
        up = x[tok] @ wide(st["w13"][j], st["s13"][j]).t()
        g, u = up[:, :i], up[:, i:]
        a = g / (1 + torch.exp(-g)) * u
        out.index_add_(0, tok, (a @ wide(st["w2"][j], st["s2"][j]).t()) * st["weights"][tok, place].double()[:, None])
    return out
