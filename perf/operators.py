"""Performance cases of the FP8 key/value cache operators.

Four operators of serving a language model with a paged 8-bit cache:

  append    quantize new tokens' keys and values into the cache (cache_append)
  attention attention over the cache, for prompts and single tokens
            (cache_attention)
  weights   the attention weight each cached token received, added to a running
            sum (cache_attention_weights)
  evict     keep each head's most attended tokens and move them to new pages
            (cache_evict)

The cache: E4M3 codes k, v [pages][Hkv][P][D] and one FP32 scale per page and
head, ks, vs [pages][Hkv]; a sequence's slot t lies in page table[b][t // P] at
row t % P.  q_offsets[b] .. q_offsets[b + 1] are sequence b's rows of this call
and kv_lens[b] its cached tokens, this call's included.

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
        # One decoding step of a full serving batch: one new token per sequence.
        {"name": "append_step", "op": "append", "batch": 64, "new": 1, "kv": 4096, "hkv": 8, "d": 128, "page": 64},
        # Prompts of very different lengths written at once, some behind a cached prefix.
        {"name": "append_prompts", "op": "append", "batch": 6, "new": 4000, "kv": 6000, "hkv": 8, "d": 128,
         "page": 128},
        # The smallest call: one request, one token, a short cache of small pages.
        {"name": "attend_one", "op": "attention", "batch": 1, "new": 1, "kv": 777, "hkv": 2, "group": 4, "d": 64,
         "page": 16, "cap": 0.0},
        # An ordinary decoding step: a batch of ragged lengths, grouped heads.
        {"name": "attend_step", "op": "attention", "batch": 48, "new": 1, "kv": 8192, "hkv": 8, "group": 4, "d": 128,
         "page": 64, "cap": 0.0},
        # Two requests with very long contexts: the work has to be split over the cache.
        {"name": "attend_long", "op": "attention", "batch": 2, "new": 1, "kv": 131000, "hkv": 8, "group": 8, "d": 128,
         "page": 128, "cap": 0.0},
        # Several draft tokens verified per sequence, capped scores, one key head per query head.
        {"name": "attend_drafts", "op": "attention", "batch": 16, "new": 5, "kv": 3001, "hkv": 12, "group": 1, "d": 128,
         "page": 32, "cap": 30.0},
        # Fresh prompts, causal: the matrix-bound end.
        {"name": "attend_prompts", "op": "attention", "batch": 2, "new": 6000, "kv": 6000, "hkv": 8, "group": 4,
         "d": 128, "page": 64, "cap": 0.0},
        # A chunk of each prompt behind a long cached prefix, small heads, capped scores.
        {"name": "attend_chunks", "op": "attention", "batch": 4, "new": 513, "kv": 9000, "hkv": 4, "group": 6, "d": 64,
         "page": 64, "cap": 50.0},
        # Bookkeeping of a decoding step: the weight each cached token received.
        {"name": "weights_step", "op": "weights", "batch": 32, "new": 1, "kv": 8192, "hkv": 8, "group": 4, "d": 128,
         "page": 64, "cap": 0.0},
        # The same for a prompt.
        {"name": "weights_prompt", "op": "weights", "batch": 1, "new": 3500, "kv": 4100, "hkv": 8, "group": 4, "d": 128,
         "page": 64, "cap": 0.0},
        # A few short sequences cut back to a small budget.
        {"name": "evict_few", "op": "evict", "batch": 3, "kv": 1100, "budget": 500, "recent": 64, "hkv": 4, "d": 64,
         "page": 16},
        # A batch of long sequences cut back to a quarter.
        {"name": "evict_batch", "op": "evict", "batch": 16, "kv": 16384, "budget": 4096, "recent": 512, "hkv": 8,
         "d": 128, "page": 64},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    top = [work(c) for c in listed()]
    max_bytes, max_flops = max(w["bytes"] for w in top), max(w["flops"] for w in top)
    while True:
        op = rng.choice(["append", "attention", "attention", "weights", "evict"])
        case = {"op": op, "hkv": rng.choice([1, 2, 3, 4, 8, 12, 16]), "d": rng.choice([64, 128]),
                "page": rng.choice([16, 32, 64, 128])}
        if op == "evict":
            case["batch"] = _log_int(rng, 1, 32)
            case["kv"] = _log_int(rng, 200, 16384)
            case["budget"] = max(16, int(case["kv"] * rng.uniform(0.1, 0.9)))
            case["recent"] = int(case["budget"] * rng.uniform(0.0, 0.5))
        else:
            case["batch"] = _log_int(rng, 1, 64)
            step = rng.random() < 0.5
            case["new"] = rng.choice([1, 1, 2, 3, 5, 8]) if step else _log_int(rng, 16, 6000)
            past = _log_int(rng, 1, 131072 if op == "attention" and step else 16384) if step or rng.random() < 0.5 else 0
            case["kv"] = case["new"] + past
        if op in ("attention", "weights"):
            case["group"] = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
            case["cap"] = rng.choice([0.0, 0.0, 30.0, 50.0])
        w = work(case)
        # what the plain form holds at once (its whole score matrix, or the unpacked cache) stays moderate
        scores = case["batch"] * case["hkv"] * case.get("group", 1) * case.get("new", 1) * case["kv"] * 4
        unpacked = case["batch"] * case["hkv"] * case["kv"] * case["d"] * 4
        if w["bytes"] <= max_bytes and w["flops"] <= max_flops and scores <= 10e9 and unpacked <= 5e9:
            return case


# ---- sizes of a case (plain integers, the same for every seed) ----


def _sizes(case):
    """(new tokens, cached tokens) per sequence: the first one has the case's
    sizes, the others fractions of them spread evenly over (0.1, 1)."""
    new, kv = [], []
    for b in range(case["batch"]):
        f = 1.0 if b == 0 else 0.1 + 0.9 * ((b * 0.6180339887) % 1.0)
        n = max(1, int(case.get("new", 0) * f)) if case.get("new", 0) > 16 else case.get("new", 0)
        new.append(n)
        past = case["kv"] - case.get("new", 0)
        kv.append(n + int(past * f) if past else n)
    return new, [max(1, x) for x in kv]


def _pairs(new, kv):
    """Visible (query, slot) pairs of one sequence under the causal rule."""
    return new * (kv - new) + new * (new + 1) // 2


def work(case):
    new, kv = _sizes(case)
    B, H, D, P = case["batch"], case["hkv"], case["d"], case["page"]
    pages = [-(-x // P) for x in kv]
    if case["op"] == "append":
        # BF16 keys and values in, codes out; the scales of the touched pages
        touched = sum(-(-n // P) + 1 for n in new)
        return {"bytes": sum(new) * H * D * 2 * (2 + 1) + touched * H * 16 + 4 * sum(pages), "flops": 6 * sum(new) * H * D}
    if case["op"] == "evict":
        kept = [min(x, case["budget"]) for x in kv]
        cap = max(pages) * P
        # running sums in (all slots) and out, kept codes in and out, indexes, scales
        by = sum(kv) * H * 4 + B * H * cap * 4 + sum(kept) * H * D * 4 + B * H * case["budget"] * 4
        return {"bytes": by + sum(pages) * H * 8 + sum(-(-x // P) for x in kept) * H * 8, "flops": 4 * sum(kept) * H * D}
    Hq = H * case["group"]
    pairs = sum(_pairs(n, x) for n, x in zip(new, kv)) * Hq
    rows = sum(new) * Hq
    if case["op"] == "attention":
        by = sum(kv) * H * D * 2 + sum(pages) * (H * 8 + 4) + rows * (D * 4 + 4)
        return {"bytes": by, "flops": 4 * D * pairs}
    cap = max(pages) * P
    by = sum(kv) * H * D + sum(pages) * (H * 4 + 4) + rows * (D * 2 + 4) + sum(kv) * H * 4 + B * H * cap * 4
    return {"bytes": by, "flops": 2 * D * pairs}


# ---- inputs ----


def _fill(gen, pages, H, P, D, spread):
    """Codes and scales of a filled cache: BF16-sized normal values, a few
    channels much larger than the rest, each page quantized by its largest."""
    x = torch.randn(pages, H, P, D, generator=gen, device=DEV)
    x *= torch.exp(spread * torch.randn(H, 1, D, generator=gen, device=DEV))
    s = (x.abs().amax(dim=(2, 3)) / E4M3_MAX).clamp_min(2.0 ** -100)
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def _table(gen, pages, first, width):
    """Block table: the sequences' pages scattered over the pool."""
    total = sum(pages)
    order = torch.randperm(total, generator=gen, device=DEV).to(torch.int32) + first
    rows, at = [], 0
    for n in pages:
        rows.append(torch.nn.functional.pad(order[at:at + n], (0, width - n)))
        at += n
    return torch.stack(rows).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    new, kv = _sizes(case)
    B, H, D, P = case["batch"], case["hkv"], case["d"], case["page"]
    pages = [-(-x // P) for x in kv]
    width = max(pages)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    st = {"case": case, "kv_lens": i32(kv), "max_kv": max(kv), "max_new": max(new), "page": P}
    st["q_offsets"] = i32([sum(new[:b]) for b in range(B + 1)])
    T = sum(new)
    if case["op"] == "evict":
        kept = [-(-min(x, case["budget"]) // P) for x in kv]
        total = sum(pages) + sum(kept)
        st["k"], st["ks"] = _fill(gen, total, H, P, D, 0.5)
        st["v"], st["vs"] = _fill(gen, total, H, P, D, 0.2)
        st["table"] = _table(gen, pages, 0, width)
        st["dst_table"] = _table(gen, kept, sum(pages), max(kept))
        # few tokens hold most of the weight; many were hardly ever attended
        acc = torch.exp(2.5 * torch.randn(B, H, width * P, generator=gen, device=DEV))
        acc = torch.where(torch.rand(acc.shape, generator=gen, device=DEV) < 0.05, torch.zeros_like(acc), acc)
        st["acc"] = acc
        return st
    st["k"], st["ks"] = _fill(gen, sum(pages), H, P, D, 0.5)
    st["v"], st["vs"] = _fill(gen, sum(pages), H, P, D, 0.2)
    st["table"] = _table(gen, pages, 0, width)
    if case["op"] == "append":
        # new tokens of varying size: some fit the scale of the page they go to, some do not
        size = torch.exp(0.7 * torch.randn(T, 1, 1, generator=gen, device=DEV))
        st["k_new"] = (torch.randn(T, H, D, generator=gen, device=DEV) * size).to(torch.bfloat16)
        st["v_new"] = (torch.randn(T, H, D, generator=gen, device=DEV) * size).to(torch.bfloat16)
        return st
    Hq = H * case["group"]
    st["q"] = torch.randn(T, Hq, D, generator=gen, device=DEV).to(torch.bfloat16)
    st["scale"] = 1.0 / math.sqrt(D)
    if case["op"] == "weights":
        st["lse"] = _plain_attention(st)[1]
        st["acc"] = torch.rand(B, H, width * P, generator=gen, device=DEV)
    return st


# ---- plain forms (FP32) ----


def _unpack(codes, scales, table, P, lens):
    """[B][H][slots][D] FP32 values of the cache, zero past each length."""
    B, W = table.shape
    pg = table.long()
    x = codes[pg].float() * scales[pg][..., None, None]              # [B][W][H][P][D]
    x = x.transpose(1, 2).reshape(B, x.shape[2], W * P, x.shape[4])
    live = torch.arange(W * P, device=x.device)[None, :] < lens[:, None]
    return torch.where(live[:, None, :, None], x, torch.zeros((), device=x.device))


def _rows(st):
    """Row numbers of the packed queries per sequence [B][max_new], and which exist."""
    off = st["q_offsets"].long()
    i = torch.arange(st["max_new"], device=off.device)
    n = off[1:] - off[:-1]
    there = i[None, :] < n[:, None]
    return (off[:-1, None] + i[None, :]).clamp_max(st["q"].shape[0] - 1), there, n


def _scores(st, rows, there, n):
    """Capped and masked scores [B][Hkv][group * max_new][slots], FP32."""
    case = st["case"]
    H, G, D, P = case["hkv"], case["group"], case["d"], st["page"]
    k = _unpack(st["k"], st["ks"], st["table"], P, st["kv_lens"])
    B, L, N = k.shape[0], k.shape[2], rows.shape[1]
    q = st["q"][rows].float().view(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    s = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    pos = (st["kv_lens"].long() - n)[:, None] + torch.arange(N, device=q.device)[None, :]
    seen = (torch.arange(L, device=q.device)[None, None, :] <= pos[:, :, None]) & there[:, :, None]
    seen = seen[:, None, None].expand(B, 1, G, N, L).reshape(B, 1, G * N, L)
    return s.masked_fill_(~seen, float("-inf"))


def _pack(x, st, there):
    """[B][H][G * N][...] -> the packed rows [T][Hq][...]."""
    case = st["case"]
    B, H, N, G = x.shape[0], case["hkv"], there.shape[1], case["group"]
    x = x.reshape(B, H, G, N, -1).permute(0, 3, 1, 2, 4).reshape(B, N, H * G, -1)
    T = st["q"].shape[0]
    off = st["q_offsets"].long()
    t = torch.arange(T, device=x.device)
    b = torch.searchsorted(off[1:], t, right=True)
    return x[b, t - off[b]]


def _plain_attention(st):
    rows, there, n = _rows(st)
    s = _scores(st, rows, there, n)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    s = s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    v = _unpack(st["v"], st["vs"], st["table"], st["page"], st["kv_lens"])
    o = torch.matmul(s, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = top + torch.log(total)
    return _pack(o, st, there).to(torch.bfloat16), _pack(lse, st, there)[..., 0]


def _plain_weights(st):
    rows, there, n = _rows(st)
    s = _scores(st, rows, there, n)
    case = st["case"]
    B, H, G, N = s.shape[0], case["hkv"], case["group"], rows.shape[1]
    lse = st["lse"][rows].view(B, N, H, G).permute(0, 2, 3, 1).reshape(B, H, G * N, 1)
    w = s.sub_(lse).exp_().sum(2)
    slot = torch.arange(w.shape[2], device=w.device)[None, :]
    old = slot < (st["kv_lens"].long() - n)[:, None]
    return w + torch.where(old[:, None], st["acc"], torch.zeros_like(w))


def _block_scale(amax):
    return torch.where(amax > 0, (amax / E4M3_MAX).clamp_min(2.0 ** -149), torch.zeros_like(amax))


def _encode(x, s):
    """E4M3 codes of x / s; zero where the scale is zero."""
    y = torch.where(s > 0, x / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x))
    return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _plain_append(st):
    P = st["page"]
    off, lens, table = st["q_offsets"].long(), st["kv_lens"].long(), st["table"].long()
    n = off[1:] - off[:-1]
    B = n.numel()
    t = torch.arange(st["k_new"].shape[0], device=off.device)
    b = torch.searchsorted(off[1:], t, right=True)
    slot = lens[b] - n[b] + t - off[b]
    page, row = table[b, slot // P], slot % P
    start = lens - n                                               # first new slot per sequence
    first = table[torch.arange(B, device=off.device), (start // P).clamp_max(table.shape[1] - 1)]
    older = torch.arange(P, device=off.device)[None, :] < (start % P)[:, None]
    older = older & (n > 0)[:, None]                               # rows that stay, in each first page
    out = []
    for x, codes, scales in ((st["k_new"], st["k"], st["ks"]), (st["v_new"], st["v"], st["vs"])):
        x = x.float()
        amax = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(-1), "amax")
        touched = torch.zeros(scales.shape[0], dtype=torch.bool, device=x.device).index_fill_(0, page, True)
        kept = torch.zeros_like(scales)
        kept[first] = torch.where(older.any(1)[:, None], scales[first], torch.zeros_like(scales[first]))
        s = torch.maximum(kept, _block_scale(amax))
        held, s_old, s_new = codes[first], scales[first][..., None, None], s[first][..., None, None]
        again = _encode(held.float() * s_old, s_new.expand(held.shape))
        change = older[:, None, :, None] & (s_old != s_new)
        codes.view(torch.uint8)[first] = torch.where(change, again.view(torch.uint8), held.view(torch.uint8))
        codes.view(torch.uint8)[page, :, row] = _encode(x, s[page][..., None].expand(x.shape)).view(torch.uint8)
        scales.copy_(torch.where(touched[:, None], s, scales))
        out += [codes, scales]
    return tuple(out)


def _plain_evict(st):
    case, P = st["case"], st["page"]
    acc, lens = st["acc"], st["kv_lens"].long()
    B, H, S = acc.shape
    budget, D = case["budget"], case["d"]
    slot = torch.arange(S, device=acc.device)
    count = lens.clamp_max(budget)
    recent = count.clamp_max(case["recent"])
    key = torch.where((slot >= (lens - recent)[:, None])[:, None], torch.full_like(acc, float("inf")), acc)
    key = torch.where((slot < lens[:, None])[:, None], key, torch.full_like(acc, float("-inf")))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    if budget > S:
        order = torch.nn.functional.pad(order, (0, budget - S))
    live = (torch.arange(budget, device=acc.device) < count[:, None])[:, None]
    kept = torch.sort(torch.where(live, order, torch.full_like(order, S)), dim=-1).values
    live = live.expand(B, H, budget)
    src = torch.where(live, kept, torch.zeros_like(kept))
    acc_out = torch.zeros_like(acc)
    m = min(budget, S)
    acc_out[..., :m] = torch.where(live, acc.gather(-1, src), torch.zeros_like(acc[..., :1]))[..., :m]
    # move the codes, one scale per destination page: the largest of its tokens' scales
    table, dst = st["table"].long(), st["dst_table"].long()
    blocks = dst.shape[1]
    pad = blocks * P - budget
    if pad >= 0:
        src, live = torch.nn.functional.pad(src, (0, pad)), torch.nn.functional.pad(live, (0, pad))
    else:
        src, live = src[..., :pad], live[..., :pad]
    page = torch.gather(table[:, None].expand(B, H, -1), 2, src // P)
    head = torch.arange(H, device=acc.device)[None, :, None]
    there = live.view(B, H, blocks, P)
    used = there[..., 0].all(1)                                       # destination pages that hold tokens, [B][blocks]
    out = []
    for codes, scales in ((st["k"], st["ks"]), (st["v"], st["vs"])):
        held = codes[page, head, src % P]
        s_old = torch.where(live, scales[page, head], torch.zeros_like(scales[page, head]))
        s_new = s_old.view(B, H, blocks, P).amax(-1)
        s_tok = s_new[..., None].expand(B, H, blocks, P).reshape(B, H, -1)
        moved = _encode(held.float() * s_old[..., None], s_tok[..., None].expand(held.shape))
        moved = torch.where((s_old != s_tok)[..., None], moved.view(torch.uint8), held.view(torch.uint8))
        moved = torch.where(live[..., None], moved, torch.zeros_like(moved))
        moved = moved.view(B, H, blocks, P, D).transpose(1, 2).reshape(B * blocks, H, P, D)
        to, use = dst.reshape(-1), used.reshape(-1)
        # pages that receive nothing go to where the first page goes, with its contents
        first = to[0]
        to = torch.where(use, to, first)
        moved = torch.where(use[:, None, None, None], moved, moved[:1])
        flat = s_new.transpose(1, 2).reshape(B * blocks, H)
        flat = torch.where(use[:, None], flat, flat[:1])
        codes.view(torch.uint8)[to] = moved
        scales[to] = flat
        out += [codes, scales]
    kept = torch.where(live[..., :budget] if pad >= 0 else torch.nn.functional.pad(live, (0, -pad)), kept,
                       torch.full_like(kept, -1)).to(torch.int32)
    return kept, count.to(torch.int32), acc_out, tuple(out)


# ---- one pass ----


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"append": _plain_append, "attention": _plain_attention, "weights": _plain_weights,
                "evict": _plain_evict}[op](st)
    import fp8_block_scaled_04_amd as fb

    cache = (st["k"], st["ks"], st["v"], st["vs"])
    if op == "append":
        fb.cache_append(st["k_new"], st["v_new"], cache, st["table"], st["q_offsets"], st["kv_lens"], st["max_new"])
        return cache
    if op == "attention":
        return fb.cache_attention(st["q"], cache, st["table"], st["q_offsets"], st["kv_lens"], st["max_new"],
                                  st["max_kv"], st["scale"], softcap=st["case"]["cap"], return_lse=True)
    if op == "weights":
        return fb.cache_attention_weights(st["q"], st["lse"], cache, st["table"], st["q_offsets"], st["kv_lens"],
                                          st["max_new"], st["max_kv"], st["scale"], st["acc"],
                                          softcap=st["case"]["cap"])
    kept, lens, acc = fb.cache_evict(st["acc"], cache, st["table"], st["dst_table"], st["kv_lens"], st["max_kv"],
                                     st["case"]["budget"], st["case"]["recent"])
    return kept, lens, acc, cache


# ---- the definitions in 64 bits ----


def _exact_rows(st, b, head):
    """Sequence b, one key head: scores [group][n][len] (masked: -inf) and the page list."""
    case, P = st["case"], st["page"]
    G, D = case["group"], case["d"]
    lo, hi = int(st["q_offsets"][b]), int(st["q_offsets"][b + 1])
    length, n = int(st["kv_lens"][b]), hi - lo
    pg = st["table"][b, : -(-length // P)].long()
    k = (st["k"][pg, head].double() * st["ks"][pg, head].double()[:, None, None]).reshape(-1, D)[:length]
    q = st["q"][lo:hi, head * G:(head + 1) * G].double().permute(1, 0, 2).reshape(-1, D)
    s = (q @ k.t()).mul_(st["scale"])
    if case["cap"]:
        s = s.div_(case["cap"]).tanh_().mul_(case["cap"])
    s = s.view(G, n, length)
    hide = torch.ones(n, length, dtype=torch.bool, device=s.device).triu_(length - n + 1)
    return s.masked_fill_(hide, float("-inf")), pg, lo, hi, length, n


def _e4m3_64(x):
    """Nearest E4M3 value of float64 numbers up to 448 (ties to even)."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return torch.round(x / step).mul_(step).clamp_(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    st = prepare(case, seed)
    op, H, D, P = case["op"], case["hkv"], case["d"], case["page"]
    B = case["batch"]
    if op == "attention":
        T, G = st["q"].shape[0], case["group"]
        out = torch.empty(T, H * G, D, dtype=torch.float64, device=DEV)
        lse = torch.empty(T, H * G, dtype=torch.float64, device=DEV)
        for b in range(B):
            for h in range(H):
                s, pg, lo, hi, length, n = _exact_rows(st, b, h)
                v = (st["v"][pg, h].double() * st["vs"][pg, h].double()[:, None, None]).reshape(-1, D)[:length]
                z = torch.logsumexp(s, -1)
                p = s.sub_(z[..., None]).exp_()
                out[lo:hi, h * G:(h + 1) * G] = torch.matmul(p.view(-1, length), v).view(G, n, D).transpose(0, 1)
                lse[lo:hi, h * G:(h + 1) * G] = z.t()
        return out, lse
    if op == "weights":
        acc, G = torch.zeros_like(st["acc"], dtype=torch.float64), case["group"]
        for b in range(B):
            for h in range(H):
                s, pg, lo, hi, length, n = _exact_rows(st, b, h)
                z = st["lse"][lo:hi, h * G:(h + 1) * G].double().t()
                acc[b, h, :length] = s.sub_(z[..., None]).exp_().sum((0, 1))
                acc[b, h, :length - n] += st["acc"][b, h, :length - n].double()
        return acc
    if op == "append":
        got = []
        for new, codes, scales in (("k_new", "k", "ks"), ("v_new", "v", "vs")):
            x, c, s = st[new].double(), st[codes].double(), st[scales].double()
            for b in range(B):
                lo, hi, length = int(st["q_offsets"][b]), int(st["q_offsets"][b + 1]), int(st["kv_lens"][b])
                at = length - (hi - lo)
                while lo < hi:
                    page, row = int(st["table"][b, at // P]), at % P
                    n = min(hi - lo, P - row)
                    piece = x[lo:lo + n].transpose(0, 1)                     # [H][n][D]
                    want = piece.abs().amax((1, 2)) / E4M3_MAX
                    if row:
                        want = torch.maximum(want, s[page])
                        grown = (want > s[page])[:, None, None]
                        again = _e4m3_64(c[page, :, :row] * (s[page] / want)[:, None, None])
                        c[page, :, :row] = torch.where(grown, again, c[page, :, :row])
                    s[page] = want
                    c[page, :, row:row + n] = _e4m3_64(piece / want[:, None, None])
                    lo, at = lo + n, at + n
            got += [c, s]
        return tuple(got)
    # evict: the indexes and counts are whole numbers; the rest are sums, scales and codes that move
    acc = torch.zeros_like(st["acc"], dtype=torch.float64)
    pools = [st["k"].double(), st["ks"].double(), st["v"].double(), st["vs"].double()]
    for b in range(B):
        length = int(st["kv_lens"][b])
        count = min(length, case["budget"])
        recent = min(count, case["recent"])
        a = st["acc"][b, :, : length - recent].double()
        best = torch.sort(-a, dim=1, stable=True).indices[:, : count - recent]
        last = torch.arange(length - recent, length, device=DEV).expand(H, -1)
        keep = torch.sort(torch.cat([best, last], 1), 1).values             # [H][count]
        acc[b, :, :count] = st["acc"][b].double().gather(1, keep)
        pg, row = st["table"][b].long()[keep // P], keep % P
        head = torch.arange(H, device=DEV)[:, None]
        blocks = -(-count // P)
        to = st["dst_table"][b, :blocks].long()
        for ci, si, codes, scales in ((0, 1, st["k"], st["ks"]), (2, 3, st["v"], st["vs"])):
            s = torch.zeros(H, blocks * P, dtype=torch.float64, device=DEV)
            c = torch.zeros(H, blocks * P, D, dtype=torch.float64, device=DEV)
            s[:, :count] = scales[pg, head].double()
            c[:, :count] = codes[pg, head, row].double()
            top = s.view(H, blocks, P).amax(-1)
            c = _e4m3_64(c * (s.view(H, blocks, P) / top[..., None]).reshape(H, -1, 1))
            pools[ci][to] = c.view(H, blocks, P, D).transpose(0, 1)
            pools[si][to] = top.t()
    return None, None, acc, tuple(pools)
