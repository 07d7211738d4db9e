"""One FP8 attention layer served from the paged FP8 cache.

    python examples/cached_decode.py [--batch 8] [--prompt 1000] [--steps 64]

Prompts of different lengths go through the QKV projection (FP8 GEMM), are
appended to the cache and attended to; then every sequence decodes one token at
a time, while the attention weight of each cached token is summed up.  When the
longest sequence passes the budget, all are cut back to it: the most attended
tokens and the latest ones stay, in fresh pages, and the old pages are freed.
Random weights and activations.  The end prints the time per step and how far the last step is from attention over the unquantized
keys and values of the tokens still cached.
"""

import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_04_amd as fb  # noqa: E402


class PagePool:
    """Free pages of one cache: host bookkeeping only."""

    def __init__(self, pages):
        self.free = list(range(pages))

    def take(self, n):
        if n > len(self.free):
            raise RuntimeError(f"{n} pages asked for, {len(self.free)} free")
        return [self.free.pop() for _ in range(n)]

    def give(self, pages):
        self.free.extend(pages)


class CachedAttention:
    """QKV projection, attention over the cache, output projection."""

    def __init__(self, hidden, q_heads, heads, dim, pages, page, budget, recent, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        draw = lambda n, k: (torch.randn(n, k, generator=g, device=device) * k ** -0.5).to(torch.bfloat16)  # noqa: E731
        self.wqkv = fb.quantize_128x128(draw((q_heads + 2 * heads) * dim, hidden))
        self.wo = fb.quantize_128x128(draw(hidden, q_heads * dim))
        self.q_heads, self.heads, self.dim, self.page = q_heads, heads, dim, page
        self.budget, self.recent, self.device = budget, recent, device
        codes = lambda: torch.zeros(pages, heads, page, dim, dtype=torch.float8_e4m3fn, device=device)  # noqa: E731
        scale = lambda: torch.zeros(pages, heads, device=device)  # noqa: E731
        self.cache = (codes(), scale(), codes(), scale())
        self.pool = PagePool(pages)
        self.pages_of, self.lens, self.sums = [], [], None
        self.scale = 1.0 / math.sqrt(dim)

    def _i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device=self.device)

    def _table(self, rows):
        width = max(1, max(len(r) for r in rows))
        return self._i32([r + [0] * (width - len(r)) for r in rows])

    def _grow(self, new):
        """Pages for `new` more tokens per sequence."""
        for b, n in enumerate(new):
            self.lens[b] += n
            need = -(-self.lens[b] // self.page) - len(self.pages_of[b])
            self.pages_of[b] += self.pool.take(max(0, need))

    def start(self, batch):
        self.pages_of, self.lens, self.sums = [[] for _ in range(batch)], [0] * batch, None

    def forward(self, x, new):
        """x: BF16 [sum(new)][hidden], the rows of all sequences one after the
        other -> BF16 of the same shape."""
        self._grow(new)
        offsets = self._i32([sum(new[:b]) for b in range(len(new) + 1)])
        lens, table, most = self._i32(self.lens), self._table(self.pages_of), max(self.lens)
        q, s = fb.quantize_1x128(x)
        qkv = fb.gemm(q, s, *self.wqkv).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split([self.q_heads, self.heads, self.heads], dim=1)     # views: no copies
        fb.cache_append(k, v, self.cache, table, offsets, lens, max(new))
        out, lse = fb.cache_attention(q, self.cache, table, offsets, lens, max(new), most, self.scale, return_lse=True)
        slots = table.shape[1] * self.page
        if self.sums is not None and self.sums.shape[2] < slots:
            self.sums = torch.nn.functional.pad(self.sums, (0, slots - self.sums.shape[2]))
        self.sums = fb.cache_attention_weights(q, lse, self.cache, table, offsets, lens, max(new), most, self.scale,
                                               self.sums, slots=slots)
        self.last = (q, k, v, out)
        oq, os_ = fb.quantize_1x128(out.view(x.shape[0], -1))
        return fb.gemm(oq, os_, *self.wo)

    def evict(self):
        """Cut every sequence back to the budget if one is past it; -> the kept
        slots, or None."""
        if max(self.lens) <= self.budget:
            return None
        keep = [min(n, self.budget) for n in self.lens]
        fresh = [self.pool.take(-(-n // self.page)) for n in keep]
        kept, _, self.sums = fb.cache_evict(self.sums, self.cache, self._table(self.pages_of), self._table(fresh),
                                            self._i32(self.lens), max(self.lens), self.budget, self.recent)
        for pages in self.pages_of:
            self.pool.give(pages)
        self.pages_of, self.lens = fresh, keep
        return kept


def serve(batch=8, prompt=1000, steps=64, hidden=1024, q_heads=16, heads=4, dim=128, page=64, seed=0):
    """Runs prompts and decoding; -> (time per step in seconds, relative error
    of the last step's attention output, tokens cached at the end)."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    act = lambda n: torch.randn(n, hidden, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    new = [max(1, prompt - b * prompt // (2 * batch)) for b in range(batch)]
    budget = prompt + steps // 2
    pages = batch * 2 * (-(-(budget + steps) // page) + 1)
    layer = CachedAttention(hidden, q_heads, heads, dim, pages, page, budget, budget // 4, seed=seed)
    layer.start(batch)
    layer.forward(act(sum(new)), new)
    # unquantized keys and values per sequence and head, in slot order
    _, k, v, _ = layer.last
    at = [sum(new[:b]) for b in range(batch + 1)]
    keys = [k[at[b]:at[b + 1]].transpose(0, 1).float() for b in range(batch)]
    vals = [v[at[b]:at[b + 1]].transpose(0, 1).float() for b in range(batch)]
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(steps):
        kept = layer.evict()
        if kept is not None:
            for b in range(batch):
                i = kept[b, :, :layer.lens[b]].long()[..., None].expand(-1, -1, dim)
                keys[b], vals[b] = keys[b].gather(1, i), vals[b].gather(1, i)
        layer.forward(act(batch), [1] * batch)
        _, k, v, _ = layer.last
        keys = [torch.cat([keys[b], k[b][:, None].float()], 1) for b in range(batch)]
        vals = [torch.cat([vals[b], v[b][:, None].float()], 1) for b in range(batch)]
    torch.cuda.synchronize()
    took = (time.perf_counter() - began) / steps
    q, _, _, out = layer.last
    off = norm = 0.0
    for b in range(batch):
        for hq in range(q_heads):
            h = hq // (q_heads // heads)
            p = torch.softmax((keys[b][h] @ q[b, hq].float()) * layer.scale, 0)
            want = p @ vals[b][h]
            off += float((out[b, hq].float() - want).square().sum())
            norm += float(want.square().sum())
    return took, math.sqrt(off / norm), list(layer.lens)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    took, err, lens = serve(a.batch, a.prompt, a.steps)
    print(f"{took * 1e6:.0f} us per step of {a.batch} tokens (bookkeeping of the check included); cached {lens}; "
          f"attention output {err:.3f} (relative) from unquantized keys and values")


if __name__ == "__main__":
    main()
