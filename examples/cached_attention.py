"""One attention layer served over packed rows: the token vectors come from an
INT8 embedding table by the pooled lookup, the keys and values live in a paged
cache of INT8 rows, and the cache is cut when a sequence outgrows its budget.

    python examples/cached_attention.py

For a few ragged prompts: lookup -> projection -> norm + rotation + append ->
prompt attention; then one token at a time: lookup -> projection -> norm +
rotation + append -> attention over the pages (adding each key's weight to the
running mass) -> eviction.  Before the first eviction the outputs are compared
with plain torch attention over the same keys and values held in fp32.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import int4_row_wise_amd as q  # noqa: E402

VOCAB, WIDTH = 5000, 512
Q_HEADS, KV_HEADS, DIM = 8, 2, 64
PAGE, BITS = 16, 8
BUDGET, KEEP, SINKS, RECENT = 160, 96, 4, 32
DEV = "cuda"


class Cache:
    """Pages of packed rows, and which of them each sequence owns (host lists)."""

    def __init__(self, batch: int, pages: int):
        shape = (pages, KV_HEADS, PAGE, q.row_stride(DIM, BITS))
        self.k = torch.zeros(shape, dtype=torch.uint8, device=DEV)
        self.v = torch.zeros(shape, dtype=torch.uint8, device=DEV)
        self.free = list(range(pages))
        self.owned = [[] for _ in range(batch)]
        self.lens = [0] * batch

    def grow(self, b: int, n: int) -> list:
        """Makes room for n more rows of sequence b: their flat slots."""
        first, self.lens[b] = self.lens[b], self.lens[b] + n
        while len(self.owned[b]) * PAGE < self.lens[b]:
            self.owned[b].append(self.free.pop())
        return [self.owned[b][s // PAGE] * PAGE + s % PAGE for s in range(first, self.lens[b])]

    def table(self, owned=None) -> torch.Tensor:
        owned = self.owned if owned is None else owned
        width = max(len(o) for o in owned)
        return torch.tensor([o + [0] * (width - len(o)) for o in owned], dtype=torch.int32, device=DEV)

    def seq_lens(self) -> torch.Tensor:
        return torch.tensor(self.lens, dtype=torch.int32, device=DEV)

    def cut(self, mass: torch.Tensor) -> torch.Tensor:
        """Evicts down to KEEP rows a head into fresh pages; the rows' mass."""
        fresh = [[self.free.pop() for _ in range(-(-KEEP // PAGE))] for _ in self.owned]
        new_mass = torch.zeros_like(mass)
        q.evict(self.k, self.v, self.table(), self.seq_lens(), mass, KEEP, self.k, self.v, self.table(fresh),
                sinks=SINKS, recent=RECENT, new_mass=new_mass)
        for b, old in enumerate(self.owned):
            self.free += old
            self.owned[b], self.lens[b] = fresh[b], min(self.lens[b], KEEP)
        return new_mass


def plain_attention(x, k, v):
    """x [Hq, d] over k, v [n, Hkv, d], in fp32."""
    g = Q_HEADS // KV_HEADS
    k, v = k.float().repeat_interleave(g, 1), v.float().repeat_interleave(g, 1)
    w = torch.softmax((k * x.float()).sum(-1) * DIM ** -0.5, 0)
    return (w[..., None] * v).sum(0)


def main(prompts=(37, 5, 90), steps: int = 100, seed: int = 0, verbose: bool = True) -> dict:
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rows = q.quantize_rowwise(torch.randn((VOCAB, WIDTH), generator=g, device=DEV) * 0.05, BITS)
    w_qkv = (torch.randn((WIDTH, (Q_HEADS + 2 * KV_HEADS) * DIM), generator=g, device=DEV) * 0.5).bfloat16()
    w_out = torch.randn((Q_HEADS * DIM, VOCAB), generator=g, device=DEV).bfloat16()
    gain_q, gain_k = ((1 + 0.1 * torch.randn(DIM, generator=g, device=DEV)).bfloat16() for _ in range(2))
    places = torch.arange(4096, device=DEV)[:, None] * 10000.0 ** (-torch.arange(0, DIM, 2, device=DEV) / DIM)
    cos_sin = torch.cat((places.cos(), places.sin()), 1).contiguous()
    table_offsets = torch.tensor([0, VOCAB], device=DEV)

    def project(ids: torch.Tensor):
        """Token ids -> strided q, k, v [n, heads, dim] of one fused projection."""
        n = ids.numel()
        x = q.bag_forward(rows, table_offsets, n, WIDTH, BITS, ids, torch.arange(n + 1, device=DEV))[:, 0]
        t = (x.bfloat16() @ w_qkv).view(n, -1, DIM)
        return t.split((Q_HEADS, KV_HEADS, KV_HEADS), 1)

    batch = len(prompts)
    cache = Cache(batch, pages=2 * batch * (-(-(BUDGET + 1) // PAGE) + 1))
    plain_k, plain_v = [[] for _ in prompts], [[] for _ in prompts]
    errors = {"prompt": 0.0, "step": 0.0}

    def append(ids, positions, slots):
        xq, xk, xv = project(ids)
        k_out = torch.empty((ids.numel(), KV_HEADS, DIM), dtype=xq.dtype, device=DEV)
        xq, _ = q.norm_rope(xq, xk, positions, cos_sin, gain_q, gain_k, v=xv, k_pages=cache.k, v_pages=cache.v,
                            slots=torch.tensor(slots, device=DEV), bits=BITS, k_out=k_out)
        return xq, k_out, xv

    def off(got, want):
        return float((got.float() - want).norm() / want.norm())

    # prompts, all at once
    ids = torch.randint(0, VOCAB, (sum(prompts),), generator=g, device=DEV)
    slots = [s for b, n in enumerate(prompts) for s in cache.grow(b, n)]
    positions = torch.cat([torch.arange(n, device=DEV) for n in prompts])
    xq, xk, xv = append(ids, positions, slots)
    offsets = torch.tensor([sum(prompts[:i]) for i in range(batch + 1)], dtype=torch.int32, device=DEV)
    out = q.prompt_attention(xq, xk, xv, offsets, offsets, max_q=max(prompts))
    last = []
    for b, (lo, hi) in enumerate(zip(offsets.tolist(), offsets.tolist()[1:])):
        plain_k[b].append(xk[lo:hi])
        plain_v[b].append(xv[lo:hi])
        errors["prompt"] = max(errors["prompt"], off(out[hi - 1], plain_attention(xq[hi - 1], xk[lo:hi], xv[lo:hi])))
        last.append(hi - 1)
    out = out[last]

    # one token at a time
    mass = torch.zeros((batch, KV_HEADS, BUDGET + 1), device=DEV)
    place, cuts = list(prompts), 0
    for step in range(steps):
        ids = (out.reshape(batch, -1) @ w_out).argmax(-1)
        slots = [cache.grow(b, 1)[0] for b in range(batch)]
        xq, xk, xv = append(ids, torch.tensor(place, device=DEV), slots)
        place = [p + 1 for p in place]
        out = q.decode_attention(xq, cache.k, cache.v, cache.table(), cache.seq_lens(), bits=BITS, mass=mass)
        if not cuts:
            for b in range(batch):
                plain_k[b].append(xk[b:b + 1])
                plain_v[b].append(xv[b:b + 1])
                errors["step"] = max(errors["step"], off(out[b], plain_attention(xq[b], torch.cat(plain_k[b]), torch.cat(plain_v[b]))))
        if max(cache.lens) >= BUDGET:
            mass = cache.cut(mass)
            cuts += 1
    torch.cuda.synchronize()
    row, plain = q.row_stride(DIM, BITS), 2 * DIM
    if verbose:
        print("prompt attention: relative error %.2g; steps over INT8 rows: %.2g" % (errors["prompt"], errors["step"]))
        print("%d tokens, %d evictions, caches now of %s rows a head; a row takes %d bytes instead of %d" % (
            sum(place), cuts, cache.lens, row, plain))
    return {"errors": errors, "cuts": cuts, "lens": cache.lens, "mass": float(mass.sum()), "finite": bool(torch.isfinite(out).all())}


if __name__ == "__main__":
    main()
