"""Operators of a serving loop beside the paged cache, as measured cases: rotation by several axes with the append,
attention of a batch that shares prefixes, the residual's addition with a norm, and log probabilities of tokens.

Each case names one operator and its sizes; `prepare` makes what a serving program holds before the call, `run`
makes one call, in plain torch operations or (where `own` is set) through the package's entry points, and `exact`
computes the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one decoding step of 64 sequences whose prompts held images: three axes in blocks; launch latency counts
        dict(name="axes step", op="axes", tokens=64, hq=32, hkv=8, d=128, rot=128, axes=3, turns="blocks", pairs="half", dtype="bf16", norm=True, bits=16, page=16),
        # a prompt of 16384 tokens, most of them a video's patches: axes in turn, appended to 16-bit pages; streaming
        dict(name="axes video prompt", op="axes", tokens=16384, hq=32, hkv=8, d=128, rot=128, axes=3, turns="one by one", pairs="half", dtype="bf16", norm=True, bits=16, page=16),
        # an image encoder's heads: two axes, rotation alone, an odd number of patches, no cache
        dict(name="axes image encoder", op="axes", tokens=8191, hq=16, hkv=16, d=64, rot=64, axes=2, turns="blocks", pairs="neighbours", dtype="fp16", norm=False, bits=0, page=16),
        # four answers to one short prompt: few rows, latency counts
        dict(name="shared few", op="shared", batch=4, groups=1, prefix=2048, own_len=128, hq=32, hkv=8, d=128, dtype="bf16", bits=16, page=16),
        # 64 answers to one long document
        dict(name="shared batch", op="shared", batch=64, groups=1, prefix=32768, own_len=1024, hq=32, hkv=8, d=128, dtype="bf16", bits=16, page=16),
        # 200 requests under three instructions of different lengths, over packed INT8 rows
        dict(name="shared groups int8", op="shared", batch=200, groups=3, prefix=8191, own_len=512, hq=16, hkv=4, d=128, dtype="fp16", bits=8, page=32),
        # one decoding step: 64 tokens; launch latency counts
        dict(name="add norm step", op="add_norm", tokens=64, dim=4096, dtype="bf16", form="values", group=0),
        # a prompt batch of 16384 tokens; streaming
        dict(name="add norm prompt", op="add_norm", tokens=16384, dim=8192, dtype="bf16", form="values", group=0),
        # an odd number of tokens quantized to INT8 for the next product, a scale for every 128 elements
        dict(name="add norm int8", op="add_norm", tokens=4099, dim=5120, dtype="fp16", form="int8", group=128),
        # one step of 8 sequences: the sampled tokens' log probabilities with 20 alternatives; latency counts
        dict(name="logprobs step", op="logprobs", tokens=8, vocab=131072, dtype="bf16", top=20, masked=False),
        # a prompt's tokens scored under a large vocabulary
        dict(name="logprobs prompt", op="logprobs", tokens=4096, vocab=131072, dtype="bf16", top=5, masked=False),
        # a batch in 32 bits over an odd vocabulary, most of it ruled out by a grammar
        dict(name="logprobs masked fp32", op="logprobs", tokens=301, vocab=50021, dtype="fp32", top=8, masked=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("axes", "shared", "add_norm", "logprobs"))
    dtype = rng.choice(("bf16", "fp16"))
    if op == "axes":
        hkv, d = rng.choice((1, 2, 4, 8)), rng.choice((64, 96, 128))
        bits = rng.choice((0, 16, 16, 8))
        return dict(op=op, tokens=_log_int(rng, 1, 16384), hq=hkv * rng.choice((1, 2, 3, 4)), hkv=hkv, d=d, rot=rng.choice((d, d // 2)), axes=rng.choice((2, 3, 4)),
                    turns=rng.choice(("blocks", "one by one")), pairs=rng.choice(("half", "neighbours")), dtype=dtype, norm=rng.choice((True, False)), bits=bits, page=rng.choice((8, 16, 64)))
    if op == "shared":
        hkv, group, batch = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 7, 8)), _log_int(rng, 1, 256)
        return dict(op=op, batch=batch, groups=rng.choice((1, 1, 2, 5)), prefix=_log_int(rng, 1, min(32768, 4194304 // (batch * group))), own_len=_log_int(rng, 1, min(2048, 65536 // batch)),
                    hq=hkv * group, hkv=hkv, d=rng.choice((64, 96, 128)), dtype=dtype, bits=rng.choice((16, 16, 8, 4)), page=rng.choice((8, 16, 32, 64, 128)))
    if op == "add_norm":
        form = rng.choice(("values", "values", "int8", "fp8", "rows8"))
        dim = 8 * _log_int(rng, 8, 128 if form == "rows8" else 1024)  # packed rows end at 1024 elements
        return dict(op=op, tokens=_log_int(rng, 1, min(16384, (1 << 27) // dim)), dim=dim, dtype=dtype, form=form, group=rng.choice((0, 32, 128)) if form in ("int8", "fp8") and dim % 128 == 0 else 0)
    vocab = _log_int(rng, 500, 200000)
    dtype = rng.choice(("bf16", "fp16", "fp32"))
    return dict(op=op, tokens=_log_int(rng, 1, min(4096, (1 << 28) // vocab)), vocab=vocab, dtype=dtype, top=rng.choice((0, 1, 5, 20, 64)), masked=rng.choice((True, False)))


def _spread(n, top):
    """n lengths spread evenly over 1 .. top (the longest alone where n is 1)."""
    return [top] if n == 1 else [1 + (top - 1) * i // (n - 1) for i in range(n)]


def _groups(c):
    """(sequences, prefix length) of each group: sizes grow by one part, prefixes shrink; a batch smaller than its groups leaves some empty."""
    g = c["groups"]
    ends = [c["batch"] * (i + 1) * (i + 2) // (g * (g + 1)) for i in range(g)]
    sizes = [b - a for a, b in zip([0] + ends, ends)]
    return sizes, [max(1, c["prefix"] * (g - i) // g) for i in range(g)]


def _row_bytes(d, bits):
    return 2 * d if bits in (0, 16) else d * bits // 8 + 4


def work(case):
    c = case
    if c["op"] == "axes":
        heads = c["hq"] + (2 if c["bits"] else 1) * c["hkv"]
        out = 2 * c["hq"] * c["d"] + (2 if c["bits"] else 1) * c["hkv"] * _row_bytes(c["d"], c["bits"])
        return {"bytes": c["tokens"] * (2 * heads * c["d"] + out + 4 * c["rot"] + 4 * c["axes"] + (8 if c["bits"] else 0)), "flops": c["tokens"] * heads * c["d"] * 8}
    if c["op"] == "shared":
        sizes, prefixes = _groups(c)
        read = sum(p for n, p in zip(sizes, prefixes) if n) + sum(_spread(c["batch"], c["own_len"]))
        pairs = sum(n * p for n, p in zip(sizes, prefixes)) + sum(_spread(c["batch"], c["own_len"]))
        return {"bytes": read * c["hkv"] * 2 * _row_bytes(c["d"], c["bits"]) + c["batch"] * c["hq"] * (4 * c["d"] + 4), "flops": 4 * c["d"] * c["hq"] * pairs}
    if c["op"] == "add_norm":
        out = {"values": 2 * c["dim"], "rows8": c["dim"] + 4}.get(c["form"], c["dim"] + 4 * (c["dim"] // c["group"] if c["group"] else 1))
        return {"bytes": c["tokens"] * (6 * c["dim"] + out) + 2 * c["dim"], "flops": 5 * c["tokens"] * c["dim"]}
    size = 4 if c["dtype"] == "fp32" else 2
    return {"bytes": c["tokens"] * (c["vocab"] * size + 8 * c["top"] + 20), "flops": 6 * c["tokens"] * c["vocab"]}


# ---- what the program holds before the call ----

def _packed(x, bits=8):
    """Rows x [.., d] in 32 bits as packed rows [.., stride]: codes, scale and bias in 16 bits, padded to 16 bytes."""
    d, top = x.shape[-1], (1 << bits) - 1
    lo, hi = x.amin(-1, keepdim=True) + 0.0, x.amax(-1, keepdim=True) + 0.0
    scale, bias = ((hi - lo) / top).half(), lo.half()
    sf, bf = scale.float(), bias.float()
    codes = torch.where(sf > 0, ((x - bf) * (1.0 / sf)).round().clamp(0, top), torch.zeros_like(x)).to(torch.uint8)
    if bits == 4:
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    n = codes.shape[-1]
    rows = torch.zeros(x.shape[:-1] + ((n + 4 + 15) // 16 * 16,), dtype=torch.uint8, device=x.device)
    rows[..., :n] = codes
    rows[..., n:n + 4] = torch.cat((scale, bias), -1).view(torch.uint8)
    return rows


def _pool(g, pages, c):
    x = torch.randn((pages, c["hkv"], c["page"], c["d"]), generator=g, device="cuda")
    return x.to(DTYPES[c["dtype"]]) if c["bits"] == 16 else _packed(x, c["bits"])


def _table(g, lens, page, pool_order, used):
    """A page table [len(lens), width] of the pool's next pages in random order, and how many are used then."""
    need = [(n + page - 1) // page for n in lens]
    width = max(1, max(need))
    first = torch.tensor([used + sum(need[:i]) for i in range(len(need))], device="cuda")[:, None]
    place = torch.arange(width, device="cuda")[None]
    there = place < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(there, pool_order[(first + place).clamp(max=pool_order.numel() - 1)], 0)
    return table.to(torch.int32).contiguous(), used + sum(need)


def _axis_of_pairs(c):
    """Which axis turns each pair: the last axes share what half of the pairs leave, in blocks or one by one."""
    n, a = c["rot"] // 2, c["axes"]
    if c["turns"] == "one by one":
        return [i % a for i in range(n)]
    rest = [(n - n // 4) * (i + 1) // (a - 1) for i in range(a - 1)]
    ends = [n // 4] + [n // 4 + r for r in rest]
    return [next(k for k, e in enumerate(ends) if i < e) for i in range(n)]


def prepare(case, seed):
    c, dev = dict(case), "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": c}
    dt = DTYPES[c["dtype"]]
    if c["op"] == "axes":
        n, heads = c["tokens"], c["hq"] + 2 * c["hkv"]
        # the fused projection's output; q, k and v are its slices
        s["qkv"] = torch.randn((n, heads, c["d"]), generator=g, device=dev).mul_(1.7).to(dt)
        s["q"], s["k"], s["v"] = s["qkv"].split((c["hq"], c["hkv"], c["hkv"]), 1)
        s["wq"] = (1 + 0.2 * torch.randn(c["d"], generator=g, device=dev)).to(dt) if c["norm"] else None
        s["wk"] = (1 + 0.2 * torch.randn(c["d"], generator=g, device=dev)).to(dt) if c["norm"] else None
        places = 32768
        angle = torch.arange(places, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, c["rot"], 2, device=dev, dtype=torch.float64) / c["rot"])
        s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        s["pair_axes"] = torch.tensor(_axis_of_pairs(c), dtype=torch.uint8, device=dev)
        # frames of 24 x 32 patches after some text: time, height, width (and a constant); a step's tokens stand anywhere
        i = torch.arange(n, device=dev)
        if n > 1024:
            start = int(torch.randint(0, 1000, (1,), generator=g, device=dev))
            grid = torch.stack((start + i // 768, start + i // 32 % 24, start + i % 32, torch.full_like(i, start)))
        else:
            grid = torch.randint(0, places, (1, n), generator=g, device=dev).expand(4, -1)
        s["positions"] = (grid[1:3] if c["axes"] == 2 else grid[:c["axes"]]).to(torch.int32).contiguous()
        if not c["bits"]:
            return s
        pages = (n + c["page"] - 1) // c["page"] + 1
        s["slots"] = (torch.randperm(pages, generator=g, device=dev)[:, None] * c["page"] + torch.arange(c["page"], device=dev)).reshape(-1)[:n].contiguous()
        last, kind = (c["d"], dt) if c["bits"] == 16 else ((c["d"] * c["bits"] // 8 + 4 + 15) // 16 * 16, torch.uint8)
        s["k_pages"] = torch.zeros((pages, c["hkv"], c["page"], last), dtype=kind, device=dev)
        s["v_pages"] = torch.zeros_like(s["k_pages"])
        return s
    if c["op"] == "shared":
        sizes, prefixes = _groups(c)
        lens = torch.tensor(_spread(c["batch"], c["own_len"]), device=dev)[torch.randperm(c["batch"], generator=g, device=dev)].tolist()
        total = sum((n + c["page"] - 1) // c["page"] for n in prefixes + lens)
        order = torch.randperm(total, generator=g, device=dev)
        s["prefix_table"], used = _table(g, prefixes, c["page"], order, 0)
        s["block_table"], _ = _table(g, lens, c["page"], order, used)
        s["prefix_lens"] = torch.tensor(prefixes, dtype=torch.int32, device=dev)
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["group_offsets"] = torch.tensor([sum(sizes[:i]) for i in range(len(sizes) + 1)], dtype=torch.int32, device=dev)
        s["max_group"], s["max_prefix"], s["max_len"] = max(sizes), max(prefixes), max(lens)
        s["k_pages"], s["v_pages"] = _pool(g, total, c), _pool(g, total, c)
        s["q"] = torch.randn((c["batch"], c["hq"], c["d"]), generator=g, device=dev).mul_(1.5).to(dt)
        s["lse"] = torch.zeros((c["batch"], c["hq"]), device=dev)
        return s
    if c["op"] == "add_norm":
        s["x"] = torch.randn((c["tokens"], c["dim"]), generator=g, device=dev).to(dt)
        # a residual grown over many layers, a few channels far larger than the rest
        big = torch.where(torch.rand(c["dim"], generator=g, device=dev) < 0.005, 30.0, 3.0)
        s["residual"] = (torch.randn((c["tokens"], c["dim"]), generator=g, device=dev) * big).to(dt)
        s["weight"] = (1 + 0.2 * torch.randn(c["dim"], generator=g, device=dev)).to(dt)
        s["sum"] = torch.empty_like(s["x"])
        return s
    # logits as a trained model gives them: a wide bulk and a few likely tokens
    x = torch.randn((c["tokens"], c["vocab"]), generator=g, device=dev).mul_(2.5)
    for _ in range(4):
        at = torch.randint(0, c["vocab"], (c["tokens"], 1), generator=g, device=dev)
        x.scatter_(1, at, 8.0 + 3.0 * torch.randn((c["tokens"], 1), generator=g, device=dev))
    s["targets"] = at[:, 0].contiguous()
    if c["masked"]:  # ruled-out tokens; the target never is
        ruled = torch.rand((c["tokens"], c["vocab"]), generator=g, device=dev) < 0.9
        ruled.scatter_(1, at, False)
        x.masked_fill_(ruled, -math.inf)
    s["logits"] = x.to(dt)
    return s


# ---- the plain forms ----

def _values(rows, d, bits):
    """16-bit rows, or packed rows [.., stride], as 32-bit values [.., d]."""
    if bits == 16:
        return rows.float()
    n = d * bits // 8
    par = rows[..., n:n + 4].contiguous().view(torch.float16).float()
    codes = rows[..., :n]
    if bits == 4:
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return par[..., :1] * codes.float() + par[..., 1:]


def _plain_axes(s, c):
    # each pair's place: that of its axis
    pos = s["positions"].long()[s["pair_axes"].long()].t()  # [tokens, rot / 2]
    pair = torch.arange(c["rot"] // 2, device="cuda")
    cos, sin = s["cos_sin"][pos, pair][:, None], s["cos_sin"][pos, pair + c["rot"] // 2][:, None]

    def turned(x, w):
        x = x.float()
        if c["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["pairs"] == "half":
            a, b = r.chunk(2, -1)
            return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)
        a, b = r[..., 0::2], r[..., 1::2]
        return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), rest), -1)

    dt = s["q"].dtype
    q, k = turned(s["q"], s["wq"]).to(dt), turned(s["k"], s["wk"])
    if not c["bits"]:
        return {"q": q, "k": k.to(dt)}
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    s["k_pages"][page, :, at] = k.to(dt) if c["bits"] == 16 else _packed(k)
    s["v_pages"][page, :, at] = s["v"] if c["bits"] == 16 else _packed(s["v"].float())
    if c["bits"] == 16:
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    return {"q": q, "k_rows": _values(s["k_pages"], c["d"], c["bits"]).to(dt), "v_rows": _values(s["v_pages"], c["d"], c["bits"]).to(dt)}


def _rows_of(s, table, most, c):
    """The cached rows of each sequence of a table, padded to `most` slots: k, v [sequences, hkv, most, d] in 32 bits."""
    slot = torch.arange(most, device="cuda")
    page = table.long()[:, slot // c["page"]]
    return (_values(s[side][page, :, slot % c["page"]], c["d"], c["bits"]).transpose(1, 2).contiguous() for side in ("k_pages", "v_pages"))


def _plain_shared(s, c):
    """Scores against the prefixes, group by group at once (groups padded to the largest), and against each
    sequence's own rows; one softmax over both."""
    b, hkv, group, d = c["batch"], c["hkv"], c["hq"] // c["hkv"], c["d"]
    o = s["group_offsets"].long()
    i = torch.arange(s["max_group"], device="cuda")
    real = i < o.diff()[:, None]  # [groups, max_group]
    who = torch.where(real, o[:-1, None] + i, 0)
    k, v = _rows_of(s, s["prefix_table"], s["max_prefix"], c)
    q = s["q"].float().view(b, hkv, group, d)
    rows = q[who].permute(0, 2, 1, 3, 4).reshape(c["groups"], hkv, -1, d) * d ** -0.5
    e = torch.matmul(rows, k.transpose(-1, -2).contiguous())
    e.masked_fill_(torch.arange(s["max_prefix"], device="cuda") >= s["prefix_lens"][:, None, None, None], -math.inf)
    top = e.amax(-1, keepdim=True)
    e = (e - top).exp_()
    shape = (c["groups"], hkv, s["max_group"], group)
    of_seq = lambda t: t.reshape(shape + (-1,)).transpose(1, 2)[real]  # noqa: E731  [batch, hkv, group, ..]
    part, total, top = of_seq(torch.matmul(e, v)), of_seq(e.sum(-1, keepdim=True)), of_seq(top)
    del e
    k, v = _rows_of(s, s["block_table"], s["max_len"], c)
    e = torch.matmul(q * d ** -0.5, k.transpose(-1, -2).contiguous())
    e.masked_fill_(torch.arange(s["max_len"], device="cuda") >= s["seq_lens"][:, None, None, None], -math.inf)
    both = torch.maximum(top, e.amax(-1, keepdim=True))
    e, f = (e - both).exp_(), (top - both).exp()
    total = total * f + e.sum(-1, keepdim=True)
    out = (part * f + torch.matmul(e, v)) / total
    return {"out": out.reshape(b, c["hq"], d).to(s["q"].dtype), "lse": (both + total.log()).reshape(b, c["hq"])}


def _plain_add_norm(s, c):
    h = s["x"].float() + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    h = h.to(s["x"].dtype)
    if c["form"] == "values":
        return {"y": y.to(s["x"].dtype), "sum": h}
    if c["form"] == "rows8":
        return {"y": _values(_packed(y), c["dim"], 8).to(s["x"].dtype), "sum": h}
    y = y.view(c["tokens"], -1, c["group"] or c["dim"])
    most = 127.0 if c["form"] == "int8" else 448.0
    scale = y.abs().amax(-1, keepdim=True) / most
    y = y / torch.where(scale > 0, scale, 1.0)
    codes = y.round() if c["form"] == "int8" else y.to(torch.float8_e4m3fn).float()
    return {"y": (codes * scale).view(c["tokens"], -1).to(s["x"].dtype), "sum": h}


def _plain_logprobs(s, c):
    given = s["logits"].float() + 0.0
    top = given.amax(-1, keepdim=True)
    x = given - top
    e = x.exp()
    total = e.sum(-1, keepdim=True)
    log_total = total.log()
    out = {"logprobs": (x.gather(1, s["targets"][:, None]) - log_total)[:, 0],
           "entropy": (log_total - (e * torch.where(e > 0, x, 0.0)).sum(-1, keepdim=True) / total)[:, 0]}
    if c["top"]:
        # keys that order as the values do, and equal values from the lowest index
        bits = given.view(torch.int32)
        bits = (bits ^ ((bits >> 31) & 0x7fffffff)).long()
        ids = (bits * c["vocab"] - torch.arange(c["vocab"], device="cuda")).topk(c["top"], -1).indices
        out["top_ids"], out["top_logprobs"] = ids.to(torch.int32), x.gather(1, ids) - log_total
    return out


def _own(s, c):
    import int4_row_wise_amd as lib

    # what is held in 8 bits is returned as the values that it stands for
    if c["op"] == "axes":
        cache = dict(v=s["v"], k_pages=s["k_pages"], v_pages=s["v_pages"], slots=s["slots"], bits=c["bits"]) if c["bits"] else {}
        q, k = lib.norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], s["wq"], s["wk"], eps=EPS, interleaved=c["pairs"] == "neighbours", pair_axes=s["pair_axes"], norm=c["norm"], **cache)
        if not c["bits"]:
            return {"q": q, "k": k}
        if c["bits"] == 16:
            return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        k, v = (lib.dequantize(p.view(-1, p.shape[-1]), c["d"], c["bits"]).view(p.shape[:-1] + (c["d"],)).to(q.dtype) for p in (s["k_pages"], s["v_pages"]))
        return {"q": q, "k_rows": k, "v_rows": v}
    if c["op"] == "shared":
        out = lib.shared_attention(s["q"], s["k_pages"], s["v_pages"], s["prefix_table"], s["prefix_lens"], s["block_table"], s["seq_lens"], group_offsets=s["group_offsets"], bits=c["bits"],
                                   lse=s["lse"])
        return {"out": out, "lse": s["lse"]}
    if c["op"] == "add_norm":
        y, h, scales = lib.add_norm(s["x"], s["residual"], s["weight"], eps=EPS, form=c["form"], group=c["group"], sum_out=s["sum"])
        if c["form"] == "rows8":
            y = lib.dequantize(y, c["dim"], 8).to(h.dtype)
        elif c["form"] != "values":
            codes = y if c["form"] == "int8" else y.to(h.dtype)  # exactly
            y = torch.empty_like(h)
            torch.mul(codes.view(scales.shape + (-1,)), scales[..., None], out=y.view(scales.shape + (-1,)))
        return {"y": y, "sum": h}
    got = lib.token_logprobs(s["logits"], s["targets"], top=c["top"])
    out = {"logprobs": got[0], "entropy": got[1]}
    return out | ({"top_ids": got[2], "top_logprobs": got[3]} if c["top"] else {})


PLAIN = {"axes": _plain_axes, "shared": _plain_shared, "add_norm": _plain_add_norm, "logprobs": _plain_logprobs}


def run(state):
    c = state["case"]
    return _own(state, c) if own else PLAIN[c["op"]](state, c)


# ---- the definitions in 64 bits ----

def exact(case, seed):
    def values(rows, d, bits):
        if bits == 16:
            return rows.double()
        n = d * bits // 8
        scale, bias = (rows[..., n + o:n + o + 2].contiguous().view(torch.float16).double() for o in (0, 2))
        byte = rows[..., :n].long()
        if bits == 8:
            return scale * byte + bias
        out = torch.empty(rows.shape[:-1] + (d,), dtype=torch.float64, device=rows.device)
        out[..., 0::2], out[..., 1::2] = scale * (byte % 16) + bias, scale * (byte // 16) + bias
        return out

    def held(x):
        """Rows as packed INT8 rows hold them."""
        lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
        scale, bias = ((hi - lo) / 255).half().double(), lo.half().double()
        safe = torch.where(scale > 0, scale, 1.0)
        return torch.where(scale > 0, torch.round((x - bias) / safe).clamp(0, 255), 0.0) * scale + bias

    def axes(s, c):
        half = c["rot"] // 2
        place = s["positions"].tolist()
        table = s["cos_sin"].double()

        def one(x, w):
            y = x.double()
            if c["norm"]:
                y = y / (y.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * w.double()
            z = y.clone()
            for i, axis in enumerate(s["pair_axes"].tolist()):
                a, b = (i, i + half) if c["pairs"] == "half" else (2 * i, 2 * i + 1)
                co, si = table[where[axis], i][:, None], table[where[axis], half + i][:, None]
                z[..., a] = y[..., a] * co - y[..., b] * si
                z[..., b] = y[..., b] * co + y[..., a] * si
            return z

        where = [torch.tensor(p, device="cuda") for p in place]
        q, k = one(s["q"], s["wq"]), one(s["k"], s["wk"])
        if not c["bits"]:
            return {"q": q, "k": k}
        pages = torch.zeros((2,) + s["k_pages"].shape[:3] + (c["d"],), dtype=torch.float64, device="cuda")
        for i, x in enumerate((k, s["v"].double())):
            pages[i, s["slots"] // c["page"], :, s["slots"] % c["page"]] = x if c["bits"] == 16 else held(x)
        names = ("k_pages", "v_pages") if c["bits"] == 16 else ("k_rows", "v_rows")
        return {"q": q, names[0]: pages[0], names[1]: pages[1]}

    def shared(s, c):
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        o, per = s["group_offsets"].tolist(), c["hq"] // c["hkv"]

        def rows(side, table, n):
            got = values(s[side][table[:(n + c["page"] - 1) // c["page"]].long()], c["d"], c["bits"])
            return got.transpose(0, 1).reshape(c["hkv"], -1, c["d"])[:, :n]

        for g, n in enumerate(s["prefix_lens"].tolist()):
            pk, pv = (rows(side, s["prefix_table"][g], n) for side in ("k_pages", "v_pages"))
            for b in range(o[g], o[g + 1]):
                m = int(s["seq_lens"][b])
                k, v = (torch.cat((p, rows(side, s["block_table"][b], m)), 1) for p, side in ((pk, "k_pages"), (pv, "v_pages")))
                e = torch.bmm(k, s["q"][b].double().view(c["hkv"], per, -1).transpose(1, 2).contiguous()) / math.sqrt(c["d"])
                z = torch.logsumexp(e, 1)
                lse[b] = z.reshape(-1)
                out[b] = torch.bmm(torch.exp(e - z[:, None]).transpose(1, 2).contiguous(), v).reshape(c["hq"], -1)
        return {"out": out, "lse": lse}

    def add_norm(s, c):
        h = s["x"].double() + s["residual"].double()
        y = h / (h.pow(2).sum(-1, keepdim=True) / c["dim"] + EPS).sqrt() * s["weight"].double()
        if c["form"] == "rows8":
            y = held(y)
        if c["form"] in ("int8", "fp8"):
            y = y.reshape(c["tokens"], -1, c["group"] or c["dim"])
            largest = y.abs().max(-1, keepdim=True).values
            if c["form"] == "int8":
                y = torch.round(y * 127 / largest.clamp(min=1e-300)) * largest / 127
            else:  # three bits after the leading one, down to steps of 2^-9
                t = y * 448 / largest.clamp(min=1e-300)
                step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
                y = torch.round(t / step) * step * largest / 448
            y = y.reshape(c["tokens"], -1)
        return {"y": y, "sum": h}

    def logprobs(s, c):
        got = {"logprobs": [], "entropy": [], "top_logprobs": []}
        for lo in range(0, c["tokens"], 256):
            x = s["logits"][lo:lo + 256].double()
            p = torch.softmax(x, -1)
            lp = x - torch.logsumexp(x, -1, keepdim=True)
            got["logprobs"].append(lp[torch.arange(x.shape[0], device="cuda"), s["targets"][lo:lo + 256]])
            got["entropy"].append(-torch.where(p > 0, p * lp, 0.0).sum(-1))
            got["top_logprobs"].append(lp.topk(min(c["top"], c["vocab"]), -1).values)
        out = {"logprobs": torch.cat(got["logprobs"]), "entropy": torch.cat(got["entropy"])}
        return out | ({"top_ids": None, "top_logprobs": torch.cat(got["top_logprobs"])} if c["top"] else {})

    forms = {"axes": axes, "shared": shared, "add_norm": add_norm, "logprobs": logprobs}
    return forms[case["op"]](prepare(case, seed), case)
