"""The attention operators over a key-value cache of 16-bit or packed INT8 / INT4 rows, as measured cases.

Each case names one operator and its sizes; `prepare` makes what a serving program holds before the call, `run`
makes one call, in plain torch operations or (where `own` is set) through the package's entry points, and `exact`
computes the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


def listed():
    return [
        # one decoding step of 64 sequences: 64 tokens normed, rotated and appended; launch latency counts
        dict(name="norm_rope step", op="norm_rope", tokens=64, hq=32, hkv=8, d=128, rot=128, pairs="half", dtype="bf16", bits=16, page=16),
        # a prompt batch of 16384 tokens into 16-bit pages; streaming
        dict(name="norm_rope prompt", op="norm_rope", tokens=16384, hq=32, hkv=8, d=128, rot=128, pairs="half", dtype="bf16", bits=16, page=16),
        # an odd prompt length into packed INT8 rows, half of each head rotated, neighbouring pairs
        dict(name="norm_rope prompt int8", op="norm_rope", tokens=8191, hq=16, hkv=4, d=64, rot=32, pairs="neighbours", dtype="fp16", bits=8, page=32),
        # many short prompts of 1 to 512 tokens, some of them continuing keys that are there already
        dict(name="prompt short ragged", op="prompt", batch=32, max_q=512, prefix=100, hq=32, hkv=8, d=128, dtype="bf16", window=0, sinks=0),
        # one long document read through a window of 1024 keys with 4 sinks
        dict(name="prompt window sinks", op="prompt", batch=1, max_q=16384, prefix=0, hq=16, hkv=4, d=128, dtype="bf16", window=1024, sinks=4),
        # a full causal prompt of 8192 tokens: matrix-product bound
        dict(name="prompt causal 8k", op="prompt", batch=1, max_q=8192, prefix=0, hq=32, hkv=8, d=128, dtype="bf16", window=0, sinks=0),
        # one user's next token over a long cache: few rows, so the length is split
        dict(name="decode one sequence", op="decode", batch=1, max_len=32768, hq=32, hkv=8, d=128, dtype="bf16", bits=16, page=16, window=0, sinks=0, mass=False),
        # a ragged serving batch over 16-bit pages that keeps the accumulated weights
        dict(name="decode batch mass", op="decode", batch=64, max_len=8192, hq=32, hkv=8, d=128, dtype="bf16", bits=16, page=16, window=0, sinks=0, mass=True),
        # the same batch over packed INT8 rows
        dict(name="decode batch int8", op="decode", batch=64, max_len=8192, hq=32, hkv=8, d=128, dtype="bf16", bits=8, page=16, window=0, sinks=0, mass=False),
        # long caches of packed INT4 rows read through a window with sinks, d = 64
        dict(name="decode int4 window", op="decode", batch=128, max_len=16384, hq=16, hkv=8, d=64, dtype="fp16", bits=4, page=64, window=4096, sinks=4, mass=True),
        # a few short caches cut to a quarter: selection latency counts
        dict(name="evict few", op="evict", batch=4, max_len=2048, hkv=8, d=128, dtype="bf16", bits=16, page=16, keep=512, sinks=4, recent=128),
        # a serving batch of INT8 caches cut to at most 4096 rows
        dict(name="evict batch", op="evict", batch=32, max_len=16384, hkv=8, d=128, dtype="bf16", bits=8, page=16, keep=4096, sinks=4, recent=512),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("norm_rope", "prompt", "decode", "evict"))
    hkv, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 7, 8))
    d, dtype = rng.choice((64, 96, 128)), rng.choice(("bf16", "fp16"))
    page = rng.choice((8, 16, 32, 64, 128))
    if op == "norm_rope":
        group = min(group, 4)
        return dict(op=op, tokens=_log_int(rng, 1, 16384), hq=hkv * group, hkv=hkv, d=d, rot=rng.choice((d, d // 2)), pairs=rng.choice(("half", "neighbours")), dtype=dtype,
                    bits=rng.choice((16, 16, 8)), page=page)
    if op == "prompt":
        hq, batch = min(32, hkv * group), _log_int(rng, 1, 16)
        hq -= hq % hkv
        max_q = _log_int(rng, 1, min(8192, int(math.sqrt(8192 * 8192 / batch))))
        window = rng.choice((0, 0, _log_int(rng, 16, 4096)))
        return dict(op=op, batch=batch, max_q=max_q, prefix=rng.choice((0, 0, _log_int(rng, 1, 300))), hq=hq, hkv=hkv, d=d, dtype=dtype, window=window, sinks=rng.choice((0, 1, 4)) if window else 0)
    if op == "decode":
        batch = _log_int(rng, 1, 128)
        max_len = _log_int(rng, 1, min(32768, 524288 // batch))
        window = rng.choice((0, 0, _log_int(rng, 16, 8192)))
        return dict(op=op, batch=batch, max_len=max_len, hq=hkv * group, hkv=hkv, d=d, dtype=dtype, bits=rng.choice((16, 8, 4)), page=page, window=window, sinks=rng.choice((0, 4, 13)) if window else 0,
                    mass=rng.choice((True, False)))
    batch = _log_int(rng, 1, 32)
    max_len = _log_int(rng, 64, 16384)
    keep = max(8, int(max_len * rng.uniform(0.1, 0.6)))
    return dict(op=op, batch=batch, max_len=max_len, hkv=hkv, d=d, dtype=dtype, bits=rng.choice((16, 8, 4)), page=page, keep=keep, sinks=rng.choice((0, 4)), recent=rng.randrange(0, keep - 4))


def _spread(n, top):
    """n lengths spread evenly over 1 .. top (the longest alone where n is 1)."""
    return [top] if n == 1 else [1 + (top - 1) * i // (n - 1) for i in range(n)]


def _visible(p, keys, window, sinks):
    """How many of `keys` keys a query at place p sees."""
    last = min(p, keys - 1)
    if last < 0:
        return 0
    if not window:
        return last + 1
    first = max(0, p - window + 1)
    return max(0, last - first + 1) + min(sinks, first, last + 1)


def _row_bytes(d, bits):
    return 2 * d if bits == 16 else d * bits // 8 + 4


def work(case):
    c = case
    if c["op"] == "norm_rope":
        heads = c["hq"] + 2 * c["hkv"]
        out = 2 * c["hq"] * c["d"] + 2 * c["hkv"] * _row_bytes(c["d"], c["bits"])
        return {"bytes": c["tokens"] * (2 * heads * c["d"] + out + 4 * c["rot"] + 16), "flops": c["tokens"] * heads * c["d"] * 8}
    if c["op"] == "prompt":
        qs = _spread(c["batch"], c["max_q"])
        ks = [n + c["prefix"] * (i % 2) for i, n in enumerate(qs)]
        pairs = 0
        for nq, nk in zip(qs, ks):
            pairs += sum(_visible(i + nk - nq, nk, c["window"], c["sinks"]) for i in range(nq))
        return {"bytes": 2 * c["d"] * (2 * sum(qs) * c["hq"] + 2 * sum(ks) * c["hkv"]) + 4 * sum(qs) * c["hq"], "flops": 4 * c["d"] * c["hq"] * pairs}
    lens = _spread(c["batch"], c["max_len"])
    if c["op"] == "decode":
        seen = sum(_visible(n - 1, n, c["window"], c["sinks"]) for n in lens)
        cache = seen * c["hkv"] * 2 * _row_bytes(c["d"], c["bits"])
        mass = 8 * seen * c["hkv"] if c["mass"] else 0
        return {"bytes": cache + mass + c["batch"] * c["hq"] * (4 * c["d"] + 4) + 4 * c["batch"] * (max(lens) // c["page"] + 1), "flops": 4 * c["d"] * c["hq"] * seen}
    kept = sum(min(n, c["keep"]) for n in lens)
    return {"bytes": c["hkv"] * (4 * sum(lens) + kept * (4 * _row_bytes(c["d"], c["bits"]) + 8)), "flops": 0}


# ---- what the program holds before the call ----

def _packed(x, bits):
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


def _pool(g, pages, c, dev):
    x = torch.randn((pages, c["hkv"], c["page"], c["d"]), generator=g, device=dev)
    return x.to(DTYPES[c["dtype"]]) if c["bits"] == 16 else _packed(x, c["bits"])


def _table(g, lens, page, width, dev):
    """A page table [batch, width] of pages in random order, each sequence's own, and the number of pages."""
    need = (lens + page - 1) // page
    total = int(need.sum())
    place = torch.arange(width, device=dev)[None] + (need.cumsum(0) - need)[:, None]
    order = torch.randperm(total, generator=g, device=dev)
    table = torch.where(torch.arange(width, device=dev)[None] < need[:, None], order[place.clamp(max=total - 1)], 0)
    return table.to(torch.int32).contiguous(), total


def prepare(case, seed):
    c, dev = dict(case), "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "norm_rope":
        n, heads, dt = c["tokens"], c["hq"] + 2 * c["hkv"], DTYPES[c["dtype"]]
        # the fused projection's output; q, k and v are its slices
        s["qkv"] = torch.randn((n, heads, c["d"]), generator=g, device=dev).mul_(1.7).to(dt)
        s["q"], s["k"], s["v"] = s["qkv"].split((c["hq"], c["hkv"], c["hkv"]), 1)
        s["wq"] = (1 + 0.2 * torch.randn(c["d"], generator=g, device=dev)).to(dt)
        s["wk"] = (1 + 0.2 * torch.randn(c["d"], generator=g, device=dev)).to(dt)
        places = max(32768, n)
        angle = torch.arange(places, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, c["rot"], 2, device=dev, dtype=torch.float64) / c["rot"])
        s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        start = 0 if n > 1024 else int(torch.randint(0, places - n + 1, (1,), generator=g, device=dev))
        s["positions"] = torch.arange(start, start + n, device=dev, dtype=torch.int32)
        pages = (n + c["page"] - 1) // c["page"] + 1
        s["slots"] = torch.randperm(pages * c["page"], generator=g, device=dev)[:n] if n <= 1024 else \
            (torch.randperm(pages, generator=g, device=dev)[:, None] * c["page"] + torch.arange(c["page"], device=dev)).reshape(-1)[:n].contiguous()
        shape = (pages, c["hkv"], c["page"])
        last, kind = (c["d"], dt) if c["bits"] == 16 else ((c["d"] * c["bits"] // 8 + 4 + 15) // 16 * 16, torch.uint8)
        s["k_pages"] = torch.zeros(shape + (last,), dtype=kind, device=dev)
        s["v_pages"] = torch.zeros(shape + (last,), dtype=kind, device=dev)
        return s
    if c["op"] == "prompt":
        qs = torch.tensor(_spread(c["batch"], c["max_q"]), device=dev)
        ks = qs + c["prefix"] * (torch.arange(c["batch"], device=dev) % 2)
        order = torch.randperm(c["batch"], generator=g, device=dev)
        qs, ks = qs[order], ks[order]
        zero = torch.zeros(1, dtype=torch.int64, device=dev)
        s["q_offsets"] = torch.cat((zero, qs.cumsum(0))).to(torch.int32)
        s["k_offsets"] = torch.cat((zero, ks.cumsum(0))).to(torch.int32)
        s["max_k"] = c["max_q"] + c["prefix"]
        nq, nk, dt = int(qs.sum()), int(ks.sum()), DTYPES[c["dtype"]]
        s["q"] = torch.randn((nq, c["hq"], c["d"]), generator=g, device=dev).mul_(1.5).to(dt)
        s["k"] = torch.randn((nk, c["hkv"], c["d"]), generator=g, device=dev).to(dt)
        s["v"] = torch.randn((nk, c["hkv"], c["d"]), generator=g, device=dev).to(dt)
        s["lse"] = torch.zeros((nq, c["hq"]), device=dev)
        return s
    lens = torch.tensor(_spread(c["batch"], c["max_len"]), device=dev)[torch.randperm(c["batch"], generator=g, device=dev)]
    width = (c["max_len"] + c["page"] - 1) // c["page"]
    s["seq_lens"] = lens.to(torch.int32)
    s["block_table"], pages = _table(g, lens, c["page"], width, dev)
    s["k_pages"], s["v_pages"] = _pool(g, pages, c, dev), _pool(g, pages, c, dev)
    if c["op"] == "decode":
        s["q"] = torch.randn((c["batch"], c["hq"], c["d"]), generator=g, device=dev).mul_(1.5).to(DTYPES[c["dtype"]])
        s["lse"] = torch.zeros((c["batch"], c["hq"]), device=dev)
        s["mass"] = torch.rand((c["batch"], c["hkv"], c["max_len"]), generator=g, device=dev).mul_(1e-3) if c["mass"] else None
        return s
    # weight accumulated over many steps: a few heavy rows, many light ones, zeros and equal values among them
    m = torch.randn((c["batch"], c["hkv"], c["max_len"]), generator=g, device=dev).mul_(2.0).exp_().mul_(0.01)
    m[..., ::17] = 0.0
    s["mass"] = (m * 1024).round_().div_(1024)
    new_lens = lens.clamp(max=c["keep"])
    new_width = (c["keep"] + c["page"] - 1) // c["page"]
    s["new_table"], new_pages = _table(g, new_lens, c["page"], new_width, dev)
    s["new_k_pages"] = torch.zeros((new_pages,) + s["k_pages"].shape[1:], dtype=s["k_pages"].dtype, device=dev)
    s["new_v_pages"] = torch.zeros_like(s["new_k_pages"])
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


def _softmax(s, see, dim):
    """(weights, sums' logarithm) over `dim`, nothing where `see` is false; a row that sees nothing has no weight."""
    s = torch.where(see, s, -math.inf)
    top = s.amax(dim, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (s - top).exp_()
    total = p.sum(dim, keepdim=True)
    return p.div_(torch.where(total > 0, total, 1.0)), (total.log() + top).squeeze(dim)


def _plain_norm_rope(s, c):
    def normed(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        cos, sin = s["cos_sin"][s["positions"].long()][:, None].chunk(2, -1)
        r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["pairs"] == "half":
            a, b = r.chunk(2, -1)
            return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)
        a, b = r[..., 0::2], r[..., 1::2]
        return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), rest), -1)

    dt = s["q"].dtype
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    k, v = normed(s["k"], s["wk"]), s["v"].float()
    s["k_pages"][page, :, at] = k.to(dt) if c["bits"] == 16 else _packed(k, c["bits"])
    s["v_pages"][page, :, at] = v.to(dt) if c["bits"] == 16 else _packed(v, c["bits"])
    out = {"q": normed(s["q"], s["wq"]).to(dt)}
    if c["bits"] == 16:
        return out | {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    return out | {"k_rows": _values(s["k_pages"], c["d"], c["bits"]).to(dt), "v_rows": _values(s["v_pages"], c["d"], c["bits"]).to(dt)}


def _plain_prompt(s, c):
    qo, ko = s["q_offsets"].long(), s["k_offsets"].long()
    nq, nk = qo.diff(), ko.diff()
    iq, ik = torch.arange(c["max_q"], device="cuda"), torch.arange(s["max_k"], device="cuda")
    group, b, d = c["hq"] // c["hkv"], c["batch"], c["d"]
    q = s["q"].float()[(qo[:-1, None] + iq).clamp(max=s["q"].shape[0] - 1)]  # [b, max_q, hq, d]
    k = s["k"].float()[(ko[:-1, None] + ik).clamp(max=s["k"].shape[0] - 1)]
    v = s["v"].float()[(ko[:-1, None] + ik).clamp(max=s["v"].shape[0] - 1)]
    q = q.view(b, c["max_q"], c["hkv"], group, d).permute(0, 2, 3, 1, 4).reshape(b, c["hkv"], group * c["max_q"], d)
    sc = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).mul_(d ** -0.5).view(b, c["hkv"], group, c["max_q"], s["max_k"])
    p = (iq[None] + (nk - nq)[:, None])[:, :, None]  # the query's place among the keys
    see = (ik <= p) & (ik < nk[:, None, None])
    if c["window"]:
        see &= (ik > p - c["window"]) | (ik < c["sinks"])
    w, lse = _softmax(sc, see[:, None, None], -1)
    o = torch.matmul(w.view(b, c["hkv"], group * c["max_q"], s["max_k"]), v.permute(0, 2, 1, 3).contiguous())
    real = iq[None] < nq[:, None]
    o = o.view(b, c["hq"], c["max_q"], d).transpose(1, 2)[real]
    return {"out": o.to(s["q"].dtype), "lse": lse.reshape(b, c["hq"], c["max_q"]).transpose(1, 2)[real]}


def _plain_decode(s, c):
    n = s["seq_lens"].long()
    b, group, d = c["batch"], c["hq"] // c["hkv"], c["d"]
    if c["window"]:
        first = (n - c["window"]).clamp(min=c["sinks"])
        i = torch.arange(c["sinks"] + c["window"], device="cuda")
        at = torch.where(i < c["sinks"], i, first[:, None] + i - c["sinks"])
    else:
        at = torch.arange(c["max_len"], device="cuda").expand(b, -1)
    see = at < n[:, None]
    at = torch.where(see, at, 0)
    page = s["block_table"].long().gather(1, at // c["page"])
    k = _values(s["k_pages"][page, :, at % c["page"]], d, c["bits"]).transpose(1, 2).contiguous()  # [b, hkv, seen, d]
    v = _values(s["v_pages"][page, :, at % c["page"]], d, c["bits"]).transpose(1, 2).contiguous()
    q = s["q"].float().view(b, c["hkv"], group, d).transpose(-1, -2).contiguous()
    w, lse = _softmax(torch.matmul(k, q) * d ** -0.5, see[:, None, :, None], 2)
    o = torch.matmul(w.transpose(-1, -2).contiguous(), v)
    out = {"out": o.reshape(b, c["hq"], d).to(s["q"].dtype), "lse": lse.reshape(b, c["hq"])}
    if c["mass"]:
        out["mass"] = s["mass"].scatter_add_(2, at[:, None].expand(-1, c["hkv"], -1), w.sum(-1))
    return out


def _plain_evict(s, c):
    n, keep = s["seq_lens"].long()[:, None, None], c["keep"]
    i = torch.arange(c["max_len"], device="cuda")
    held = (i < c["sinks"]) | (i >= n - c["recent"])
    m = torch.where(i < n, torch.where(held, math.inf, torch.nan_to_num(s["mass"], nan=-math.inf, posinf=math.inf, neginf=-math.inf)), -math.inf)
    real = i.expand_as(m) < n
    order = m.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.where(real.gather(-1, order), order, c["max_len"]).sort(-1).values
    there = kept < c["max_len"]
    at = torch.where(there, kept, 0)
    j = torch.arange(kept.shape[-1], device="cuda").expand_as(kept)
    head = torch.arange(c["hkv"], device="cuda")[None, :, None].expand_as(kept)
    seq = torch.arange(c["batch"], device="cuda")[:, None, None].expand_as(kept)
    src = s["block_table"].long()[seq, at // c["page"]][there], head[there], (at % c["page"])[there]
    dst = s["new_table"].long()[seq, j // c["page"]][there], head[there], (j % c["page"])[there]
    s["new_k_pages"][dst] = s["k_pages"][src]
    s["new_v_pages"][dst] = s["v_pages"][src]
    mass = torch.where(there, s["mass"].gather(-1, at), 0.0)
    full = torch.nn.functional.pad(torch.where(there, kept, -1), (0, keep - kept.shape[-1]), value=-1)
    return {"kept": full.to(torch.int32), "mass": torch.nn.functional.pad(mass, (0, keep - kept.shape[-1])), "seq_lens": s["seq_lens"].clamp(max=keep), "k": s["new_k_pages"], "v": s["new_v_pages"]}


def _own(s, c):
    import int4_row_wise_amd as lib

    if c["op"] == "norm_rope":
        q, _ = lib.norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], s["wq"], s["wk"], eps=EPS, interleaved=c["pairs"] == "neighbours", v=s["v"], k_pages=s["k_pages"], v_pages=s["v_pages"],
                             slots=s["slots"], bits=c["bits"])
        if c["bits"] == 16:
            return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        # what is held in 8 bits as the values that it stands for
        k, v = (lib.dequantize(p.view(-1, p.shape[-1]), c["d"], c["bits"]).view(p.shape[:-1] + (c["d"],)).to(q.dtype) for p in (s["k_pages"], s["v_pages"]))
        return {"q": q, "k_rows": k, "v_rows": v}
    if c["op"] == "prompt":
        out = lib.prompt_attention(s["q"], s["k"], s["v"], s["q_offsets"], s["k_offsets"], max_q=c["max_q"], window=c["window"], sinks=c["sinks"], lse=s["lse"])
        return {"out": out, "lse": s["lse"]}
    if c["op"] == "decode":
        out = lib.decode_attention(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"], bits=c["bits"], window=c["window"], sinks=c["sinks"], mass=s["mass"], lse=s["lse"])
        return {"out": out, "lse": s["lse"]} | ({"mass": s["mass"]} if c["mass"] else {})
    kept, mass, lens = lib.evict(s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"], s["mass"], c["keep"], s["new_k_pages"], s["new_v_pages"], s["new_table"], sinks=c["sinks"], recent=c["recent"])
    return {"kept": kept, "mass": mass, "seq_lens": lens, "k": s["new_k_pages"], "v": s["new_v_pages"]}


PLAIN = {"norm_rope": _plain_norm_rope, "prompt": _plain_prompt, "decode": _plain_decode, "evict": _plain_evict}


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

    def norm_rope(s, c):
        cos = s["cos_sin"][s["positions"].long(), :c["rot"] // 2].double()
        sin = s["cos_sin"][s["positions"].long(), c["rot"] // 2:].double()
        step = c["rot"] // 2

        def one(x, w):
            x = x.double()
            y = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * w.double()
            z = y.clone()
            for i in range(step):
                a, b = (i, i + step) if c["pairs"] == "half" else (2 * i, 2 * i + 1)
                z[..., a] = y[..., a] * cos[:, None, i] - y[..., b] * sin[:, None, i]
                z[..., b] = y[..., b] * cos[:, None, i] + y[..., a] * sin[:, None, i]
            return z

        def held(x):
            if c["bits"] == 16:
                return x
            top = 2 ** c["bits"] - 1
            lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            scale, bias = ((hi - lo) / top).half().double(), lo.half().double()
            return torch.round((x - bias) / scale).clamp(0, top) * scale + bias

        pages = torch.zeros((2,) + s["k_pages"].shape[:3] + (c["d"],), dtype=torch.float64, device="cuda")
        for i, x in enumerate((one(s["k"], s["wk"]), s["v"].double())):
            pages[i, s["slots"] // c["page"], :, s["slots"] % c["page"]] = held(x)
        names = ("k_pages", "v_pages") if c["bits"] == 16 else ("k_rows", "v_rows")
        return {"q": one(s["q"], s["wq"]), names[0]: pages[0], names[1]: pages[1]}

    def attend(q, k, v, see):
        """q [n, d], k and v [m, d], see [n, m] -> (o, lse, weights)."""
        e = (q @ k.t().contiguous()) / math.sqrt(q.shape[1])
        e.masked_fill_(~see, -math.inf)
        lse = torch.logsumexp(e, 1)
        w = torch.exp(e - torch.where(lse == -math.inf, 0.0, lse)[:, None])
        return w @ v, lse, w

    def prompt(s, c):
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        qo, ko, group = s["q_offsets"].tolist(), s["k_offsets"].tolist(), c["hq"] // c["hkv"]
        for b in range(c["batch"]):
            nq, nk = qo[b + 1] - qo[b], ko[b + 1] - ko[b]
            place, key = torch.arange(nk - nq, nk, device="cuda")[:, None], torch.arange(nk, device="cuda")[None]
            see = key <= place
            if c["window"]:
                see = see & ((place - key < c["window"]) | (key < c["sinks"]))
            for h in range(c["hq"]):
                kv = slice(ko[b], ko[b + 1]), h // group
                for lo in range(0, nq, 4096):
                    at = slice(qo[b] + lo, min(qo[b] + lo + 4096, qo[b + 1]))
                    out[at, h], lse[at, h], _ = attend(s["q"][at, h].double(), s["k"][kv].double(), s["v"][kv].double(), see[lo:lo + 4096])
        return {"out": out, "lse": lse}

    def decode(s, c):
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        mass = s["mass"].double() if c["mass"] else None
        group = c["hq"] // c["hkv"]
        for b, n in enumerate(s["seq_lens"].tolist()):
            own_pages = s["block_table"][b, :(n + c["page"] - 1) // c["page"]].long()
            k, v = (values(p[own_pages], c["d"], c["bits"]).transpose(0, 1).reshape(c["hkv"], -1, c["d"])[:, :n] for p in (s["k_pages"], s["v_pages"]))
            key = torch.arange(n, device="cuda")
            see = (n - 1 - key < c["window"]) | (key < c["sinks"]) if c["window"] else key >= 0
            for h in range(c["hkv"]):
                at = slice(h * group, (h + 1) * group)
                out[b, at], lse[b, at], w = attend(s["q"][b, at].double(), k[h], v[h], see[None].expand(group, -1))
                if c["mass"]:
                    mass[b, h, :n] += w.sum(0)
        return {"out": out, "lse": lse} | ({"mass": mass} if c["mass"] else {})

    def evict(s, c):
        m = s["mass"].cpu()
        got = torch.zeros((c["batch"], c["hkv"], c["keep"]), dtype=torch.float64)
        for b, n in enumerate(s["seq_lens"].tolist()):
            for h in range(c["hkv"]):
                if n <= c["keep"]:
                    got[b, h, :n] = m[b, h, :n].double()
                    continue
                middle = m[b, h, c["sinks"]:n - c["recent"]].tolist()
                best = sorted(range(len(middle)), key=lambda i: (-middle[i], i))[:c["keep"] - c["sinks"] - c["recent"]]
                ids = list(range(c["sinks"])) + sorted(i + c["sinks"] for i in best) + list(range(n - c["recent"], n))
                got[b, h] = m[b, h, ids].double()
        return {"kept": None, "mass": got.cuda(), "seq_lens": None, "k": None, "v": None}  # the others are whole numbers and copies

    forms = {"norm_rope": norm_rope, "prompt": prompt, "decode": decode, "evict": evict}
    return forms[case["op"]](prepare(case, seed), case)
