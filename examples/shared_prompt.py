"""Many answers to one prompt with an image in it: the prompt's keys and values
are cached once, each answer's own behind them.

    python examples/shared_prompt.py

The prompt (text, the patches of a picture by row and column, text): lookup in an
INT8 table -> residual addition + norm -> projection -> norm + rotation by three
axes + append -> prompt attention; then one token of every answer at a time, its
attention over the shared prefix and its own rows, its logits scored: the log
probability of the token that was drawn, the entropy and the likeliest tokens.
Every step is compared with plain torch operations in fp32 on the same weights.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import int4_row_wise_amd as q  # noqa: E402

VOCAB, WIDTH = 4000, 512
Q_HEADS, KV_HEADS, DIM = 8, 2, 64
PAGE = 16
SECTIONS = (12, 10, 10)  # pairs of a head that turn by time, height and width
EPS = 1e-6
DEV = "cuda"


def prompt_positions(before: int, rows: int, cols: int, after: int) -> torch.Tensor:
    """[3, tokens]: text advances on all axes alike, a picture stands at one time and
    spreads over height and width, and what follows goes on behind the largest."""
    text = torch.arange(before)
    patch = torch.arange(rows * cols)
    picture = torch.stack((torch.full_like(patch, before), before + patch // cols, before + patch % cols))
    rest = before + max(rows, cols) + torch.arange(after)
    return torch.cat((text.expand(3, -1), picture, rest.expand(3, -1)), 1).to(torch.int32).to(DEV)


def plain_norm(x, gain):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.float()


def plain_turn(x, gain, cos_sin, positions, axes):
    """Norm and rotation of [n, heads, DIM] in fp32."""
    x = plain_norm(x, gain)
    where = positions.long()[axes.long()].t()  # [n, pairs]
    pair = torch.arange(DIM // 2, device=DEV)
    cos, sin = cos_sin[where, pair][:, None], cos_sin[where, DIM // 2 + pair][:, None]
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def plain_attention(x, k, v):
    """x [Hq, d] over k, v [n, Hkv, d], in fp32."""
    g = Q_HEADS // KV_HEADS
    k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    w = torch.softmax((k * x).sum(-1) * DIM ** -0.5, 0)
    return (w[..., None] * v).sum(0)


def main(answers: int = 12, steps: int = 6, seed: int = 0, verbose: bool = True) -> dict:
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def weights(*shape, scale):
        return (torch.randn(shape, generator=g, device=DEV) * scale).bfloat16()

    table = q.quantize_rowwise(torch.randn((VOCAB, WIDTH), generator=g, device=DEV), 8)
    w_qkv = weights(WIDTH, (Q_HEADS + 2 * KV_HEADS) * DIM, scale=WIDTH ** -0.5)
    w_out, head = weights(Q_HEADS * DIM, WIDTH, scale=WIDTH ** -0.5), weights(WIDTH, VOCAB, scale=2 * WIDTH ** -0.5)
    gain_in, gain_out = (1 + weights(WIDTH, scale=0.1) for _ in range(2))
    gain_q, gain_k = (1 + weights(DIM, scale=0.1) for _ in range(2))
    angle = torch.arange(512, device=DEV)[:, None] * 10000.0 ** (-torch.arange(0, DIM, 2, device=DEV) / DIM)
    cos_sin = torch.cat((angle.cos(), angle.sin()), 1).contiguous()
    axes = q.rotary_axes(SECTIONS, in_turn=True, device=DEV)
    offsets = torch.tensor([0, VOCAB], device=DEV)
    errors = {"prompt": 0.0, "step": 0.0, "logprob": 0.0}

    def lookup(ids):
        n = ids.numel()
        return q.bag_forward(table, offsets, n, WIDTH, 8, ids, torch.arange(n + 1, device=DEV))[:, 0].bfloat16()

    def heads_of(x):
        """Normed and projected rows as strided q, k, v."""
        y, _, _ = q.add_norm(x, weight=gain_in, eps=EPS)
        return (y @ w_qkv).view(x.shape[0], -1, DIM).split((Q_HEADS, KV_HEADS, KV_HEADS), 1)

    def off(got, want):
        return float((got.float() - want).norm() / want.norm())

    # the prompt, once
    positions = prompt_positions(20, 6, 9, 11)
    n = positions.shape[1]
    own_pages = -(-steps // PAGE)
    pages = -(-n // PAGE) + answers * own_pages
    k_pages = torch.zeros((pages, KV_HEADS, PAGE, DIM), dtype=torch.bfloat16, device=DEV)
    v_pages = torch.zeros_like(k_pages)
    prefix = torch.arange(-(-n // PAGE), dtype=torch.int32, device=DEV)[None].contiguous()
    ids = torch.randint(0, VOCAB, (n,), generator=g, device=DEV)
    xq, xk, xv = heads_of(lookup(ids))
    k_out = torch.empty((n, KV_HEADS, DIM), dtype=xq.dtype, device=DEV)
    turned, _ = q.norm_rope(xq, xk, positions, cos_sin, gain_q, gain_k, eps=EPS, v=xv, k_pages=k_pages, v_pages=v_pages,
                            slots=torch.arange(n, device=DEV), k_out=k_out, pair_axes=axes)
    whole = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    out = q.prompt_attention(turned, k_out, xv, whole, whole, max_q=n)
    plain_k, plain_v = plain_turn(xk.float(), gain_k, cos_sin, positions, axes), xv.float()
    plain_q = plain_turn(xq.float(), gain_q, cos_sin, positions, axes)
    errors["prompt"] = off(out[-1], plain_attention(plain_q[-1], plain_k, plain_v))

    # every answer, a token at a time
    tables = prefix.shape[1] + torch.arange(answers * own_pages, dtype=torch.int32, device=DEV).view(answers, own_pages)
    own_k, own_v = [[] for _ in range(answers)], [[] for _ in range(answers)]
    length = torch.tensor([n], dtype=torch.int32, device=DEV)
    ids = torch.randint(0, VOCAB, (answers,), generator=g, device=DEV)
    last, scores = int(positions.max()), torch.zeros(answers, device=DEV)
    for step in range(steps):
        x = lookup(ids)
        xq, xk, xv = heads_of(x)
        at = torch.full((3, answers), last + 1 + step, dtype=torch.int32, device=DEV)
        slots = tables[:, step // PAGE].long() * PAGE + step % PAGE
        turned, _ = q.norm_rope(xq, xk, at, cos_sin, gain_q, gain_k, eps=EPS, v=xv, k_pages=k_pages, v_pages=v_pages, slots=slots, pair_axes=axes)
        lens = torch.full((answers,), step + 1, dtype=torch.int32, device=DEV)
        out = q.shared_attention(turned, k_pages, v_pages, prefix, length, tables, lens)
        delta = out.view(answers, -1) @ w_out
        y, x, _ = q.add_norm(delta, x, gain_out, eps=EPS)
        logits = y @ head
        drawn = torch.multinomial(torch.softmax(logits.float(), -1), 1, generator=g)[:, 0]
        logprobs, entropy, top_ids, top_logprobs = q.token_logprobs(logits, drawn, top=4)

        new_q, new_k = (plain_turn(t.float(), w, cos_sin, at, axes) for t, w in ((xq, gain_q), (xk, gain_k)))
        for b in range(answers):
            own_k[b].append(new_k[b:b + 1])
            own_v[b].append(xv[b:b + 1].float())
            want = plain_attention(new_q[b], torch.cat([plain_k] + own_k[b]), torch.cat([plain_v] + own_v[b]))
            errors["step"] = max(errors["step"], off(out[b], want))
        every = torch.log_softmax(logits.float(), -1)
        errors["logprob"] = max(errors["logprob"], float((every.gather(1, drawn[:, None])[:, 0] - logprobs).abs().max()),
                                float((every.gather(1, top_ids.long()) - top_logprobs).abs().max()),
                                float((-(every.exp() * every).sum(-1) - entropy).abs().max()))
        scores += logprobs
        ids = drawn
    torch.cuda.synchronize()
    if verbose:
        print("relative error: prompt attention %.2g, steps over the shared prefix %.2g; log probabilities off by %.2g" % (
            errors["prompt"], errors["step"], errors["logprob"]))
        print("%d answers of %d tokens, the likeliest of log probability %.2f" % (answers, steps, float(scores.max())))
    return {"errors": errors, "scores": scores.tolist(), "top": top_ids.tolist()}


if __name__ == "__main__":
    main()
