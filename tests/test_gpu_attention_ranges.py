"""Attention on the GPU at the ends of its arguments' ranges, against float64:
windows and sinks up to 2^31 - 1, scales, strides that are never used, and sizes
that reach every dispatched kernel (bounds and formulas: attention_model.py)."""
from __future__ import annotations

import numpy as np
import pytest

from tests import attention_model as model
from tests.gpu_common import host
from tests.test_gpu_attention import Cache, check_decode, check_prompt, close, f64, q, rand16, rope_table  # noqa: F401

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("window", [2 ** 30, MOST - 6, MOST])
@pytest.mark.parametrize("nq,nk", [(10, 5), (300, 70), (5, 10)])
def test_prompt_window_past_every_key(q, d, window, nq, nk):
    """A window wider than the cache hides nothing, also where the first queries see no key."""
    g = np.random.default_rng(2000 + nq + d)
    check_prompt(q, g, [nq, 4], [nk, 4], 2, 1, d, "bf16", window, 0)
    check_prompt(q, g, [nq, 4], [nk, 4], 2, 1, d, "bf16", window, 3)


@pytest.mark.parametrize("d", [64, 200])
@pytest.mark.parametrize("window", [1, 40])
@pytest.mark.parametrize("sinks", [MOST - 33, MOST - 30, MOST])
def test_prompt_sinks_past_every_key(q, d, window, sinks):
    """More sinks than keys: a window hides nothing."""
    g = np.random.default_rng(2100 + d)
    check_prompt(q, g, [200, 30], [200, 90], 2, 1, d, "bf16", window, sinks)


def test_prompt_small_scale(q):
    """Products of 2^100 and a scale of 2^-103."""
    import torch
    g = np.random.default_rng(2200)
    n, d, scale = 90, 64, 2.0 ** -103
    (qt, qv), (kt, kv), (vt, vv) = (rand16(g, (n, 1, d), "bf16", s) for s in (2.0 ** 50, 2.0 ** 50, 1.0))
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out = f64(q.prompt_attention(qt, kt, vt, off, off, scale=scale))
    for i in range(n):
        o, ob, *_ = model.attend(qv[i, 0], kv[:, 0], vv[:, 0], model.visible(i, n, 0, 0), scale, "bf16")
        close(out[i, 0], o, ob, "row %d" % i)


def odd(t, dim, stride):
    """t with an odd stride along a dimension of size 1."""
    strides = list(t.stride())
    assert t.shape[dim] == 1
    strides[dim] = stride
    return t.as_strided(t.shape, strides)


def test_stride_of_one_token_or_head_is_not_used(q):
    import torch
    g = np.random.default_rng(2300)
    qt, _ = rand16(g, (1, 3, 64), "bf16")
    kt, _ = rand16(g, (1, 1, 64), "bf16")
    vt, _ = rand16(g, (1, 1, 64), "bf16")
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    pos, cs = torch.tensor([7], dtype=torch.int32, device="cuda"), torch.from_numpy(rope_table(10, 64)).cuda()
    pages = [torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    slot = torch.zeros(1, dtype=torch.int64, device="cuda")
    want = q.prompt_attention(qt, kt, vt, off, off)
    want_q, _ = q.norm_rope(qt, kt, pos, cs, v=vt, k_pages=pages[0], v_pages=pages[1], slots=slot)
    for stride in (5, 1 << 40):
        qs, ks, vs = odd(qt, 0, stride), odd(odd(kt, 0, stride), 1, 3), odd(odd(vt, 0, 1), 1, stride)
        assert torch.equal(q.prompt_attention(qs, ks, vs, off, off), want)
        got_q, _ = q.norm_rope(qs, ks, pos, cs, v=vs, k_pages=pages[2], v_pages=pages[3], slots=slot)
        assert torch.equal(got_q, want_q)
        assert torch.equal(pages[2], pages[0]) and torch.equal(pages[3], pages[1])


def test_numbers_past_32_bits_are_refused(q):
    """An argument that a 32-bit integer does not hold is refused, not cut."""
    import torch
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    pages = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    lens = torch.ones(4, dtype=torch.int32, device="cuda")
    mass = torch.zeros((4, 2, 16), device="cuda")
    for n in (2 ** 31, 2 ** 32 + 2, 2 ** 63 - 1, -2 ** 32):
        for name in ("window", "sinks"):
            with pytest.raises(ValueError):
                q.prompt_attention(x, x, x, off, off, **{name: n})
            with pytest.raises(ValueError):
                q.decode_attention(x, pages, pages, table, lens, **{name: n})
            with pytest.raises(ValueError):
                q.decode_workspace_bytes(4, 2, 2, 64, 1, 16, **{name: n})
        with pytest.raises(ValueError):
            q.evict(pages, pages, table, lens, mass, n, pages, pages, table)


# ---- scales ----

SCALES = [0.05, 0.7, -0.125, 0.0]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("window", [0, 30])
def test_prompt_scale(q, scale, window):
    """A caller's scale, also in rows that are computed again (a NaN value that they do not see)."""
    import torch
    g = np.random.default_rng(2400)
    n, hq, hkv, d, at = 150, 4, 2, 64, 100
    (qt, qv), (kt, kv), (vt, vv) = (rand16(g, (n, h, d), "bf16") for h in (hq, hkv, hkv))
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lse = torch.zeros((n, hq), device="cuda")
    bad = vt.clone()
    bad[at] = float("nan")
    clean = f64(q.prompt_attention(qt, kt, vt, off, off, scale=scale, window=window, sinks=1, lse=lse))
    again = f64(q.prompt_attention(qt, kt, bad, off, off, scale=scale, window=window, sinks=1))
    for i in range(n):
        see = model.visible(i, n, window, 1)
        for h in range(hq):
            o, ob, ls, lb, *_ = model.attend(qv[i, h], kv[:, h // 2], vv[:, h // 2], see, scale, "bf16")
            close(clean[i, h], o, ob, "row %d head %d" % (i, h))
            close(f64(lse)[i, h], ls, lb, "lse of row %d head %d" % (i, h))
            if not see[at]:
                close(again[i, h], o, ob, "row %d head %d beside a NaN" % (i, h))
            else:
                assert np.isnan(again[i, h]).all()


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("bits", [16, 8, 4])
def test_decode_scale(q, bits, scale):
    import torch
    g = np.random.default_rng(2410 + bits)
    cache = Cache(g, q, [1, 70, 333], 2, 64, bits, 16, "fp16")
    qt, qv = rand16(g, (3, 6, 64), "fp16")
    lse, mass = torch.zeros((3, 6), device="cuda"), torch.zeros((3, 2, 333), device="cuda")
    out = f64(q.decode_attention(qt, cache.pool[0], cache.pool[1], cache.table, cache.seq_lens, bits=bits, scale=scale, lse=lse, mass=mass))
    for b, n in enumerate(cache.lens):
        want, bound = np.zeros((2, n)), np.zeros((2, n))
        for h in range(6):
            (k, kr), (v, vr) = cache.rows(0, b, h // 3), cache.rows(1, b, h // 3)
            o, ob, ls, lb, w, wb = model.attend(qv[b, h], k, v, np.ones(n, bool), scale, "fp16", kr, vr)
            close(out[b, h], o, ob, "sequence %d head %d" % (b, h))
            close(f64(lse)[b, h], ls, lb, "lse of sequence %d head %d" % (b, h))
            want[h // 3] += w
            bound[h // 3] += wb + 2.0 ** -22 * w
        close(f64(mass)[b, :, :n], want, bound, "mass of sequence %d" % b)


# ---- every kernel that a call can reach ----

@pytest.mark.parametrize("bits", [16, 8, 4])
def test_decode_more_chunks_than_lanes(q, bits):
    """66 chunks a head: the join's statistics take a second turn of the wave."""
    g = np.random.default_rng(2500)
    cache = Cache(g, q, [33500, 40], 1, 64, bits, 64, "bf16")
    check_decode(q, g, cache, 2, "bf16", mass=True, q_scale=2.0)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1100, 3)])
def test_decode_chunks_of_a_wide_table(q, bits, window, sinks):
    """64 sequences in tables for 16384 slots: chunks of 2048 keys (and, through the window, of 512)."""
    g = np.random.default_rng(2510)
    lens = [4500, 2049, 2048, 2047, 1104, 1103, 0] + [5] * 57
    cache = Cache(g, q, lens, 8, 64, bits, 16, "bf16", width=1024)
    check_decode(q, g, cache, 8, "bf16", window, sinks, mass=True)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("hq", [64, 65, 150])
def test_decode_many_heads_with_mass(q, bits, hq):
    """The mass of a group of more than 64 query heads is summed in several turns."""
    g = np.random.default_rng(2520)
    check_decode(q, g, Cache(g, q, [600, 33, 1], 1, 64, bits, 16, "bf16"), hq, "bf16", mass=True)


@pytest.mark.parametrize("slots,keep,sinks,recent", [(8193, 2000, 4, 100), (12000, 5000, 0, 0), (16384, 1, 0, 0), (16385, 9000, 3, 500),
                                                     (20000, 700, 0, 650), (32768, 32767, 1, 1), (32769, 4000, 4, 0)])
def test_evict_every_length(q, slots, keep, sinks, recent):
    """Eviction around the numbers of slots that a thread holds, with many ties."""
    import torch
    g = np.random.default_rng(2600 + slots)
    lens = [slots, slots - 1, keep + 1]
    cache = Cache(g, q, lens, 1, 8, 16, 64, "bf16")
    mass = (g.integers(0, 40, (len(lens), 1, slots)) / 8.0).astype(np.float32)
    mass[0, 0, ::97] = np.nan
    new_width = -(-keep // 64)
    new = [torch.zeros((len(lens) * new_width,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda") for t in cache.pool]
    table = torch.arange(len(lens) * new_width, dtype=torch.int32, device="cuda").view(len(lens), new_width)
    kept, m, n = q.evict(cache.pool[0], cache.pool[1], cache.table, cache.seq_lens, torch.from_numpy(mass).cuda(), keep, new[0], new[1], table,
                         sinks=sinks, recent=recent)
    assert host(n).tolist() == [keep] * 3
    for b, length in enumerate(lens):
        ids = np.array(model.evict_ids(mass[b, 0], length, keep, sinks, recent))
        assert np.array_equal(host(kept)[b, 0], ids), b
        assert np.array_equal(host(m)[b, 0], mass[b, 0, ids], equal_nan=True)
        for side in range(2):
            rows = new[side][table[b].long(), 0].reshape(-1, 8)[:keep]
            assert np.array_equal(f64(rows), cache.rows(side, b, 0)[0][ids])


# ---- what packed rows cost in accuracy ----

@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d", [64, 128, 200])
def test_decode_packed_rows_bf16_output(q, bits, d):
    """Packed rows meet weights of binary16 whatever the queries' type, so a bf16
    output is within binary16's bound and its own last rounding."""
    g = np.random.default_rng(2700 + bits + d)
    lens = [3, 90, 700]
    cache = Cache(g, q, lens, 2, d, bits, 16, "bf16")
    qt, qv = rand16(g, (len(lens), 8, d), "bf16")
    out = f64(q.decode_attention(qt, cache.pool[0], cache.pool[1], cache.table, cache.seq_lens, bits=bits))
    for b, n in enumerate(lens):
        for h in range(8):
            (k, kr), (v, vr) = cache.rows(0, b, h // 4), cache.rows(1, b, h // 4)
            o, ob, *_ = model.attend(qv[b, h], k, v, np.ones(n, bool), d ** -0.5, "fp16", kr, vr)
            close(out[b, h], o, ob + model.U["bf16"] * (np.abs(o) + ob), "sequence %d head %d" % (b, h))
