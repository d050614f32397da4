"""Attention over the paged cache on the GPU against float64 (bounds and
formulas: attention_model.py): prompts and one-token calls over 16-bit, INT8
and INT4 rows, windows, sinks, empty sequences, NaN and infinities where
nothing is visible, strides, streams and graphs."""
from __future__ import annotations

import numpy as np
import pytest

from tests import attention_model as model
from tests.gpu_common import host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    lib = require_gpu()
    from int4_row_wise_amd import build
    build.ensure_built()
    lib.load_attention_library()
    return lib


def torch_type(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def rand16(g, shape, dtype, scale=1.0):
    """Normal values of the 16-bit type on the GPU, and their float64 values."""
    import torch
    t = torch.from_numpy((g.standard_normal(shape) * scale).astype(np.float32)).to(torch_type(dtype))
    return t.cuda(), t.double().numpy()


def f64(t):
    return t.detach().cpu().double().numpy()


def close(got, want, bound, what):
    bad = ~(np.abs(got - want) <= bound)
    bad &= ~((got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), "%s: %d of %d outside, worst %g against %g" % (
        what, bad.sum(), bad.size, np.abs(got - want)[bad].max(), bound[bad].min() if np.ndim(bound) else bound)


class Cache:
    """A paged cache of random rows with its float64 values: k, v [B][n, Hkv, d]."""

    def __init__(self, g, lib, lens, hkv, d, bits, page, dtype, width=None, spread=1.0):
        import torch
        need = [-(-n // page) for n in lens]
        self.page, self.bits, self.d, self.hkv, self.lens = page, bits, d, hkv, lens
        pages = max(1, sum(need)) + 2  # two that nobody owns
        order = g.permutation(pages)
        self.width = width if width is not None else max(1, max(need, default=1))
        table = np.full((len(lens), self.width), -7, np.int32)  # unused entries are garbage
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table_np = table
        self.table = torch.from_numpy(table).cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32).cuda()
        self.pool, self.values, self.ranges = [], [], []
        for _ in range(2):
            if bits == 16:
                t, val = rand16(g, (pages, hkv, page, d), dtype, spread)
                rng = np.zeros((pages, hkv, page))
            else:
                x = torch.from_numpy((g.standard_normal((pages * hkv * page, d)) * spread + 0.3).astype(np.float32)).cuda()
                t = lib.quantize_rowwise(x, bits).view(pages, hkv, page, -1)
                val, rng = model.unpack_rows(host(t), d, bits)
            self.pool.append(t)
            self.values.append(val)
            self.ranges.append(rng)

    def rows(self, side, b, h):
        n = self.lens[b]
        j = np.arange(n)
        page = self.table_np[b, j // self.page] if n else np.zeros(0, int)
        return self.values[side][page, h, j % self.page], self.ranges[side][page, h, j % self.page]

    def poison_unowned(self, value):
        """Overwrites every row that no sequence owns (page ends, free pages)."""
        import torch
        owned = np.zeros(self.values[0].shape[:1] + (self.page,), bool)
        for b, n in enumerate(self.lens):
            j = np.arange(n)
            owned[self.table_np[b, j // self.page], j % self.page] = True
        mask = torch.from_numpy(~owned).cuda()
        for t in self.pool:
            t.permute(0, 2, 1, 3)[mask] = value


def check_decode(lib, g, cache, hq, dtype, window=0, sinks=0, mass=False, q_scale=1.0, what=""):
    import torch
    b, d, group = len(cache.lens), cache.d, hq // cache.hkv
    qt, qv = rand16(g, (b, hq, d), dtype, q_scale)
    lse = torch.full((b, hq), 7.0, device="cuda")
    m0 = g.random((b, cache.hkv, max(1, max(cache.lens)))).astype(np.float32) if mass else None
    mt = torch.from_numpy(m0.copy()).cuda() if mass else None
    out = lib.decode_attention(qt, cache.pool[0], cache.pool[1], cache.table, cache.seq_lens, bits=cache.bits, window=window,
                               sinks=sinks, mass=mt, lse=lse)
    torch.cuda.synchronize()
    got, got_lse = f64(out), f64(lse)
    for i, n in enumerate(cache.lens):
        see = model.visible(n - 1, n, window, sinks)
        want_mass = m0[i].astype(np.float64) if mass else None
        mass_bound = np.abs(m0[i]) * 2.0 ** -22 if mass else None
        for h in range(hq):
            (k, kr), (v, vr) = cache.rows(0, i, h // group), cache.rows(1, i, h // group)
            o, ob, ls, lb, w, wb = model.attend(qv[i, h], k, v, see, d ** -0.5, dtype, kr, vr)
            close(got[i, h], o, ob, "%s out of sequence %d (length %d) head %d" % (what, i, n, h))
            close(got_lse[i, h], ls, lb, "%s lse of sequence %d head %d" % (what, i, h))
            if mass:
                want_mass[h // group, :n] += w
                mass_bound[h // group, :n] += wb + 2.0 ** -22 * w
        if mass:
            close(f64(mt)[i], want_mass, mass_bound, "%s mass of sequence %d" % (what, i))
    return out


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [8, 40, 64, 96, 128, 200, 256])
def test_decode_dims(q, bits, dtype, d):
    g = np.random.default_rng(100 + d + bits)
    cache = Cache(g, q, [1, 0, 7, 33, 130, 517], 2, d, bits, 16, dtype)
    check_decode(q, g, cache, 6, dtype, mass=True)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("heads", [(1, 1), (8, 8), (5, 1), (32, 4), (17, 1), (40, 2)])
def test_decode_heads(q, bits, heads):
    g = np.random.default_rng(200 + bits)
    cache = Cache(g, q, [65, 300, 2], heads[1], 64, bits, 32, "bf16")
    check_decode(q, g, cache, heads[0], "bf16", mass=True)


@pytest.mark.parametrize("page", [1, 2, 8, 16, 64, 256])
@pytest.mark.parametrize("bits", [16, 4])
def test_decode_pages_that_end_inside_a_tile(q, page, bits):
    g = np.random.default_rng(300 + page)
    lens = [page - 1, page, page + 1, 3 * page + 5, 31, 32, 33, 64, 65, 127, 128, 129]
    check_decode(q, g, Cache(g, q, lens, 2, 128, bits, page, "bf16"), 8, "bf16", mass=True)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (16, 0), (50, 3), (128, 1), (1000, 7), (100, 5000)])
def test_decode_windows(q, bits, window, sinks):
    g = np.random.default_rng(400 + window + sinks)
    cache = Cache(g, q, [0, 1, 15, 16, 17, 50, 53, 54, 200, 1003, 2001], 2, 64, bits, 16, "fp16")
    check_decode(q, g, cache, 4, "fp16", window, sinks, mass=True)


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_decode_long_split(q, bits):
    g = np.random.default_rng(500)
    cache = Cache(g, q, [20011, 3], 1, 128, bits, 64, "bf16")
    check_decode(q, g, cache, 4, "bf16", mass=True, q_scale=2.0)


@pytest.mark.parametrize("spread", [1e-3, 30.0])
def test_decode_flat_and_peaked(q, spread):
    """Scores all alike, and scores of hundreds where one key takes all."""
    g = np.random.default_rng(510)
    for bits in (16, 8, 4):
        check_decode(q, g, Cache(g, q, [700, 90], 2, 64, bits, 16, "bf16", spread=spread), 8, "bf16", mass=True, what="%d bits" % bits)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_decode_ignores_rows_that_are_not_visible(q, bits, poison):
    """Page ends and free pages full of NaN or infinities change nothing."""
    g = np.random.default_rng(520)
    cache = Cache(g, q, [1, 5, 17, 100, 0, 259], 2, 128, bits, 16, "bf16")
    cache.poison_unowned(poison if bits == 16 else 0xff)  # 0xffff: a NaN as scale and bias
    check_decode(q, g, cache, 8, "bf16", mass=True)


def test_decode_window_hides_nan(q):
    """Keys before the window hold NaN; the result is the clean one."""
    import torch
    g = np.random.default_rng(530)
    cache = Cache(g, q, [500], 1, 64, 16, 16, "bf16")
    for side in range(2):
        j = np.arange(2, 500 - 100)  # neither sink nor window
        page = torch.from_numpy(cache.table_np[0, j // 16].astype(np.int64)).cuda()
        cache.pool[side][page, 0, torch.from_numpy(j % 16).cuda()] = float("nan")
    check_decode(q, g, cache, 4, "bf16", window=100, sinks=2, mass=True)


def test_decode_infinite_scores(q):
    """A visible key of -inf score has no weight; all of them: zeros."""
    import torch
    g = np.random.default_rng(540)
    cache = Cache(g, q, [40], 1, 64, 16, 16, "bf16")
    qt = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    cache.pool[0][int(cache.table_np[0, 0]), 0, 3] = float("-inf")
    out = q.decode_attention(qt, cache.pool[0], cache.pool[1], cache.table, cache.seq_lens)
    k, v = cache.rows(0, 0, 0)[0].copy(), cache.rows(1, 0, 0)[0]
    see = np.ones(40, bool)
    see[3] = False
    o, ob, *_ = model.attend(np.ones(64), k, v, see, 0.125, "bf16")
    close(f64(out)[0, 0], o, ob, "one infinite score")
    cache.pool[0].fill_(float("-inf"))
    lse = torch.zeros((1, 1), device="cuda")
    out = q.decode_attention(qt, cache.pool[0], cache.pool[1], cache.table, cache.seq_lens, lse=lse)
    assert (f64(out) == 0).all() and f64(lse)[0, 0] == -np.inf


def test_decode_visible_nan_is_seen(q):
    """A NaN in a visible value reaches its element and no other."""
    g = np.random.default_rng(550)
    cache = Cache(g, q, [40], 1, 64, 16, 16, "bf16")
    cache.pool[1][int(cache.table_np[0, 1]), 0, 2, 5] = float("nan")
    qt, _ = rand16(g, (1, 2, 64), "bf16")
    out = f64(q.decode_attention(qt, cache.pool[0], cache.pool[1], cache.table, cache.seq_lens))
    assert np.isnan(out[:, :, 5]).all() and np.isfinite(np.delete(out, 5, 2)).all()


def test_decode_bad_data_is_counted(q):
    import torch
    g = np.random.default_rng(560)
    cache = Cache(g, q, [40, 40, 40], 2, 64, 16, 16, "bf16")
    qt, qv = rand16(g, (3, 4, 64), "bf16")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.tensor([-1, 49, 40], dtype=torch.int32, device="cuda")
    lse = torch.zeros((3, 4), device="cuda")
    table = cache.table.clone()
    table[2, 1] = cache.pool[0].shape[0]  # past the cache: slots 16..31 are not visible
    mass = torch.zeros((3, 2, 48), device="cuda")
    out = f64(q.decode_attention(qt, cache.pool[0], cache.pool[1], table, lens, mass=mass, lse=lse, err_count=err))
    assert (out[:2] == 0).all() and (f64(lse)[:2] == -np.inf).all() and (f64(mass)[:2] == 0).all()
    assert int(err[0]) >= 3
    see = np.ones(40, bool)
    see[16:32] = False
    for h in range(4):
        o, ob, *_ = model.attend(qv[2, h], cache.rows(0, 2, h // 2)[0], cache.rows(1, 2, h // 2)[0], see, 0.125, "bf16")
        close(out[2, h], o, ob, "bad page, head %d" % h)
    assert (f64(mass)[2, :, 16:32] == 0).all()


def test_decode_mass_repeats_and_adds(q):
    """Two calls add twice the weight, and equal inputs give equal bits."""
    import torch
    g = np.random.default_rng(570)
    cache = Cache(g, q, [900, 300], 2, 64, 8, 16, "bf16")
    qt, _ = rand16(g, (2, 8, 64), "bf16")
    runs = []
    for _ in range(2):
        mass = torch.zeros((2, 2, 900), device="cuda")
        a = q.decode_attention(qt, cache.pool[0], cache.pool[1], cache.table, cache.seq_lens, bits=8, mass=mass)
        first = mass.clone()
        b = q.decode_attention(qt, cache.pool[0], cache.pool[1], cache.table, cache.seq_lens, bits=8, mass=mass)
        assert torch.equal(a, b) and torch.equal(mass, first + first)
        assert abs(float(first.double().sum()) - 16) < 1e-3
        runs.append((a, mass))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])


def test_decode_page_table_past_2_31_bytes(q):
    """A cache of 4.3 GB a side: rows beyond 32-bit byte offsets."""
    import torch
    pages, page, d = 2 ** 16 + 40, 256, 128
    g = np.random.default_rng(580)
    k = torch.zeros((pages, 1, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    ids = [pages - 1, 3, pages - 30]
    kt, kv = rand16(g, (3, 1, page, d), "bf16")
    vt, vv = rand16(g, (3, 1, page, d), "bf16")
    for i, p in enumerate(ids):
        k[p], v[p] = kt[i], vt[i]
    qt, qv = rand16(g, (1, 2, d), "bf16")
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    lens = torch.tensor([700], dtype=torch.int32, device="cuda")
    out = f64(q.decode_attention(qt, k, v, table, lens))
    for h in range(2):
        o, ob, *_ = model.attend(qv[0, h], kv.reshape(-1, d)[:700], vv.reshape(-1, d)[:700], np.ones(700, bool), d ** -0.5, "bf16")
        close(out[0, h], o, ob, "head %d" % h)


# ---- prompts ----

def check_prompt(lib, g, nqs, nks, hq, hkv, d, dtype, window=0, sinks=0, strided=False, max_q=0, rows=None, spread=1.0):
    import torch
    tq, tk = sum(nqs), sum(nks)
    if strided:  # slices of one fused projection (queries and keys alike in number)
        assert nqs == nks
        t, val = rand16(g, (tq, hq + 2 * hkv, d), dtype, spread)
        (qt, kt, vt), (qv, kv, vv) = t.split((hq, hkv, hkv), 1), np.split(val, (hq, hq + hkv), 1)
    else:
        (qt, qv), (kt, kv), (vt, vv) = (rand16(g, (n, h, d), dtype, spread) for n, h in ((tq, hq), (tk, hkv), (tk, hkv)))
    qo, ko = np.concatenate(([0], np.cumsum(nqs))), np.concatenate(([0], np.cumsum(nks)))
    lse = torch.full((tq, hq), 7.0, device="cuda")
    out = lib.prompt_attention(qt, kt, vt, torch.tensor(qo, dtype=torch.int32).cuda(), torch.tensor(ko, dtype=torch.int32).cuda(),
                               window=window, sinks=sinks, lse=lse, max_q=max_q)
    torch.cuda.synchronize()
    got, got_lse = f64(out), f64(lse)
    for b, (nq, nk) in enumerate(zip(nqs, nks)):
        some = range(nq) if rows is None else sorted({int(r) for r in g.integers(0, nq, rows)} | {0, nq - 1}) if nq else []
        for i in some:
            see = model.visible(i + nk - nq, nk, window, sinks)
            for h in range(hq):
                ks, hk = slice(ko[b], ko[b + 1]), h // (hq // hkv)
                o, ob, ls, lb, *_ = model.attend(qv[qo[b] + i, h], kv[ks, hk], vv[ks, hk], see, d ** -0.5, dtype)
                close(got[qo[b] + i, h], o, ob, "sequence %d row %d head %d" % (b, i, h))
                close(got_lse[qo[b] + i, h], ls, lb, "lse of sequence %d row %d head %d" % (b, i, h))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [8, 40, 64, 96, 128, 200, 256])
def test_prompt_dims(q, dtype, d):
    g = np.random.default_rng(600 + d)
    check_prompt(q, g, [1, 0, 5, 33, 130], [1, 0, 5, 33, 130], 4, 2, d, dtype)


@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (8, 1), (12, 4)])
def test_prompt_heads_and_strides(q, heads):
    g = np.random.default_rng(610)
    check_prompt(q, g, [70, 200], [70, 200], *heads, 64, "bf16", strided=True)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257])
def test_prompt_lengths(q, n):
    g = np.random.default_rng(620 + n)
    check_prompt(q, g, [n], [n], 2, 1, 128, "bf16")


@pytest.mark.parametrize("nq,nk", [(1, 300), (5, 64), (64, 65), (100, 333), (128, 1000)])
def test_prompt_after_a_prefix(q, nq, nk):
    g = np.random.default_rng(630 + nq)
    check_prompt(q, g, [nq, 3], [nk, 9], 4, 2, 64, "bf16")


@pytest.mark.parametrize("nq,nk", [(10, 0), (200, 50), (129, 128), (3, 1)])
def test_prompt_rows_without_a_key(q, nq, nk):
    """More queries than keys: the first ones see nothing."""
    g = np.random.default_rng(640 + nq)
    check_prompt(q, g, [nq, 4], [nk, 4], 2, 2, 64, "bf16")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (50, 2), (64, 64), (100, 70), (200, 1), (1000, 4)])
def test_prompt_windows(q, window, sinks):
    g = np.random.default_rng(650 + window + sinks)
    check_prompt(q, g, [300, 40], [300, 140], 2, 1, 64, "fp16", window, sinks)


def test_prompt_long(q):
    g = np.random.default_rng(660)
    check_prompt(q, g, [2500], [2500], 2, 1, 128, "bf16", rows=40)
    check_prompt(q, g, [2500, 700], [2600, 700], 2, 1, 128, "bf16", 333, 5, rows=40)


@pytest.mark.parametrize("spread", [1e-3, 8.0])
def test_prompt_flat_and_peaked(q, spread):
    g = np.random.default_rng(670)
    check_prompt(q, g, [300], [300], 2, 2, 64, "bf16", spread=spread)


def test_prompt_max_q_is_only_a_hint(q):
    g = np.random.default_rng(680)
    check_prompt(q, g, [300, 10], [300, 10], 2, 2, 64, "bf16", max_q=1)


def test_prompt_neighbours_full_of_nan(q):
    """Sequences beside NaN rows: nothing leaks over an end."""
    import torch
    g = np.random.default_rng(690)
    n, d = 75, 128
    (qt, qv), (kt, kv), (vt, vv) = (rand16(g, (3 * n, 2, d), "bf16") for _ in range(3))
    for t in (qt, kt, vt):
        t[:n], t[2 * n:] = float("nan"), float("inf")
    off = torch.tensor([n, 2 * n], dtype=torch.int32, device="cuda")
    out = torch.full((3 * n, 2, d), 5.0, dtype=torch.bfloat16, device="cuda")
    q.prompt_attention(qt, kt, vt, off, off, out=out)
    got = f64(out)
    assert (got[:n] == 5).all() and (got[2 * n:] == 5).all()
    for i in range(n):
        for h in range(2):
            o, ob, *_ = model.attend(qv[n + i, h], kv[n:2 * n, h], vv[n:2 * n, h], model.visible(i, n, 0, 0), d ** -0.5, "bf16")
            close(got[n + i, h], o, ob, "row %d" % i)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
def test_prompt_later_rows_do_not_reach_earlier_ones(q, bad, where):
    """A NaN or an infinity in one key row leaves every query that does not see
    it as it was, bit for bit; one in a value row leaves it within the bounds (a
    row beside it is summed in another order); a window ends what it reaches."""
    import torch
    g = np.random.default_rng(700)
    n, d, at, window = 200, 64, 100, 60
    qt, qv = rand16(g, (n, 2, d), "bf16")
    kt, kv = rand16(g, (n, 1, d), "bf16")
    vt, vv = rand16(g, (n, 1, d), "bf16")
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for w in (0, window):
        clean = q.prompt_attention(qt, kt, vt, off, off, window=w)
        t = (kt if where == "k" else vt).clone()
        t[at, 0, 7] = bad
        got = q.prompt_attention(qt, t if where == "k" else kt, t if where == "v" else vt, off, off, window=w)
        last = at + w if w else n
        if where == "k":
            assert torch.equal(got[:at], clean[:at])
            assert torch.equal(got[last:], clean[last:])
        else:
            for i in [*range(at), *range(last, n)]:
                for h in range(2):
                    o, ob, *_ = model.attend(qv[i, h], kv[:, 0], vv[:, 0], model.visible(i, n, w, 0), d ** -0.5, "bf16")
                    close(f64(got[i, h]), o, ob, "row %d" % i)
            assert not torch.isfinite(got[at:last, :, 7]).any()
            keep = [i for i in range(d) if i != 7]
            assert torch.isfinite(got[at:last][:, :, keep]).all()


def test_prompt_bad_offsets_are_counted(q):
    import torch
    g = np.random.default_rng(710)
    qt, _ = rand16(g, (20, 2, 64), "bf16")
    kt, _ = rand16(g, (20, 2, 64), "bf16")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((20, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    qo = torch.tensor([0, 8, 4, 30, 20], dtype=torch.int32, device="cuda")  # falls, leaves, falls
    ko = torch.tensor([0, 8, 12, 16, 20], dtype=torch.int32, device="cuda")
    q.prompt_attention(qt, kt, kt, qo, ko, out=out, err_count=err)
    assert int(err[0]) == 3
    assert (f64(out)[8:] == 5).all() and not (f64(out)[:8] == 5).any()


# ---- norm, rotation, append ----

def rope_table(places, r):
    a = np.arange(places)[:, None] * 10000.0 ** (-np.arange(0, r, 2) / max(r, 1))
    return np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)


def norm_bound(want, x, w, eps, dtype, d):
    """One rounding to 16 bits, and binary32 sums of d squares and two products."""
    y = np.abs(x) / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.abs(w)
    return model.U[dtype] * np.abs(want) + (d + 16) * 2.0 ** -24 * 2 * y.max(-1, keepdims=True) + 2.0 ** -25


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,rot", [(8, 0), (16, 16), (40, 32), (64, 64), (96, 48), (128, 128), (200, 16), (256, 256)])
def test_norm_rope(q, interleaved, dtype, d, rot):
    import torch
    g = np.random.default_rng(800 + d)
    n, hq, hkv, eps = 13, 3, 2, 1e-5
    (qt, qv), (kt, kv) = rand16(g, (n, hq, d), dtype, 2.0), rand16(g, (n, hkv, d), dtype, 0.1)
    (wq, wqv), (wk, wkv) = rand16(g, (d,), dtype), rand16(g, (d,), dtype)
    table = rope_table(50, rot)
    pos = g.integers(0, 50, n)
    for index in (torch.int32, torch.int64):
        qo, ko = q.norm_rope(qt, kt, torch.from_numpy(pos).to(index).cuda(), torch.from_numpy(table).cuda(), wq, wk, eps=eps, interleaved=interleaved)
        for got, x, w in ((qo, qv, wqv), (ko, kv, wkv)):
            want = model.norm_rope(x, w, table[pos, :rot // 2].astype(np.float64), table[pos, rot // 2:].astype(np.float64), eps, interleaved)
            close(f64(got), want, norm_bound(want, x, w, eps, dtype, d), "norm")


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("d", [8, 64, 96, 128, 256])
def test_norm_rope_append(q, bits, d):
    """Rows land in their slots (and only there), from slices of a fused projection."""
    import torch
    g = np.random.default_rng(900 + d + bits)
    n, hq, hkv, page, pages = 21, 4, 2, 8, 5
    t, val = rand16(g, (n, hq + 2 * hkv, d), "bf16", 1.5)
    qt, kt, vt = t.split((hq, hkv, hkv), 1)
    kv, vv = val[:, hq:hq + hkv], val[:, hq + hkv:]
    rot = d // 16 * 16
    table = rope_table(64, rot)
    pos = np.arange(n)
    slots = g.permutation(pages * page)[:n]
    slots[3] = -1
    row = d if bits == 16 else q.row_stride(d, bits)
    kind = torch.bfloat16 if bits == 16 else torch.uint8
    pool = [torch.full((pages, hkv, page, row), 77, dtype=kind, device="cuda") for _ in range(2)]
    k_out = torch.zeros((n, hkv, d), dtype=torch.bfloat16, device="cuda")
    qo, ko = q.norm_rope(qt, kt, torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda(), v=vt, k_pages=pool[0], v_pages=pool[1],
                         slots=torch.from_numpy(slots).cuda(), bits=bits, k_out=k_out)
    assert ko is k_out
    cos, sin = (table[pos, s].astype(np.float64) for s in (slice(0, rot // 2), slice(rot // 2, rot)))
    want_k = model.norm_rope(kv, np.ones(d), cos, sin, 1e-6, False)
    close(f64(k_out), want_k, norm_bound(want_k, kv, np.ones(d), 1e-6, "bf16", d), "k_out")
    for side, want in ((0, want_k), (1, vv)):
        flat = pool[side].permute(0, 2, 1, 3).reshape(pages * page, hkv, row)
        free = np.setdiff1d(np.arange(pages * page), slots)
        assert (f64(flat.float())[free] == 77).all()
        used = slots >= 0
        rows = flat[torch.from_numpy(slots[used]).cuda()]
        if bits == 16:
            assert side == 0 or np.array_equal(f64(rows), want[used])
            close(f64(rows), want[used], norm_bound(want[used], kv[used], np.ones(d), 1e-6, "bf16", d), "rows")
            continue
        values, rng = model.unpack_rows(host(rows), d, bits)
        # half a step, the fp16 rounding of scale (at the last code) and bias, and binary32 before
        step = rng[..., None] / (2 ** bits - 1)
        bound = 0.5 * step * (1 + 2.0 ** -9) + 2.0 ** -11 * (rng[..., None] + np.abs(want[used]).max(-1, keepdims=True)) + (d + 16) * 2.0 ** -22 * np.abs(want[used]).max(-1, keepdims=True)
        close(values, want[used], np.broadcast_to(bound, values.shape), "packed rows")
        n_codes = d * bits // 8
        assert (host(rows)[..., n_codes + 4:] == 0).all()
        if side == 1:  # values are packed as the table quantizer packs them
            ref = q.quantize_rowwise(torch.from_numpy(want[used].astype(np.float32)).cuda().reshape(-1, d), bits)
            assert np.array_equal(host(ref), host(rows).reshape(-1, row))


def test_norm_rope_bad_data_is_counted(q):
    import torch
    g = np.random.default_rng(950)
    qt, _ = rand16(g, (4, 2, 64), "bf16")
    kt, _ = rand16(g, (4, 1, 64), "bf16")
    pool = [torch.full((2, 1, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, -1, 50, 3], dtype=torch.int32, device="cuda")
    slots = torch.tensor([1, 2, 3, 8], dtype=torch.int64, device="cuda")  # the last is past the cache
    qo, _ = q.norm_rope(qt, kt, pos, torch.from_numpy(rope_table(50, 64)).cuda(), v=kt, k_pages=pool[0], v_pages=pool[1], slots=slots, err_count=err)
    assert int(err[0]) == 3
    assert (f64(qo)[1:3] == 0).all() and not (f64(qo)[[0, 3]] == 0).all()
    for p in pool:
        flat = f64(p)[:, 0].reshape(8, 64)
        assert (np.delete(flat, 1, 0) == 7).all() and not (flat[1] == 7).all()


# ---- eviction ----

@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (40, 4, 10), (64, 64, 0), (64, 0, 64), (257, 3, 100), (2000, 4, 8)])
def test_evict(q, bits, keep, sinks, recent):
    import torch
    g = np.random.default_rng(1000 + keep + sinks)
    lens, hkv, d, page = [0, 1, 39, 40, 41, 300, 1500, 3000], 2, 64, 16
    cache = Cache(g, q, lens, hkv, d, bits, page, "bf16")
    mass = (g.integers(0, 50, (len(lens), hkv, 3000)) / 8.0).astype(np.float32)  # many ties
    mass[:, :, ::11] = -0.0
    mass[5:, 0, 20:60] = [np.nan, np.inf, -np.inf, -1.5] * 10
    new_width = -(-keep // page)
    pages = len(lens) * new_width + 1
    new = [torch.full((pages,) + tuple(t.shape[1:]), 3, dtype=t.dtype, device="cuda") for t in cache.pool]
    table = g.permutation(pages)[:len(lens) * new_width].reshape(len(lens), new_width).astype(np.int32)
    new_mass = torch.full((len(lens), hkv, keep + 5), 9.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, m, n = q.evict(cache.pool[0], cache.pool[1], cache.table, cache.seq_lens, torch.from_numpy(mass).cuda(), keep, new[0], new[1],
                         torch.from_numpy(table).cuda(), sinks=sinks, recent=recent, new_mass=new_mass, err_count=err)
    assert int(err[0]) == 0 and m is new_mass
    assert host(n).tolist() == [min(x, keep) for x in lens]
    for b, length in enumerate(lens):
        for h in range(hkv):
            ids = model.evict_ids(mass[b, h], length, keep, sinks, recent)
            assert host(kept)[b, h].tolist() == ids + [-1] * (keep - len(ids)), (b, h)
            want = np.zeros(keep + 5, np.float32)
            want[:len(ids)] = mass[b, h, ids]
            assert np.array_equal(host(m)[b, h], want, equal_nan=True)
            ids = np.array(ids, int)
            j = np.arange(len(ids))
            for side in range(2):
                old = cache.pool[side][torch.from_numpy(cache.table_np[b, ids // page].astype(np.int64)).cuda(), h, torch.from_numpy(ids % page).cuda()]
                to = new[side][torch.from_numpy(table[b, j // page].astype(np.int64)).cuda(), h, torch.from_numpy(j % page).cuda()]
                assert torch.equal(old, to)
                tail = np.arange(len(ids), new_width * page)  # slots past the kept rows stay as they were
                rest = new[side][torch.from_numpy(table[b, tail // page].astype(np.int64)).cuda(), h, torch.from_numpy(tail % page).cuda()]
                assert bool((rest == 3).all())


def test_evict_long(q):
    import torch
    g = np.random.default_rng(1100)
    n, keep = 40003, 9001
    cache = Cache(g, q, [n, 9002], 1, 8, 16, 64, "bf16")
    mass = np.exp(3 * g.standard_normal((2, 1, n))).astype(np.float32)
    new = [torch.zeros((300,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda") for t in cache.pool]
    table = torch.arange(2 * 141, dtype=torch.int32, device="cuda").view(2, 141)
    kept, _, _ = q.evict(cache.pool[0], cache.pool[1], cache.table, cache.seq_lens, torch.from_numpy(mass).cuda(), keep, new[0], new[1], table,
                         sinks=2, recent=500)
    for b, length in enumerate((n, 9002)):
        assert host(kept)[b, 0].tolist() == model.evict_ids(mass[b, 0], length, keep, 2, 500)


def test_evict_within_one_pool_and_bad_data(q):
    """The new pages may lie in the same arrays; bad lengths and pages are counted."""
    import torch
    g = np.random.default_rng(1110)
    cache = Cache(g, q, [60, 60], 1, 64, 16, 16, "bf16")
    pool = [torch.cat((t, torch.zeros((4,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda"))) for t in cache.pool]
    base = cache.pool[0].shape[0]
    table = torch.tensor([[base, base + 1], [base + 2, base + 4]], dtype=torch.int32, device="cuda")  # the last is past the arrays
    mass = torch.from_numpy(g.random((2, 1, 64)).astype(np.float32)).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, _, n = q.evict(pool[0], pool[1], cache.table, cache.seq_lens, mass, 20, pool[0], pool[1], table, recent=4, err_count=err)
    assert int(err[0]) == 4  # slots 16..19 of the second sequence
    ids = host(kept)[0, 0]
    assert ids.tolist() == model.evict_ids(host(mass)[0, 0], 60, 20, 0, 4)
    for side in range(2):
        old = cache.pool[side][torch.from_numpy(cache.table_np[0, ids // 16].astype(np.int64)).cuda(), 0, torch.from_numpy(ids % 16).cuda()]
        assert torch.equal(pool[side][base:base + 2, 0].reshape(32, 64)[:20], old)
    err.zero_()
    _, m, n = q.evict(pool[0], pool[1], cache.table, torch.tensor([-3, 65], dtype=torch.int32, device="cuda"), mass, 20, pool[0], pool[1], table, err_count=err)
    assert int(err[0]) == 2 and host(n).tolist() == [0, 0] and (host(m) == 0).all()


# ---- streams and graphs ----

def test_another_stream(q):
    import torch
    g = np.random.default_rng(1200)
    cache = Cache(g, q, [300, 77], 2, 64, 4, 16, "bf16")
    qt, _ = rand16(g, (2, 8, 64), "bf16")
    want = q.decode_attention(qt, cache.pool[0], cache.pool[1], cache.table, cache.seq_lens, bits=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = q.decode_attention(qt, cache.pool[0], cache.pool[1], cache.table, cache.seq_lens, bits=4)
    side.synchronize()
    assert torch.equal(got, want)


def test_captured_step_replays(q):
    """One decoding step (append, attention with mass, eviction) in a HIP graph,
    replayed on new inputs against eager calls, bit for bit."""
    import torch
    g = np.random.default_rng(1210)
    b, hq, hkv, d, page, bits = 3, 4, 2, 64, 16, 8
    cache = Cache(g, q, [200, 33, 120], hkv, d, bits, page, "bf16")
    S = cache.pool[0].shape[-1]
    x = torch.zeros((b, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(b, dtype=torch.int64, device="cuda")
    slots = torch.zeros(b, dtype=torch.int64, device="cuda")
    cos_sin = torch.from_numpy(rope_table(256, d)).cuda()
    table = torch.arange(b * 4, dtype=torch.int32, device="cuda").view(b, 4)

    def step(x, pos, slots, pool, mass, new):
        qt, kt, vt = x.split((hq, hkv, hkv), 1)
        qr, _ = q.norm_rope(qt, kt, pos, cos_sin, v=vt, k_pages=pool[0], v_pages=pool[1], slots=slots, bits=bits)
        out = q.decode_attention(qr, pool[0], pool[1], cache.table, cache.seq_lens, bits=bits, mass=mass)
        return (out, mass) + q.evict(pool[0], pool[1], cache.table, cache.seq_lens, mass, 64, new[0], new[1], table, sinks=2, recent=16)

    def fresh():
        return [t.clone() for t in cache.pool], torch.zeros((b, hkv, 256), device="cuda"), \
            [torch.zeros((b * 4, hkv, page, S), dtype=torch.uint8, device="cuda") for _ in range(2)]

    pool, mass, new = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, pos, slots, pool, mass, new)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(x, pos, slots, pool, mass, new)
    for t, c in zip(pool, cache.pool):
        t.copy_(c)
    mass.zero_()
    e_pool, e_mass, e_new = fresh()
    for rep in range(4):
        print("graph replay %d" % rep, flush=True)
        xt, _ = rand16(g, tuple(x.shape), "bf16")
        x.copy_(xt)
        last = [n - 1 for n in cache.lens]
        pos.copy_(torch.tensor(last) - rep)
        slots.copy_(torch.tensor([int(cache.table_np[i, n // page]) * page + n % page for i, n in enumerate(last)]))
        graph.replay()
        torch.cuda.synchronize()
        want = step(x.clone(), pos.clone(), slots.clone(), e_pool, e_mass, e_new)
        torch.cuda.synchronize()
        for a, w in zip(res, want):
            assert torch.equal(a, w), rep
        for a, w in zip(pool + new, e_pool + e_new):
            assert torch.equal(a, w), rep


# ---- nothing to do, and refusals ----

def test_empty_calls(q):
    import torch
    bf, i32, dev = torch.bfloat16, torch.int32, "cuda"

    def empty(*shape, dtype=bf):
        return torch.empty(shape, dtype=dtype, device=dev)

    off = torch.zeros(1, dtype=i32, device=dev)
    table = empty(0, 64, dtype=torch.float32)
    out, k_out = q.norm_rope(empty(0, 4, 64), empty(0, 2, 64), empty(0, dtype=i32), table)
    assert out.shape == (0, 4, 64) and k_out.shape == (0, 2, 64)
    assert q.prompt_attention(empty(0, 4, 64), empty(0, 2, 64), empty(0, 2, 64), off, off).shape == (0, 4, 64)
    pages = empty(0, 2, 16, 64)
    assert q.decode_attention(empty(0, 4, 64), pages, pages, empty(0, 3, dtype=i32), empty(0, dtype=i32)).shape == (0, 4, 64)
    # a batch whose caches are all empty, with no page at all
    lse = torch.ones((2, 4), device=dev)
    lens = torch.zeros(2, dtype=i32, device=dev)
    out = q.decode_attention(torch.ones((2, 4, 64), dtype=bf, device=dev), pages, pages, empty(2, 0, dtype=i32), lens, lse=lse)
    assert (f64(out) == 0).all() and (f64(lse) == -np.inf).all()
    err = torch.zeros(1, dtype=i32, device=dev)
    out = q.decode_attention(torch.ones((2, 4, 64), dtype=bf, device=dev), pages, pages, torch.zeros((2, 1), dtype=i32, device=dev),
                             lens + 5, err_count=err)
    assert (f64(out) == 0).all() and int(err[0]) >= 2
    kept, mass, n = q.evict(pages, pages, empty(0, 1, dtype=i32), empty(0, dtype=i32), empty(0, 2, 16, dtype=torch.float32), 4, pages, pages,
                            empty(0, 1, dtype=i32))
    assert kept.shape == (0, 2, 4) and mass.shape == (0, 2, 4) and n.shape == (0,)


def test_refusals(q):
    import torch
    dev, i32 = "cuda", torch.int32
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device=dev)
    pos = torch.zeros(4, dtype=i32, device=dev)
    cs = torch.zeros((8, 64), device=dev)
    off = torch.tensor([0, 4], dtype=i32, device=dev)
    pages = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16, device=dev)
    table = torch.zeros((4, 1), dtype=i32, device=dev)
    lens = torch.ones(4, dtype=i32, device=dev)
    mass = torch.zeros((4, 2, 16), device=dev)
    cases = [
        (TypeError, lambda: q.norm_rope(x.float(), x, pos, cs)),
        (TypeError, lambda: q.norm_rope(x, x.half(), pos, cs)),
        (TypeError, lambda: q.norm_rope(x, x, pos.short(), cs)),
        (ValueError, lambda: q.norm_rope(x, x[:2], pos, cs)),
        (ValueError, lambda: q.norm_rope(x.transpose(1, 2), x.transpose(1, 2), pos, cs)),
        (ValueError, lambda: q.norm_rope(x, x, pos, cs, v=x)),
        (ValueError, lambda: q.norm_rope(x, x, pos, cs, v=x, k_pages=pages, v_pages=pages, slots=pos.long(), bits=2)),
        (ValueError, lambda: q.norm_rope(x, x, pos, cs, v=x, k_pages=pages, v_pages=pages, slots=pos.long(), bits=8)),
        (q.QembError, lambda: q.norm_rope(x, x, pos, cs[:, :24].contiguous())),
        (TypeError, lambda: q.prompt_attention(x, x, x, off.long(), off.long())),
        (ValueError, lambda: q.prompt_attention(x, x, x[:3], off, off)),
        (q.QembError, lambda: q.prompt_attention(x, x, x, off, off, window=-1)),
        (TypeError, lambda: q.prompt_attention(x, x, x, off, off, lse=torch.zeros((4, 2), dtype=torch.float64, device=dev))),
        (ValueError, lambda: q.decode_attention(x, pages[:, :, :15], pages[:, :, :15], table, lens)),
        (ValueError, lambda: q.decode_attention(x, pages, pages, table[:2], lens)),
        (ValueError, lambda: q.decode_attention(x, pages, pages, table, lens, mass=mass[:, :1].contiguous())),
        (ValueError, lambda: q.decode_attention(x, pages, pages, table, lens, mass=mass, workspace=torch.zeros(4, dtype=torch.uint8, device=dev))),
        (TypeError, lambda: q.decode_attention(x, pages, pages, table.long(), lens)),
        (ValueError, lambda: q.decode_attention(x, pages.transpose(1, 2), pages.transpose(1, 2), table, lens)),
        (ValueError, lambda: q.evict(pages, pages, table, lens, mass, 17, pages, pages, table)),
        (ValueError, lambda: q.evict(pages, pages, table, lens, mass, 4, pages, pages, table, sinks=3, recent=2)),
        (ValueError, lambda: q.evict(pages, pages, table, lens, mass, 4, pages[:, :1].contiguous(), pages, table)),
        (TypeError, lambda: q.evict(pages, pages, table, lens, mass.double(), 4, pages, pages, table)),
    ]
    for i, (error, call) in enumerate(cases):
        with pytest.raises(error):
            call()
            print("case %d was taken" % i)


def test_own_workspace(q):
    """A caller's workspace, whatever it holds, gives the result of the library's own."""
    import torch
    g = np.random.default_rng(1300)
    cache = Cache(g, q, [3000, 700], 2, 64, 8, 16, "bf16")
    qt, _ = rand16(g, (2, 8, 64), "bf16")
    args = (qt, cache.pool[0], cache.pool[1], cache.table, cache.seq_lens)
    m0, m1 = (torch.zeros((2, 2, 3000), device="cuda") for _ in range(2))
    want = q.decode_attention(*args, bits=8, mass=m0)
    n = q.decode_workspace_bytes(2, 8, 2, 64, cache.width, 16, with_mass=True)
    ws = torch.full((n + 16,), 0xff, dtype=torch.uint8, device="cuda")
    assert torch.equal(q.decode_attention(*args, bits=8, mass=m1, workspace=ws[:n]), want) and torch.equal(m0, m1)
    assert bool((ws[n:] == 0xff).all())


def test_prompt_in_a_graph(q):
    """Prompt attention captured once and replayed on new inputs, bit for bit."""
    import torch
    g = np.random.default_rng(1310)
    n = 150
    x = torch.zeros((n, 8, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 60, n], dtype=torch.int32, device="cuda")

    def call(t):
        qt, kt, vt = t.split((4, 2, 2), 1)
        return q.prompt_attention(qt, kt, vt, off, off, max_q=90, window=40, sinks=2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(x)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(x)
    for rep in range(3):
        print("graph replay %d" % rep, flush=True)
        x.copy_(rand16(g, tuple(x.shape), "bf16")[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call(x.clone())), rep
