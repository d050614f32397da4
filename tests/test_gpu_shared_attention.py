"""Attention over shared prefixes on the GPU against float64 (bounds and formulas:
attention_model.py): group sizes, lengths from nothing on, all row formats, bad
data, rows that nobody sees, streams and graphs."""
from __future__ import annotations

import numpy as np
import pytest

from tests import attention_model as model
from tests.gpu_common import host, require_gpu
from tests.test_gpu_attention import Cache, close, f64, rand16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    lib = require_gpu()
    lib.load_attention_library()
    return lib


class Shared(Cache):
    """A cache whose first tables are the prefixes' and whose others are the sequences' own."""

    def __init__(self, g, lib, sizes, prefixes, own, hkv, d, bits, page, dtype, spread=1.0, wider=0):
        import torch
        assert len(sizes) == len(prefixes)
        lens = list(prefixes) + list(own)
        width = max(1, max(-(-n // page) for n in lens)) + wider
        super().__init__(g, lib, lens, hkv, d, bits, page, dtype, width=width, spread=spread)
        self.sizes, self.n_groups, self.batch = list(sizes), len(sizes), len(own)
        self.offsets_np = np.concatenate(([0], np.cumsum(sizes))).astype(np.int32)
        self.offsets = torch.from_numpy(self.offsets_np).cuda()

        def part(lo, hi):
            most = max([1] + [-(-n // page) for n in lens[lo:hi]]) + wider
            return self.table[lo:hi, :most].contiguous(), self.seq_lens[lo:hi].contiguous()

        self.prefix_table, self.prefix_lens = part(0, self.n_groups)
        self.block_table, self.own_lens = part(self.n_groups, len(lens))

    def group(self, b):
        for i in range(self.n_groups):
            if self.offsets_np[i] <= b < self.offsets_np[i + 1]:
                return i
        return None

    def seen(self, side, b, h):
        """The rows (and ranges) that sequence b sees of kv head h."""
        g = self.group(b)
        parts = ([self.rows(side, g, h)] if g is not None else []) + [self.rows(side, self.n_groups + b, h)]
        return np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts])

    def call(self, lib, qt, **more):
        args = dict(group_offsets=self.offsets, bits=self.bits) | more
        return lib.shared_attention(qt, self.pool[0], self.pool[1], self.prefix_table, self.prefix_lens, self.block_table,
                                    self.own_lens, **args)


def check(lib, g, cache, hq, dtype, scale=None, q_scale=1.0, rows=None, what="", **more):
    """All rows (or `rows` of them, drawn) against float64."""
    import torch
    group, d = hq // cache.hkv, cache.d
    qt, qv = rand16(g, (cache.batch, hq, d), dtype, q_scale)
    lse = torch.full((cache.batch, hq), 7.0, device="cuda")
    out = cache.call(lib, qt, lse=lse, scale=scale, **more)
    torch.cuda.synchronize()
    got, got_lse = f64(out), f64(lse)
    pairs = [(b, h) for b in range(cache.batch) for h in range(hq)]
    if rows is not None and rows < len(pairs):
        pairs = [pairs[i] for i in g.choice(len(pairs), rows, replace=False)]
    seen = {}
    for b, h in pairs:
        at = (b, h // group)
        if at not in seen:
            seen = {at: (cache.seen(0, *at), cache.seen(1, *at))}
        (k, kr), (v, vr) = seen[at]
        o, ob, ls, lb, _, _ = model.attend(qv[b, h], k, v, np.ones(len(k), bool), d ** -0.5 if scale is None else scale, dtype, kr, vr)
        close(got[b, h], o, ob, "%s out of sequence %d head %d" % (what, b, h))
        close(got_lse[b, h], ls, lb, "%s lse of sequence %d head %d" % (what, b, h))
    return out, lse


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [8, 40, 64, 96, 128, 200, 256])
def test_dims(q, bits, dtype, d):
    g = np.random.default_rng(2000 + d + bits)
    cache = Shared(g, q, [9], [333], [0, 1, 5, 16, 17, 40, 64, 65, 3], 2, d, bits, 16, dtype)
    check(q, g, cache, 8, dtype, what="d %d bits %d" % (d, bits))
    few = Shared(g, q, [2], [70], [3, 0], 1, d, bits, 16, dtype)
    check(q, g, few, 3, dtype, what="few rows, d %d bits %d" % (d, bits))


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("heads", [(1, 1), (8, 8), (5, 1), (32, 4), (17, 1), (40, 2)])
def test_heads(q, bits, heads):
    g = np.random.default_rng(2100 + heads[0] + bits)
    cache = Shared(g, q, [7, 4], [190, 64], list(range(0, 110, 10)), heads[1], 64, bits, 16, "bf16")
    check(q, g, cache, heads[0], "bf16", rows=60)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("size", [1, 2, 3, 4, 5, 8, 11, 12, 13, 16, 31, 32, 33, 40, 64, 65, 129])
def test_group_sizes(q, size, bits):
    """Rows of a group around the tiles that share a prefix (4 query heads a kv head)."""
    g = np.random.default_rng(2200 + size)
    own = [int(n) for n in g.integers(0, 50, size)]
    cache = Shared(g, q, [size], [300], own, 1, 64, bits, 16, "fp16")
    check(q, g, cache, 4, "fp16", rows=80)


@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 513, 1025])
def test_prefix_lengths(q, n):
    g = np.random.default_rng(2300 + n)
    for size, bits in ((2, 16), (40, 16), (40, 4)):
        cache = Shared(g, q, [size], [n], [i % 3 for i in range(size)], 2, 64, bits, 8, "bf16")
        check(q, g, cache, 4, "bf16", rows=40, what="prefix %d" % n)


@pytest.mark.parametrize("page", [1, 2, 8, 16, 64, 256])
@pytest.mark.parametrize("bits", [16, 8, 4])
def test_pages_that_end_inside_a_tile(q, page, bits):
    g = np.random.default_rng(2400 + page)
    for size in (3, 20):  # packed: tiles of 16 rows, and wide ones
        cache = Shared(g, q, [size], [301], [int(n) for n in g.integers(0, 100, size)], 2, 128, bits, page, "bf16")
        cache.poison_unowned(float("nan") if bits == 16 else 255)
        check(q, g, cache, 8, "bf16", rows=50)


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_groups_of_many_kinds(q, bits):
    """Empty groups, prefixes of nothing, sequences without rows of their own, one that sees nothing."""
    g = np.random.default_rng(2500 + bits)
    sizes, prefixes = [3, 0, 1, 50, 2, 0], [100, 30, 0, 257, 0, 0]
    own = [int(n) for n in g.integers(0, 90, sum(sizes))]
    own[1], own[3], own[-1] = 0, 0, 0  # the second: prefix alone; the others: nothing at all
    cache = Shared(g, q, sizes, prefixes, own, 2, 64, bits, 16, "bf16")
    out, lse = check(q, g, cache, 6, "bf16", rows=120)
    check_nothing = f64(out)[[3, -1]]
    assert (check_nothing == 0).all() and np.isneginf(f64(lse)[[3, -1]]).all()


def test_seventy_groups(q):
    """More groups than a wave has lanes."""
    g = np.random.default_rng(2510)
    sizes = [int(n) for n in g.integers(0, 4, 70)]
    cache = Shared(g, q, sizes, [int(n) for n in g.integers(0, 60, 70)], [int(n) for n in g.integers(0, 9, sum(sizes))], 1, 64, 16, 4, "bf16")
    check(q, g, cache, 4, "bf16", rows=150)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("size", [2, 70])
def test_long_prefix_is_split(q, bits, size):
    g = np.random.default_rng(2600 + bits)
    cache = Shared(g, q, [size], [9001], [int(n) for n in g.integers(0, 1500, size)], 2, 64, bits, 32, "fp16")
    a = check(q, g, cache, 6, "fp16", rows=25)[0]
    wide = Shared(np.random.default_rng(2600 + bits), q, [size], [9001], cache.lens[1:], 2, 64, bits, 32, "fp16", wider=700)
    b = check(q, np.random.default_rng(1), wide, 6, "fp16", rows=25)[0]  # a table far wider than any length
    assert a.shape == b.shape


@pytest.mark.parametrize("spread", [1e-3, 30.0])
@pytest.mark.parametrize("bits", [16, 8, 4])
def test_flat_and_peaked(q, spread, bits):
    """Weights all alike, and weights where few keys count."""
    g = np.random.default_rng(2650)
    for size in (2, 40):
        cache = Shared(g, q, [size], [700], [i for i in range(size)], 2, 64, bits, 16, "bf16", spread=spread)
        check(q, g, cache, 4, "bf16", rows=40)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0, -2.0, 2.0 ** -130])
def test_scales_of_any_sign(q, scale):
    g = np.random.default_rng(2660)
    for size, bits in ((2, 16), (40, 16), (40, 8), (2, 4)):
        cache = Shared(g, q, [size], [333], [i % 20 for i in range(size)], 2, 64, bits, 16, "bf16")
        check(q, g, cache, 4, "bf16", scale=scale, rows=40)


def test_one_group_without_offsets(q):
    import torch
    g = np.random.default_rng(2670)
    cache = Shared(g, q, [20], [150], [5] * 20, 2, 64, 16, 16, "bf16")
    qt, _ = rand16(g, (20, 4, 64), "bf16")
    assert torch.equal(cache.call(q, qt), cache.call(q, qt, group_offsets=None))


def test_sequences_that_no_group_holds(q):
    import torch
    g = np.random.default_rng(2680)
    cache = Shared(g, q, [4, 30], [90, 200], [int(n) for n in g.integers(1, 60, 40)], 2, 64, 16, 16, "bf16")
    check(q, g, cache, 4, "bf16", rows=160)  # sequences 34 .. 39
    cache.offsets_np += 2  # and 0, 1
    cache.offsets = torch.from_numpy(cache.offsets_np).cuda()
    check(q, g, cache, 4, "bf16", rows=160)


def test_same_rows_as_the_one_token_kernel(q):
    """A prefix and own rows together are what decode_attention sees in one table."""
    import torch
    g = np.random.default_rng(2690)
    page, size = 16, 24
    cache = Shared(g, q, [size], [320], [int(n) for n in g.integers(1, 60, size)], 2, 128, 8, page, "bf16")
    qt, _ = rand16(g, (size, 8, 128), "bf16")
    lse, want_lse = torch.zeros((size, 8), device="cuda"), torch.zeros((size, 8), device="cuda")
    got = cache.call(q, qt, lse=lse)
    table = torch.cat((cache.prefix_table[:, :20].expand(size, -1), cache.block_table), 1).contiguous()
    want = q.decode_attention(qt, cache.pool[0], cache.pool[1], table, cache.own_lens + 320, bits=8, lse=want_lse)
    # two results of one computation, each off by a bf16 rounding and by its weights' binary16 one
    assert float((got.double() - want.double()).norm() / want.double().norm()) < 2 * 2.0 ** -8
    assert float((lse - want_lse).abs().max()) < 1e-5


# ---- what must not be seen, and what must ----

@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_rows_that_nobody_sees(q, bits, poison):
    g = np.random.default_rng(2700 + bits)
    for size in (2, 37):
        cache = Shared(g, q, [size], [77], [int(n) for n in g.integers(0, 40, size)], 2, 64, bits, 16, "bf16")
        cache.poison_unowned(poison if bits == 16 else 255)  # packed: NaN scales and biases
        check(q, g, cache, 4, "bf16", rows=60)


@pytest.mark.parametrize("size", [2, 37])
def test_a_visible_nan_is_seen(q, size):
    import torch
    g = np.random.default_rng(2710)
    cache = Shared(g, q, [size], [77], [5] * size, 1, 64, 16, 16, "bf16")
    page = int(cache.table_np[0, 3])
    cache.pool[1][page, 0, 7, 5] = float("nan")  # a value of the prefix
    qt, _ = rand16(g, (size, 4, 64), "bf16")
    out = cache.call(q, qt)
    bad = torch.isnan(out)
    assert bool(bad[..., 5].all()) and int(bad.sum()) == 4 * size
    own = int(cache.table_np[1, 0])
    cache.pool[1][page, 0, 7, 5] = 0.0
    cache.pool[0][own, 0, 2, 9] = float("nan")  # a key of the first sequence
    lse = torch.zeros((size, 4), device="cuda")
    out = cache.call(q, qt, lse=lse)
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all()) and not bool(torch.isnan(out[1:]).any())


@pytest.mark.parametrize("size", [2, 37])
def test_scores_of_minus_infinity(q, size):
    """Keys that score -inf have no weight; rows that see only such keys give zeros."""
    import torch
    g = np.random.default_rng(2720)
    cache = Shared(g, q, [size], [100], [3] * size, 1, 64, 16, 16, "bf16")
    qt, _ = rand16(g, (size, 4, 64), "bf16")
    qt = qt.abs() + 0.125
    for p in range(-(-100 // 16)):  # the whole prefix
        cache.pool[0][int(cache.table_np[0, p])] = -float("inf")
    lse = torch.zeros((size, 4), device="cuda")
    got = cache.call(q, qt, lse=lse)
    want_lse = torch.zeros((size, 4), device="cuda")
    want = q.decode_attention(qt, cache.pool[0], cache.pool[1], cache.block_table, cache.own_lens, lse=want_lse)
    assert float((got.double() - want.double()).norm() / want.double().norm()) < 2 * 2.0 ** -8
    assert float((lse - want_lse).abs().max()) < 1e-5
    cache.own_lens.zero_()
    got = cache.call(q, qt, lse=lse)
    assert bool((got == 0).all()) and bool((lse == -float("inf")).all())


def test_bad_data_is_counted(q):
    import torch
    g = np.random.default_rng(2730)
    cache = Shared(g, q, [20, 3], [70, 40], [10] * 23, 2, 64, 16, 16, "bf16")
    qt, _ = rand16(g, (23, 4, 64), "bf16")

    def count(**more):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = cache.call(q, qt, err_count=err, **more)
        torch.cuda.synchronize()
        return int(err[0]), out

    n, clean = count()
    assert n == 0
    # lengths out of range: own ones, and a prefix
    lens = cache.own_lens.clone()
    cache.own_lens[4], cache.own_lens[22] = -1, 17
    cache.prefix_lens[1] = cache.prefix_table.shape[1] * 16 + 1
    n, out = count()
    assert n == 3
    keep = [i for i in range(23) if i not in (4, 20, 21, 22)]
    # the split of the work is the same, so the others' bits are
    assert torch.equal(out[keep], clean[keep])
    assert bool((out[22] == 0).all())
    cache.own_lens, cache.prefix_lens[1] = lens, 40
    # offsets that fall, or leave the batch: no groups
    alone = q.decode_attention(qt, cache.pool[0], cache.pool[1], cache.block_table, cache.own_lens)
    for bad in ([0, 21, 20], [-1, 20, 23], [0, 20, 24]):
        n, out = count(group_offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert n == 1, bad
        assert float((out.double() - alone.double()).norm() / alone.double().norm()) < 2 * 2.0 ** -8
    # pages that are none
    table = cache.prefix_table.clone()
    for page in (-1, cache.pool[0].shape[0], 2 ** 31 - 1, -2 ** 31):
        cache.prefix_table[0, 2] = page
        n, out = count()
        assert n >= 1 and bool(torch.isfinite(out).all())
        assert torch.equal(out[20:], clean[20:])
    cache.prefix_table = table
    cache.block_table[21, 0] = -5
    n, out = count()
    assert n >= 1
    keep = [i for i in range(23) if i != 21]
    assert torch.equal(out[keep], clean[keep])


def test_no_pages_at_all(q):
    import torch
    pool = torch.zeros((0, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    t = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    qt = torch.ones((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((3, 4), device="cuda")
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = q.shared_attention(qt, pool, pool, t, zero[:1], t.expand(3, -1).contiguous(), zero, lse=lse)
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
    empty = torch.zeros((3, 0), dtype=torch.int32, device="cuda")
    out = q.shared_attention(qt, pool, pool, empty[:1], zero[:1], empty, zero, lse=lse)
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
    none = q.shared_attention(qt[:0], pool, pool, t, zero[:1], empty[:0], zero[:0])
    assert none.shape == (0, 4, 64)


@pytest.mark.parametrize("size", [1, 20])
def test_pages_past_2_31_bytes(q, size):
    """Pages far beyond 2^31 bytes into the cache."""
    import torch
    g = np.random.default_rng(2750)
    page, hkv, d = 64, 8, 128
    pages = (5 << 30) // (page * hkv * d * 2)
    pool = [torch.zeros((pages, hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    far = [pages - 1, 3, pages // 2, pages - 2]
    rows = [torch.randn((len(far), hkv, page, d), device="cuda").bfloat16() for _ in range(2)]
    for p, r in zip(pool, rows):
        p[far] = r
    qt, _ = rand16(g, (size, hkv, d), "bf16")
    lens = torch.full((size,), 60, dtype=torch.int32, device="cuda")
    own = torch.full((size, 1), far[3], dtype=torch.int32, device="cuda")
    got = q.shared_attention(qt, pool[0], pool[1], torch.tensor([far[:3]], dtype=torch.int32, device="cuda"),
                             torch.tensor([180], dtype=torch.int32, device="cuda"), own, lens)
    near = torch.arange(4, dtype=torch.int32, device="cuda")
    want = q.shared_attention(qt, rows[0], rows[1], near[None, :3].contiguous(), torch.tensor([180], dtype=torch.int32, device="cuda"),
                              near[3:].expand(size, -1).contiguous(), lens)
    assert torch.equal(got, want) and bool(want.any())


# ---- streams, graphs, workspaces ----

def test_equal_calls_give_equal_bits_on_any_stream(q):
    import torch
    g = np.random.default_rng(2760)
    cache = Shared(g, q, [33, 5], [700, 90], [int(n) for n in g.integers(0, 300, 38)], 2, 64, 4, 16, "bf16")
    qt, _ = rand16(g, (38, 8, 64), "bf16")
    want = cache.call(q, qt)
    assert torch.equal(cache.call(q, qt), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = cache.call(q, qt)
    side.synchronize()
    assert torch.equal(got, want)


def test_workspace_is_enough_and_not_left(q):
    import torch
    g = np.random.default_rng(2770)
    for sizes, prefixes, hq, bits in (([40], [2000], 8, 16), ([2], [5000], 4, 8), ([3, 0, 70], [900, 5, 40], 6, 4), ([1], [1], 2, 16)):
        b = sum(sizes)
        cache = Shared(g, q, sizes, prefixes, [int(n) for n in g.integers(0, 700, b)], 2, 64, bits, 16, "bf16")
        need = q.shared_workspace_bytes(b, hq, 2, 64, len(sizes), cache.prefix_table.shape[1], cache.block_table.shape[1], 16, bits)
        room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        qt, _ = rand16(g, (b, hq, 64), "bf16")
        want = cache.call(q, qt)
        assert torch.equal(cache.call(q, qt, workspace=room), want)
        assert bool((room[need:] == 0xA5).all())
        if need:
            with pytest.raises(ValueError):
                cache.call(q, qt, workspace=room[:need - 1])


def test_two_graphs_share_a_workspace(q):
    """Captured calls of different sizes with one workspace, replayed in turn on new inputs against eager calls."""
    import torch
    g = np.random.default_rng(2780)
    caches = [Shared(g, q, [30], [1500], [int(n) for n in g.integers(0, 600, 30)], 2, 64, 16, 16, "bf16"),
              Shared(g, q, [2, 1], [700, 80], [20, 0, 300], 2, 64, 8, 16, "bf16")]
    room = torch.empty(max(q.shared_workspace_bytes(c.batch, 8, 2, 64, c.n_groups, c.prefix_table.shape[1], c.block_table.shape[1], 16, c.bits) for c in caches),
                       dtype=torch.uint8, device="cuda")
    inputs = [torch.zeros((c.batch, 8, 64), dtype=torch.bfloat16, device="cuda") for c in caches]
    lses = [torch.zeros((c.batch, 8), device="cuda") for c in caches]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c, x, l in zip(caches, inputs, lses):
            c.call(q, x, lse=l, workspace=room)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c, x, l in zip(caches, inputs, lses):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(c.call(q, x, lse=l, workspace=room))
        graphs.append(graph)
    for rep in range(4):
        print("graph replay %d" % rep, flush=True)
        for i in ((0, 1) if rep % 2 else (1, 0)):
            c = caches[i]
            xt, _ = rand16(g, tuple(inputs[i].shape), "bf16")
            inputs[i].copy_(xt)
            c.own_lens.copy_(torch.from_numpy(g.integers(0, np.array(c.lens[c.n_groups:]) + 1).astype(np.int32)))
            c.prefix_lens[0] = 500 + 30 * rep
            graphs[i].replay()
            torch.cuda.synchronize()
            lse = torch.zeros_like(lses[i])
            want = c.call(q, xt, lse=lse)
            torch.cuda.synchronize()
            assert torch.equal(outs[i], want) and torch.equal(lses[i], lse), (rep, i)


# ---- refusals ----

def test_refusals(q):
    import torch
    g = np.random.default_rng(2790)
    c = Shared(g, q, [4], [40], [5] * 4, 2, 64, 16, 16, "bf16")
    qt, _ = rand16(g, (4, 8, 64), "bf16")
    c.call(q, qt)
    i32 = dict(dtype=torch.int32, device="cuda")
    for bad, error in (
        (dict(group_offsets=torch.zeros(3, **i32)), ValueError), (dict(group_offsets=torch.zeros(2, dtype=torch.int64, device="cuda")), TypeError),
        (dict(bits=8), ValueError), (dict(bits=5), ValueError), (dict(scale=float("nan")), q.QembError), (dict(scale=float("inf")), q.QembError),
        (dict(out=torch.empty((4, 8, 32), dtype=torch.bfloat16, device="cuda")), ValueError), (dict(lse=torch.empty((4, 8))), TypeError),
        (dict(err_count=torch.zeros(2, **i32)), ValueError), (dict(workspace=torch.zeros(1 << 20, device="cuda")), TypeError),
    ):
        with pytest.raises(error):
            c.call(q, qt, **bad)
    with pytest.raises(TypeError):
        c.call(q, qt.transpose(0, 1))
    with pytest.raises(TypeError):
        c.call(q, qt.float())
    with pytest.raises(q.QembError):  # 7 query heads over 2 kv heads
        c.call(q, qt[:, :7].contiguous())
    two = torch.zeros((2, 3), **i32)
    with pytest.raises(ValueError):  # two prefixes, no offsets
        q.shared_attention(qt, c.pool[0], c.pool[1], two, torch.zeros(2, **i32), c.block_table, c.own_lens)
    with pytest.raises(ValueError):
        q.shared_attention(qt, c.pool[0], c.pool[1], two[:0], torch.zeros(0, **i32), c.block_table, c.own_lens)
    with pytest.raises(ValueError):
        q.shared_attention(qt, c.pool[0], c.pool[1], c.prefix_table, c.prefix_lens, c.block_table[:3], c.own_lens)
    assert host(c.own_lens).tolist() == [5] * 4


@pytest.mark.parametrize("page", [4, 16, 64])
@pytest.mark.parametrize("bits", [16, 8, 4])
def test_rows_of_bad_pages_are_left_out(q, bits, page):
    """In the prefix and among a sequence's own rows, against float64 without those rows."""
    import torch
    g = np.random.default_rng(2800 + page + bits)
    for size in (2, 40):
        cache = Shared(g, q, [size], [500], [150 + i for i in range(size)], 1, 64, bits, page, "bf16")
        bad = {0: 3, 1: 1}  # a page of the prefix, and one of the first sequence
        for row, at in bad.items():
            (cache.prefix_table if row == 0 else cache.block_table)[0, at] = 2 ** 31 - 1 - row
        qt, qv = rand16(g, (size, 4, 64), "bf16")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        lse = torch.zeros((size, 4), device="cuda")
        out = cache.call(q, qt, err_count=err, lse=lse)
        assert int(err[0]) >= 1
        for b in (0, size - 1):
            k, kr = cache.seen(0, b, 0)
            v, vr = cache.seen(1, b, 0)
            see = np.ones(len(k), bool)
            see[3 * page:4 * page] = False
            if b == 0:
                see[500 + page:500 + 2 * page] = False
            for h in range(4):
                o, ob, ls, lb, _, _ = model.attend(qv[b, h], k, v, see, 64 ** -0.5, "bf16", kr, vr)
                close(f64(out)[b, h], o, ob, "out")
                close(f64(lse)[b, h], ls, lb, "lse")


def test_bad_offsets_among_many_groups(q):
    """A fall beyond the 64th group is found, too."""
    import torch
    g = np.random.default_rng(2810)
    sizes = [1] * 80
    cache = Shared(g, q, sizes, [20] * 80, [5] * 80, 1, 64, 16, 4, "bf16")
    qt, _ = rand16(g, (80, 2, 64), "bf16")
    off = cache.offsets.clone()
    off[70] = 3
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = cache.call(q, qt, group_offsets=off, err_count=err)
    assert int(err[0]) == 1
    alone = q.decode_attention(qt, cache.pool[0], cache.pool[1], cache.block_table, cache.own_lens)
    assert float((out.double() - alone.double()).norm() / alone.double().norm()) < 2 * 2.0 ** -8


def test_two_calls_at_once(q):
    """On two streams, each with the workspace of its own call."""
    import torch
    g = np.random.default_rng(2820)
    caches = [Shared(g, q, [60], [4000], [50] * 60, 2, 64, bits, 16, "bf16") for bits in (16, 8)]
    qs = [rand16(g, (60, 8, 64), "bf16")[0] for _ in caches]
    want = [c.call(q, x) for c, x in zip(caches, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in caches]
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(caches[i].call(q, qs[i]))
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert all(torch.equal(o, w) for o in outs)


def test_prefixes_of_very_different_lengths(q):
    """Shares of the work that groups take from each other; one group with nearly all of it."""
    g = np.random.default_rng(2830)
    for sizes, prefixes, bits in (([1, 1, 1, 60], [30000, 3, 40, 130], 16), ([100, 2], [64, 20000], 8), ([2, 0, 3, 0, 1], [0, 5000, 9000, 1, 129], 4)):
        cache = Shared(g, q, sizes, prefixes, [int(n) for n in g.integers(0, 70, sum(sizes))], 2, 64, bits, 16, "bf16")
        check(q, g, cache, 8, "bf16", rows=40)


@pytest.mark.parametrize("groups", [4, 70])
def test_every_bad_prefix_length_is_counted(q, groups):
    """Those of groups without sequences, and those beside offsets that make no groups, among them."""
    import torch
    g = np.random.default_rng(2840)
    sizes = [0] * groups
    sizes[1], sizes[-2] = 2, 3
    cache = Shared(g, q, sizes, [20] * groups, [5] * 5, 2, 64, 16, 16, "bf16")
    qt, _ = rand16(g, (5, 4, 64), "bf16")
    clean = cache.call(q, qt)

    def count(**more):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        return cache.call(q, qt, err_count=err, **more), int(err[0])

    assert count()[1] == 0
    cache.prefix_lens[0], cache.prefix_lens[-1] = -1, 2 ** 31 - 1  # of nobody
    out, n = count()
    assert n == 2 and torch.equal(out, clean)
    cache.prefix_lens[1] = cache.prefix_table.shape[1] * 16 + 1  # of two sequences
    cache.own_lens[4] = -7
    assert count()[1] == 4
    falling = cache.offsets.clone()
    falling[-1] = 0
    assert count(group_offsets=falling)[1] == 5
