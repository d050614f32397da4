"""Attention over shared prefixes at the sizes where its launches change: joins
by one wave or four, slots around the lanes of a wave, one or two workgroups a
CU, packed rows by tiles of 16 or wide ones; all against float64."""
from __future__ import annotations

import numpy as np
import pytest

from tests import attention_model as model
from tests.gpu_common import require_gpu
from tests.test_gpu_attention import close, f64, rand16
from tests.test_gpu_shared_attention import Shared, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    lib = require_gpu()
    lib.load_attention_library()
    return lib


def own_lens(g, n, most):
    return [int(i) for i in g.integers(0, most, n)]


def widen(cache, prefix_width=0, width=0):
    """Tables with more columns than any length needs, filled with pages that are none."""
    import torch
    if prefix_width:
        cache.prefix_table = torch.nn.functional.pad(cache.prefix_table, (0, prefix_width - cache.prefix_table.shape[1]), value=-7)
    if width:
        cache.block_table = torch.nn.functional.pad(cache.block_table, (0, width - cache.block_table.shape[1]), value=-7)
    return cache


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_rows_around_a_thousand(q, d, bits):
    """1023, 1024, 1025 and 3000 query rows."""
    g = np.random.default_rng(7000 + d + bits)
    for batch, hq, hkv in ((341, 3, 1), (128, 8, 1), (205, 5, 1), (375, 8, 2)):
        cache = Shared(g, q, [batch], [900], own_lens(g, batch, 40), hkv, d, bits, 16, "bf16")
        check(q, g, cache, hq, "bf16", rows=25, what="%d rows" % (batch * hq))


@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("batch", [20, 128])
def test_slots_around_the_lanes(q, batch, d):
    """Prefixes of 15 .. 17, 31 .. 33 and 63 .. 65 chunks of 128 keys; 160 rows (four waves each) and 1024 (one)."""
    g = np.random.default_rng(7100 + d + batch)
    for chunks in (15, 16, 17, 31, 32, 33, 63, 64, 65):
        cache = Shared(g, q, [batch], [128 * chunks], own_lens(g, batch, 30), 1, d, 16, 16, "fp16")
        # a wide table: as many chunks as its width, not its length, allows
        check(q, g, widen(cache, prefix_width=8192), 8, "fp16", rows=12, what="%d chunks" % chunks)


@pytest.mark.parametrize("sizes", [[128], [100, 0, 28]])
@pytest.mark.parametrize("bits,width", [(16, 8191), (16, 8192), (8, 4095), (8, 4096), (4, 4095), (4, 4096)])
def test_one_and_two_workgroups_a_cu(q, bits, width, sizes):
    """1024 rows of one kv head (eight wide tiles), tables on both sides of what two workgroups a CU ask for; a
    few sequences that have long rows of their own besides."""
    g = np.random.default_rng(7200 + width + bits)
    own = own_lens(g, 128, 60)
    own[3], own[90] = 2000, 1100
    cache = Shared(g, q, sizes, [5000, 40, 3000][:len(sizes)], own, 1, 64, bits, 16, "bf16")
    check(q, g, widen(cache, prefix_width=width), 8, "bf16", rows=30)


@pytest.mark.parametrize("bits", [16, 8])
def test_long_prefix_of_many_rows(q, bits):
    """256 sequences of 32 query heads under a prefix of 32768."""
    g = np.random.default_rng(7300 + bits)
    cache = Shared(g, q, [256], [32768], own_lens(g, 256, 20), 8, 64, bits, 64, "bf16")
    check(q, g, cache, 32, "bf16", rows=10)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [8, 40, 64, 96, 128, 200, 256])
def test_wide_dims(q, bits, dtype, d):
    """Wide tiles over every row format (13 sequences of 4 query heads a kv head and more), one group and three."""
    g = np.random.default_rng(7400 + d + bits)
    cache = Shared(g, q, [13], [333], own_lens(g, 13, 70), 2, d, bits, 16, dtype)
    check(q, g, cache, 8, dtype, rows=60, what="d %d bits %d" % (d, bits))
    many = Shared(g, q, [30, 2, 21], [333, 70, 129], own_lens(g, 53, 20), 1, d, bits, 4, dtype)
    many.poison_unowned(float("nan") if bits == 16 else 255)
    check(q, g, many, 4, dtype, rows=60, what="three groups, d %d bits %d" % (d, bits))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("d", [64, 96])
@pytest.mark.parametrize("sizes,hq", [([12], 4), ([7], 7), ([48], 1), ([49], 1), ([24, 24], 2), ([50, 47], 1)])
def test_packed_rows_on_both_sides_of_the_wide_tiles(q, sizes, hq, d, bits):
    """48 and 49 query rows a group, on the average of groups, too."""
    g = np.random.default_rng(7500 + d + bits)
    cache = Shared(g, q, sizes, [300, 210][:len(sizes)], own_lens(g, sum(sizes), 50), 1, d, bits, 16, "bf16")
    check(q, g, cache, hq, "bf16", rows=60)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("size", [2, 70])
def test_a_table_wider_than_its_prefix_changes_little(q, bits, size):
    """The same call with tables far wider than any length: another split of the same sums."""
    import torch
    g = np.random.default_rng(7600 + bits)
    cache = Shared(g, q, [size], [9001], own_lens(g, size, 1500), 2, 64, bits, 32, "fp16")
    qt, qv = rand16(g, (size, 6, 64), "fp16")
    lses = [torch.zeros((size, 6), device="cuda") for _ in range(2)]
    tight = cache.call(q, qt, lse=lses[0])
    wide = widen(cache, prefix_width=5000, width=900).call(q, qt, lse=lses[1])
    for b in (0, size // 2, size - 1):
        for h in (0, 5):
            (k, kr), (v, vr) = cache.seen(0, b, h // 3), cache.seen(1, b, h // 3)
            _, ob, _, lb, _, _ = model.attend(qv[b, h], k, v, np.ones(len(k), bool), 64 ** -0.5, "fp16", kr, vr)
            close(f64(wide)[b, h], f64(tight)[b, h], 2 * ob, "out")  # each within its bound of the same value
            close(f64(lses[1])[b, h], f64(lses[0])[b, h], 2 * lb, "lse")
