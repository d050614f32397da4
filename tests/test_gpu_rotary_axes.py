"""Norm and rotation with positions on several axes on the GPU against float64,
and against the one-axis call where the two mean the same."""
from __future__ import annotations

import numpy as np
import pytest

from tests import attention_model as model
from tests.gpu_common import host, require_gpu
from tests.test_gpu_attention import close, f64, norm_bound, rand16, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    lib = require_gpu()
    lib.load_attention_library()
    return lib


def angles(table, pos, axis):
    """cos, sin [tokens, pairs] of each pair's own axis; a pair of no axis stands still."""
    n, r = pos.shape[1], table.shape[1] // 2
    cos, sin = np.ones((n, r)), np.zeros((n, r))
    for i, a in enumerate(axis):
        if a < pos.shape[0]:
            cos[:, i], sin[:, i] = table[pos[a], i], table[pos[a], r + i]
    return cos, sin


def expected(x, w, cos, sin, eps, interleaved, norm):
    if norm:
        return model.norm_rope(x, w, cos, sin, eps, interleaved)
    # without the norm: that of rows scaled to a mean square of one, scaled back
    size = np.sqrt((x * x).mean(-1, keepdims=True))
    size[size == 0] = 1.0
    return model.norm_rope(x / size, np.ones(x.shape[-1]), cos, sin, 0.0, interleaved) * size


def bound(want, x, w, eps, dtype, d, norm):
    if norm:
        return norm_bound(want, x, w, eps, dtype, d)
    # one rounding to 16 bits, and two products with a sum in binary32
    return model.U[dtype] * np.abs(want) + 4 * 2.0 ** -24 * np.abs(x).max(-1, keepdims=True) + 2.0 ** -25


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,rot,axes", [(16, 16, 2), (40, 32, 3), (64, 64, 1), (64, 0, 2), (96, 48, 4), (128, 128, 3), (200, 16, 2), (256, 256, 4)])
def test_axes(q, norm, interleaved, dtype, d, rot, axes):
    import torch
    g = np.random.default_rng(3000 + d + axes)
    n, hq, hkv, eps = 13, 3, 2, 1e-5
    (qt, qv), (kt, kv) = rand16(g, (n, hq, d), dtype, 2.0), rand16(g, (n, hkv, d), dtype, 0.1)
    (wq, wqv), (wk, wkv) = rand16(g, (d,), dtype), rand16(g, (d,), dtype)
    table = rope_table(50, rot)
    pos = g.integers(0, 50, (axes, n))
    ways = [g.integers(0, axes + 1, rot // 2)]  # any axis for any pair, some of none
    ways.append(np.sort(ways[0]))
    for axis in ways:
        cos, sin = angles(table, pos, axis)
        for index in (torch.int32, torch.int64):
            qo, ko = q.norm_rope(qt, kt, torch.from_numpy(pos).to(index).cuda(), torch.from_numpy(table).cuda(), wq if norm else None,
                                 wk if norm else None, eps=eps, interleaved=interleaved, norm=norm,
                                 pair_axes=torch.from_numpy(axis.astype(np.uint8)).cuda())
            for got, x, w in ((qo, qv, wqv), (ko, kv, wkv)):
                want = expected(x, w, cos, sin, eps, interleaved, norm)
                close(f64(got), want, bound(want, x, w, eps, dtype, d, norm), "axes")


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("d", [16, 64, 96, 128, 256])
def test_append(q, norm, bits, d):
    """Equal positions on all axes give the one-axis call's bits, rows and pages alike."""
    import torch
    g = np.random.default_rng(3100 + d + bits)
    n, hq, hkv, page, pages = 300, 4, 2, 8, 40
    t, val = rand16(g, (n, hq + 2 * hkv, d), "bf16", 1.5)
    qt, kt, vt = t.split((hq, hkv, hkv), 1)
    rot = d // 16 * 16
    table = torch.from_numpy(rope_table(400, rot)).cuda()
    pos = torch.arange(n, device="cuda")
    slots = g.permutation(pages * page)[:n]
    slots[3] = -1
    slots = torch.from_numpy(slots).cuda()
    row = d if bits == 16 else q.row_stride(d, bits)
    kind = torch.bfloat16 if bits == 16 else torch.uint8
    axis = torch.from_numpy(g.integers(0, 3, rot // 2).astype(np.uint8)).cuda()

    def run(**more):
        pool = [torch.full((pages, hkv, page, row), 77, dtype=kind, device="cuda") for _ in range(2)]
        k_out = torch.zeros((n, hkv, d), dtype=torch.bfloat16, device="cuda")
        qo, _ = q.norm_rope(qt, kt, cos_sin=table, v=vt, k_pages=pool[0], v_pages=pool[1], slots=slots, bits=bits, k_out=k_out, norm=norm, **more)
        return [qo, k_out] + pool

    got = run(positions=pos.expand(3, -1).contiguous(), pair_axes=axis)
    want = run(positions=pos)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    if not norm:
        cos, sin = angles(host(table), np.tile(np.arange(n), (3, 1)), host(axis))
        kv = val[:, hq:hq + hkv]
        w = expected(kv, None, cos, sin, 0.0, False, False)
        close(f64(got[1]), w, bound(w, kv, None, 0.0, "bf16", d, False), "k without the norm")


@pytest.mark.parametrize("tokens", [1, 2, 63, 1000, 5000])
def test_token_counts(q, tokens):
    import torch
    g = np.random.default_rng(3200 + tokens)
    qt, qv = rand16(g, (tokens, 5, 64), "fp16")
    kt, _ = rand16(g, (tokens, 1, 64), "fp16")
    table = rope_table(70, 64)
    pos = g.integers(0, 70, (2, tokens))
    axis = np.arange(32) % 2
    qo, _ = q.norm_rope(qt, kt, torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda(), pair_axes=torch.from_numpy(axis.astype(np.uint8)).cuda())
    cos, sin = angles(table, pos, axis)
    want = model.norm_rope(qv, np.ones(64), cos, sin, 1e-6, False)
    close(f64(qo), want, norm_bound(want, qv, np.ones(64), 1e-6, "fp16", 64), "tokens")


def test_rows_of_infinities_without_the_norm(q):
    """Values are turned as they are: zeros, infinities and NaN stay where the formula leaves them."""
    import torch
    x = torch.zeros((4, 1, 16), dtype=torch.bfloat16, device="cuda")
    x[1, 0, 3], x[2, 0, 12], x[3] = float("inf"), float("nan"), 2.0
    table = torch.from_numpy(rope_table(8, 16)).cuda()
    pos = torch.tensor([[0, 1, 2, 3], [3, 2, 1, 0]], device="cuda")
    axis = torch.tensor([0, 1, 0, 1, 255, 255, 255, 255], dtype=torch.uint8, device="cuda")
    got, _ = q.norm_rope(x, x, pos, table, pair_axes=axis, norm=False)
    assert bool((got[0] == 0).all())
    assert sorted(torch.nonzero(~torch.isfinite(got[1, 0]))[:, 0].tolist()) == [3, 11]
    assert torch.nonzero(~torch.isfinite(got[2, 0]))[:, 0].tolist() == [12]  # its pair is not turned
    assert bool((got[3, 0, 4:8] == 2).all()) and bool((got[3, 0, 12:] == 2).all())


def test_bad_positions_are_counted(q):
    import torch
    g = np.random.default_rng(3300)
    qt, _ = rand16(g, (6, 2, 64), "bf16")
    kt, _ = rand16(g, (6, 1, 64), "bf16")
    pool = [torch.full((2, 1, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.from_numpy(rope_table(50, 64)).cuda()
    axis = q.rotary_axes((16, 8, 8))
    slots = torch.tensor([0, 1, 2, 3, 8, 5], dtype=torch.int64, device="cuda")  # the fifth is past the cache
    for index, big in ((torch.int32, 2 ** 31 - 1), (torch.int64, 2 ** 62)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pos = torch.zeros((3, 6), dtype=index, device="cuda")
        pos[0, 1], pos[1, 2], pos[2, 3], pos[2, 5] = -1, 50, big, 49
        qo, _ = q.norm_rope(qt, kt, pos, table, v=kt, k_pages=pool[0], v_pages=pool[1], slots=slots, err_count=err, pair_axes=axis)
        assert int(err[0]) == 4
        assert (f64(qo)[1:4] == 0).all() and not (f64(qo)[[0, 4, 5]] == 0).any(axis=(1, 2)).all()
        for p in pool:
            flat = f64(p)[:, 0].reshape(8, 64)
            assert (flat[[1, 2, 3, 4, 6, 7]] == 7).all() and not (flat[[0, 5]] == 7).any(axis=1).all()


def test_rotary_axes(q):
    assert q.rotary_axes((3, 2, 2)).tolist() == [0, 0, 0, 1, 1, 2, 2]
    assert q.rotary_axes((3, 2, 2), in_turn=True).tolist() == [0, 1, 2, 0, 1, 2, 0]
    assert q.rotary_axes((0, 4), in_turn=True).tolist() == [1, 1, 1, 1]
    for bad in ((), (1,) * 5, (3, -1)):
        with pytest.raises(ValueError):
            q.rotary_axes(bad)


def test_refusals(q):
    import torch
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((50, 64), device="cuda")
    pos = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    axis = q.rotary_axes((16, 8, 8))
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    q.norm_rope(x, x, pos, table, w, w, pair_axes=axis)
    for args, more, error in (
        ((x, x, pos[0].contiguous(), table), dict(pair_axes=axis), ValueError), ((x, x, pos, table), {}, ValueError),
        ((x, x, torch.zeros((5, 4), dtype=torch.int32, device="cuda"), table), dict(pair_axes=axis), ValueError),
        ((x, x, torch.zeros((0, 4), dtype=torch.int32, device="cuda"), table), dict(pair_axes=axis), ValueError),
        ((x, x, pos, table), dict(pair_axes=axis[:31]), ValueError), ((x, x, pos, table), dict(pair_axes=axis.int()), TypeError),
        ((x, x, pos, table), dict(pair_axes=axis.cpu()), TypeError), ((x, x, pos.t().contiguous().t(), table), dict(pair_axes=axis), ValueError),
        ((x, x, pos, table, w), dict(pair_axes=axis, norm=False), ValueError), ((x, x, pos[:, :3].contiguous(), table), dict(pair_axes=axis), ValueError),
    ):
        with pytest.raises(error):
            q.norm_rope(*args, **more)


def test_captured_replays(q):
    import torch
    g = np.random.default_rng(3400)
    x = torch.zeros((33, 6, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((3, 33), dtype=torch.int64, device="cuda")
    table = torch.from_numpy(rope_table(256, 64)).cuda()
    axis = q.rotary_axes((12, 10, 10), in_turn=True)
    step = lambda x, pos: q.norm_rope(x[:, :4], x[:, 4:], pos, table, pair_axes=axis, norm=False)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, pos)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(x, pos)
    for rep in range(3):
        print("graph replay %d" % rep, flush=True)
        x.copy_(rand16(g, tuple(x.shape), "bf16")[0])
        pos.copy_(torch.from_numpy(g.integers(0, 256, (3, 33))))
        graph.replay()
        torch.cuda.synchronize()
        for a, w in zip(res, step(x.clone(), pos.clone())):
            assert torch.equal(a, w), rep


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("d,rot,norm", [(16, 16, True), (64, 32, False), (96, 96, True), (128, 128, True), (128, 64, False), (256, 256, False)])
def test_append_of_unequal_positions(q, d, rot, norm, bits, interleaved):
    """Keys turned by another position on each axis, in every row format, against float64."""
    import torch
    g = np.random.default_rng(3500 + d + bits)
    n, hkv, page, pages, eps = 57, 3, 8, 9, 1e-5
    (qt, _), (kt, kv), (vt, vv) = (rand16(g, (n, h, d), "bf16", 1.5) for h in (2, hkv, hkv))
    wk, wkv = rand16(g, (d,), "bf16")
    table = rope_table(90, rot)
    pos, axis = g.integers(0, 90, (3, n)), g.integers(0, 4, rot // 2)  # some pairs of no axis
    slots = g.permutation(pages * page)[:n]
    row = d if bits == 16 else q.row_stride(d, bits)
    pool = [torch.full((pages, hkv, page, row), 77, dtype=torch.bfloat16 if bits == 16 else torch.uint8, device="cuda") for _ in range(2)]
    q.norm_rope(qt, kt, torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda(), None, wk if norm else None, eps=eps, interleaved=interleaved,
                v=vt, k_pages=pool[0], v_pages=pool[1], slots=torch.from_numpy(slots).cuda(), bits=bits, norm=norm,
                pair_axes=torch.from_numpy(axis.astype(np.uint8)).cuda())
    cos, sin = angles(table, pos, axis)
    want_k = expected(kv, wkv, cos, sin, eps, interleaved, norm)
    for p, want, own in ((pool[0], want_k, bound(want_k, kv, wkv, eps, "bf16", d, norm)), (pool[1], vv, np.zeros_like(vv))):
        rows = host(p.view(torch.uint8)).transpose(0, 2, 1, 3).reshape(pages * page, hkv, -1)
        free = np.ones(pages * page, bool)
        free[slots] = False
        if bits == 16:
            close(f64(p).transpose(0, 2, 1, 3).reshape(pages * page, hkv, d)[slots], want, own, "rows")
            continue
        assert (rows[free] == 77).all()
        values, rng = model.unpack_rows(rows[slots], d, bits)
        # The packed value is off from the row by half a step, by what binary16 rounds of scale (times the last
        # code) and bias, half an ulp each (2^-11; 2^-25 below its normal range, the scale's times 255), and by
        # binary32 before, which `own` holds (its 16-bit rounding is not made here)
        most = np.abs(want).max(-1, keepdims=True)
        step = rng[..., None] / (2 ** bits - 1)
        limit = 0.5 * step * (1 + 2.0 ** -9) + 2.0 ** -11 * (rng[..., None] + most) + 2.0 ** -25 * 256 + own
        close(values, want, np.broadcast_to(limit, want.shape), "packed rows")
