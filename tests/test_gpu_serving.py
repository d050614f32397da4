"""Residual addition with a norm, and log probabilities of tokens, on the GPU against float64."""
from __future__ import annotations

import numpy as np
import pytest

from tests import attention_model as model
from tests.gpu_common import host, require_gpu
from tests.test_gpu_attention import close, f64, rand16, torch_type

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    lib = require_gpu()
    lib.load_serving_library()
    return lib


# ---- residual addition and norm ----

# y is off by binary32 sums of at most 16 x 8 squares a thread and 8 joins (half of that, from the root), and by
# five more roundings: under 100 units of 2^-24 of itself
REL = 100 * E


def normed(h, w, eps):
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w


def check_add_norm(q, g, n, d, dtype, form="values", group=0, residual=True, weight=True, eps=1e-5, strided=False, spread=3.0):
    import torch
    wide = d + 24 if strided else d
    (xt, xv), (rt, rv) = rand16(g, (n, wide), dtype), rand16(g, (n, wide), dtype, spread)
    wt, wv = rand16(g, (d,), dtype)
    x, r, xv, rv = xt[:, :d], rt[:, :d], xv[:, :d], rv[:, :d]
    h = xv + rv if residual else xv
    want = normed(h, wv if weight else np.ones(d), eps)
    out, total, scales = q.add_norm(x, r if residual else None, wt if weight else None, eps=eps, form=form, group=group)
    if residual:
        assert torch.equal(total, (x.float() + r.float()).to(x.dtype)) and total.is_contiguous()
    else:
        assert total is None
    if form == "values":
        assert scales is None and out.dtype == x.dtype
        close(f64(out), want, model.U[dtype] * np.abs(want) * (1 + REL) + REL * np.abs(want) + 2.0 ** -25, "values")
        return
    if form == "rows8":
        assert scales is None
        values, rng = model.unpack_rows(host(out), d, 8)
        most = np.abs(want).max(-1, keepdims=True)
        # half a step, the fp16 rounding of scale (at the last code) and bias, and binary32 before
        bound = 0.5 * rng[..., None] / 255 * (1 + 2.0 ** -9) + 2.0 ** -11 * (rng[..., None] + most) + REL * most + 2.0 ** -25 * 256
        close(values, want, np.broadcast_to(bound, values.shape), "packed rows")
        assert (host(out)[:, d + 4:] == 0).all()
        return
    per = group or d
    assert scales.shape == ((n, d // group) if group else (n,))
    y = want.reshape(n, -1, per)
    most = 127.0 if form == "int8" else 448.0
    s = f64(scales).reshape(n, -1, 1)
    top = np.abs(y).max(-1, keepdims=True)
    close(s, top / most, (REL + 2 * E) * top / most, "scales")
    codes = f64(out.float()).reshape(n, -1, per)
    if form == "int8":
        assert np.abs(codes).max(initial=0) <= 127
        bound = 0.5 * s + 2 * (REL + 4 * E) * top  # half a step; codes times the scale's own error
    else:
        # half a step of 3 bits after the leading one, down to steps of 2^-9
        bound = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s) * (1 + 2.0 ** -10) + 2 * (REL + 4 * E) * top
    close(codes * s, y, bound, form)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [8, 16, 64, 72, 128, 256, 264, 504, 512, 520, 1024, 1032, 2048, 2056, 4096, 5120, 8192, 8200, 16384, 32768])
def test_add_norm_dims(q, dtype, d):
    g = np.random.default_rng(4000 + d)
    check_add_norm(q, g, 5, d, dtype)
    check_add_norm(q, g, 3, d, dtype, residual=False, strided=True)
    check_add_norm(q, g, 7, d, dtype, weight=False, strided=True)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 63, 64, 65, 1000, 4099])
@pytest.mark.parametrize("d", [64, 512, 2560])
def test_add_norm_rows(q, n, d):
    g = np.random.default_rng(4100 + n)
    check_add_norm(q, g, n, d, "bf16")
    check_add_norm(q, g, n, d, "bf16", form="int8", group=32)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("form", ["int8", "fp8"])
@pytest.mark.parametrize("d,group", [(8, 0), (72, 0), (520, 0), (2048, 0), (5120, 0), (16384, 0), (32768, 0), (64, 32), (128, 128), (512, 512), (1024, 64),
                                     (1536, 512), (2560, 256), (5120, 128), (10240, 32), (32768, 512)])
def test_add_norm_codes(q, dtype, form, d, group):
    g = np.random.default_rng(4200 + d)
    check_add_norm(q, g, 6, d, dtype, form=form, group=group)
    check_add_norm(q, g, 2, d, dtype, form=form, group=group, residual=False, strided=True, spread=100.0)


@pytest.mark.parametrize("d", [8, 24, 64, 200, 512, 520, 1000, 1024])
def test_add_norm_packed_rows(q, d):
    g = np.random.default_rng(4300 + d)
    check_add_norm(q, g, 9, d, "bf16", form="rows8")
    check_add_norm(q, g, 4, d, "fp16", form="rows8", strided=True, residual=False)
    # exactly the table quantizer's rows where y is exact: a mean square of 1, powers of two
    import torch
    x = torch.from_numpy(np.where(g.random((6, d)) < 0.5, -1.0, 1.0)).bfloat16().cuda()
    w = torch.from_numpy(2.0 ** g.integers(-3, 4, d)).bfloat16().cuda()
    rows, _, _ = q.add_norm(x, None, w, eps=0.0, form="rows8")
    assert torch.equal(rows, q.quantize_rowwise((x.float() * w.float()).contiguous(), 8))


def test_add_norm_in_place(q):
    """The residual stream (or x) takes the sum in its own place."""
    import torch
    g = np.random.default_rng(4400)
    for d in (64, 2048, 5120, 20480):
        xt, _ = rand16(g, (9, d + 8), "bf16")
        rt, _ = rand16(g, (9, d + 16), "bf16")
        w, _ = rand16(g, (d,), "bf16")
        for form in ("values", "int8"):
            want, total, scales = q.add_norm(xt[:, :d], rt[:, :d], w, form=form)
            for which in (0, 1):
                x, r = xt.clone(), rt.clone()
                own = (x, r)[which]
                got, s, _ = q.add_norm(x[:, :d], r[:, :d], w, form=form, sum_out=own[:, :d])
                assert torch.equal(got, want) and torch.equal(own[:, :d], total) and s.data_ptr() == own.data_ptr()
                assert torch.equal(own[:, d:], (xt, rt)[which][:, d:])  # what stands beside the rows stays


def test_add_norm_sum_without_a_residual(q):
    import torch
    g = np.random.default_rng(4410)
    xt, _ = rand16(g, (4, 128), "fp16")
    total = torch.zeros_like(xt)
    _, got, _ = q.add_norm(xt, sum_out=total)
    assert got is total and torch.equal(total, xt)


@pytest.mark.parametrize("form", ["values", "int8", "fp8", "rows8"])
def test_add_norm_rows_of_zeros_and_of_no_numbers(q, form):
    import torch
    d = 512
    x = torch.ones((5, d), dtype=torch.bfloat16, device="cuda")
    x[1] = 0
    x[2, 300], x[3, 20] = float("nan"), float("inf")
    x[4] = 2.0 ** -60
    out, _, s = q.add_norm(x, eps=1e-6, form=form, group=128 if form in ("int8", "fp8") else 0)
    if form == "values":
        assert bool((out[1] == 0).all()) and bool(torch.isnan(out[2]).all()) and bool(torch.isnan(out[3, 20])) and bool((out[0] == 1).all())
    elif form == "rows8":
        assert bool((q.dequantize(out, d, 8)[1] == 0).all())
    else:
        assert bool((out[1].float() == 0).all()) and bool((s[1] == 0).all())
        assert bool(torch.isnan(s[2]).all()) and bool((out[2].float() == 0).all())  # the mean is no number: nor is any element
        assert torch.isnan(s[3]).tolist() == [True, False, False, False] and bool((out[3].float() == 0).all())
        assert bool((out[4].float().abs() > 0).all()) and bool((s[4] > 0).all())
    # a scale below the normal range is none
    if form in ("int8", "fp8"):
        w = torch.full((d,), 2.0 ** -126, dtype=torch.bfloat16, device="cuda")
        w[:128] = 1.0
        out, _, s = q.add_norm(x[:1], None, w, form=form, group=128)
        assert (s[0] > 0).tolist() == [True, False, False, False] and bool((out[0, 128:].float() == 0).all())


def test_add_norm_empty_and_refusals(q):
    import torch
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((4, 64), **bf)
    out, total, s = q.add_norm(x[:0], x[:0], form="int8")
    assert out.shape == (0, 64) and total.shape == (0, 64) and s.shape == (0,)
    for args, more, error in (
        ((x.float(),), {}, TypeError), ((x[0],), {}, TypeError), ((x.cpu(),), {}, TypeError), ((x, x[:3]), {}, ValueError), ((x, x.half()), {}, TypeError),
        ((x.t(),), {}, ValueError), ((x, x, x[0, :32]), {}, ValueError), ((x,), dict(form="int4"), ValueError), ((x,), dict(form="values", group=32), ValueError),
        ((x,), dict(form="int8", group=48), ValueError), ((x,), dict(form="int8", group=16), q.QembError), ((x,), dict(form="int8", group=-32), ValueError),
        ((x,), dict(scales=torch.zeros(4, device="cuda")), ValueError), ((x,), dict(out=torch.zeros((4, 64), device="cuda")), TypeError),
        ((x,), dict(form="int8", scales=torch.zeros(3, device="cuda")), ValueError), ((x,), dict(sum_out=torch.zeros((4, 32), **bf)), ValueError),
        ((torch.zeros((2, 60), **bf),), {}, q.QembError), ((torch.zeros((2, 32776), **bf),), {}, q.QembError),
        ((torch.zeros((2, 1032), **bf),), dict(form="rows8"), q.QembError), ((torch.zeros((3, 68), **bf)[:, :64],), {}, q.QembError),
        ((torch.zeros((3, 72), **bf)[:, 4:68],), {}, q.QembError), ((x,), dict(sum_out=torch.zeros((1, 64), **bf).expand(4, -1)), q.QembError),
    ):
        with pytest.raises(error):
            q.add_norm(*args, **more)
    # one row given to all, and the stride of a single row
    one = torch.ones((1, 64), **bf)
    assert torch.equal(q.add_norm(x, one.expand(4, -1))[1], torch.ones_like(x))
    q.add_norm(torch.zeros((1, 68), **bf)[:, :64])


# ---- log probabilities ----

def check_logprobs(q, x, xv, targets, top, what=""):
    """x on the GPU, xv its float64 values, targets a list or None."""
    import torch
    n, v = xv.shape
    lse = torch.full((n,), 7.0, device="cuda")
    t = None if targets is None else torch.tensor(targets, device="cuda")
    lp, ent, ids, tops = q.token_logprobs(x, t, top=top, lse=lse)
    torch.cuda.synchronize()
    m = xv.max(-1)
    p = np.exp(xv - m[:, None])
    total = p.sum(-1)
    log_total = np.log(total)
    with np.errstate(invalid="ignore"):
        moment = np.where(p > 0, p * (xv - m[:, None]), 0.0).sum(-1) / total
    # sums in binary32 of at most vocab / 256 terms a thread and some joins, each term's power off by 2^-21 of itself
    # (its argument's rounding) at most; differences and logarithms rounded a few times
    rel = (v / 256 + 64) * E + 2.0 ** -21
    close(f64(lse), m + log_total, rel + 4 * E * (np.abs(m) + log_total), what + " lse")
    close(f64(ent), log_total - moment, 2 * rel * (1 + np.abs(moment)) + 8 * E * (1 + log_total), what + " entropy")

    def at(i, j):
        return (xv[i, j] - m[i]) - log_total[i]

    if targets is not None:
        for i, j in enumerate(targets):
            w = at(i, j) if 0 <= j < v else 0.0
            close(f64(lp)[i], np.float64(w), np.float64(rel + 4 * E * (abs(w) + log_total[i]) if np.isfinite(w) else 0.0), what + " logprob")
    else:
        assert lp is None
    if not top:
        assert ids is None and tops is None
        return
    keep = min(top, v)
    got_ids, got = host(ids), f64(tops)
    for i in range(n):
        order = np.lexsort((np.arange(v), -xv[i]))[:keep]
        assert np.array_equal(got_ids[i, :keep], order), (what, i, got_ids[i, :keep], order)
        w = at(i, order)
        close(got[i, :keep], w, np.where(np.isfinite(w), rel + 4 * E * (np.abs(np.where(np.isfinite(w), w, 0)) + log_total[i]), 0.0), what + " top")
    assert (got_ids[:, keep:] == -1).all() and np.isneginf(got[:, keep:]).all()


def rand_logits(g, n, v, dtype, spread=2.5, ruled=0.0):
    import torch
    x = (g.standard_normal((n, v)) * spread).astype(np.float32)
    if ruled:
        x[g.random((n, v)) < ruled] = -np.inf
        x[:, g.integers(0, v)] = 1.0
    t = torch.from_numpy(x)
    t = t if dtype == "fp32" else t.to(torch_type(dtype))
    return t.cuda(), t.double().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("v", [1, 2, 3, 7, 8, 9, 63, 64, 65, 255, 256, 257, 1000, 2047, 2048, 2049, 4100, 16383, 16385, 32768, 50001, 131072, 200003])
def test_logprobs_vocabularies(q, dtype, v):
    g = np.random.default_rng(5000 + v)
    n = 3
    x, xv = rand_logits(g, n, v, dtype)
    check_logprobs(q, x, xv, [int(t) for t in g.integers(0, v, n)], 20, "vocab %d" % v)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 2, 16, 17, 100, 300, 1000, 2500])
def test_logprobs_rows(q, dtype, n):
    g = np.random.default_rng(5100 + n)
    for v in (1500, 9001) if n <= 300 else (1500,):
        x, xv = rand_logits(g, n, v, dtype)
        check_logprobs(q, x, xv, [int(t) for t in g.integers(0, v, n)], 5, "%d rows" % n)


@pytest.mark.parametrize("top", [0, 1, 2, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("v", [40, 700, 30000])
def test_logprobs_tops(q, top, v):
    g = np.random.default_rng(5200 + top)
    for dtype in ("bf16", "fp32"):
        x, xv = rand_logits(g, 4, v, dtype)
        check_logprobs(q, x, xv, None, top, "top %d" % top)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("v", [1000, 40000])
def test_logprobs_ties_go_to_the_lowest_id(q, dtype, v):
    """Rows of few values, of one value, of the two zeros, and large values side by side."""
    import torch
    g = np.random.default_rng(5300)
    x = g.integers(-2, 3, (8, v)).astype(np.float32)
    x[1] = 3.0
    x[2] = np.where(g.random(v) < 0.5, -0.0, 0.0)
    x[3] = -1.0
    x[3, ::2] = 0.5
    x[4] = np.arange(v) // 8 * -0.5  # falling
    x[5] = np.arange(v) // 8 * 0.25  # rising: the largest in one place
    x[6] = 0.0
    x[6, -90:] = 1.0
    x[7] = -5.0
    x[7, 128:128 + 300] = 2.0
    t = torch.from_numpy(x)
    t = t if dtype == "fp32" else t.clamp(-60000, 60000).to(torch_type(dtype))
    check_logprobs(q, t.cuda(), t.double().numpy(), [int(i) for i in g.integers(0, v, 8)], 64, "ties")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_logprobs_ruled_out_tokens(q, dtype):
    """-inf adds nothing; rows with one token left; masks of the type's lowest value."""
    import torch
    g = np.random.default_rng(5400)
    x, xv = rand_logits(g, 6, 5000, dtype, ruled=0.95)
    low = float(torch.finfo(x.dtype).min)
    x[1] = -float("inf")
    x[1, 77] = -3.0
    x[2] = low
    x[2, 4000] = 2.0
    x[3] = low
    xv = f64(x.cpu())
    check_logprobs(q, x, xv, [3, 77, 4000, 12, 0, 4999], 40, "ruled out")
    check_logprobs(q, x, xv, [3, 5, 5, 12, 0, 4999], 40, "ruled-out targets")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("v", [600, 70000])
def test_logprobs_rows_of_no_numbers(q, dtype, v):
    import torch
    g = np.random.default_rng(5500)
    x, xv = rand_logits(g, 6, v, dtype)
    x[0] = -float("inf")
    x[1, 500] = float("nan")
    x[2, 3] = float("inf")
    x[3] = float("nan")
    x[4, v - 1] = -float("nan")
    xv = f64(x.cpu())
    lse = torch.zeros(6, device="cuda")
    lp, ent, ids, tops = q.token_logprobs(x, torch.tensor([5] * 6, device="cuda"), top=9, lse=lse)
    lse, lp, ent, ids, tops = f64(lse), f64(lp), f64(ent), host(ids), f64(tops)
    assert np.isneginf(lse[0]) and np.isneginf(lp[0]) and ent[0] == 0 and np.isneginf(tops[0]).all() and ids[0].tolist() == list(range(9))
    for i in (1, 2, 3, 4):
        assert np.isnan([lse[i], lp[i], ent[i]]).all() and np.isnan(tops[i]).all()
        order = np.lexsort((np.arange(v), -np.where(np.isnan(xv[i]), -np.inf, xv[i])))[:9]
        assert np.array_equal(ids[i], order)
    check_logprobs(q, x[5:], xv[5:], [5], 9, "the clean row")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logprobs_wide_range(q, dtype):
    """Logits in the thousands, one token with all the weight, and all alike."""
    import torch
    g = np.random.default_rng(5550)
    x, xv = rand_logits(g, 4, 3001, dtype, spread=3000.0)
    x[1] = 1e30
    x[2] = -1e30
    x[2, 9] = -1e29
    xv = f64(x.cpu())
    check_logprobs(q, x, xv, [int(np.argmax(xv[0])), 5, 9, 7], 4, "wide")


def test_logprobs_strides_and_alignment(q):
    """Rows of a wider matrix, rows that begin anywhere, one row given to all; what lies beside is not read as logits."""
    import torch
    g = np.random.default_rng(5600)
    for dtype in ("bf16", "fp32"):
        for v, wide, first in ((1000, 1024, 0), (1001, 1001, 0), (4999, 5007, 3), (20001, 20010, 1), (257, 300, 7), (3, 11, 5)):
            x, xv = rand_logits(g, 5, wide, dtype)
            x[:, :first] = 99.0
            x[:, first + v:] = 99.0
            check_logprobs(q, x[:, first:first + v], xv[:, first:first + v], [int(t) for t in g.integers(0, v, 5)], 7, "stride")
    x, xv = rand_logits(g, 1, 3000, "bf16")
    check_logprobs(q, x.expand(70, -1), np.tile(xv, (70, 1)), [5] * 70, 3, "one row for all")


def test_logprobs_targets(q):
    import torch
    g = np.random.default_rng(5700)
    x, xv = rand_logits(g, 6, 900, "bf16")
    targets = [0, 899, -1, 900, -100, 2 ** 31 - 1]
    for index in (torch.int32, torch.int64):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        lp = q.token_logprobs(x, torch.tensor(targets, device="cuda").to(index), err_count=err)[0]
        assert int(err[0]) == 2 and f64(lp)[2:].tolist() == [0, 0, 0, 0]
        check_logprobs(q, x, xv, targets, 0, "targets")
    lp = q.token_logprobs(x, torch.tensor([2 ** 62, -2 ** 62] * 3, device="cuda"))[0]
    assert (f64(lp) == 0).all()


def test_logprobs_past_2_31_elements(q):
    """Rows beyond 2^31 elements (and 2^32 bytes) into the logits."""
    import torch
    g = np.random.default_rng(5750)
    v = 70001
    n = 2 ** 31 // v + 9
    x = torch.zeros((n, v), dtype=torch.bfloat16, device="cuda")
    rows, xv = rand_logits(g, 3, v, "bf16")
    x[[0, n // 2, n - 1]] = rows
    lp, ent, ids, tops = q.token_logprobs(x, torch.full((n,), 11, device="cuda"), top=3)
    want = q.token_logprobs(rows, torch.full((3,), 11, device="cuda"), top=3)
    for a, b in zip((lp, ent, ids, tops), want):
        if a.dtype == torch.int32:
            assert torch.equal(a[[0, n // 2, n - 1]], b)
        else:
            assert float((a[[0, n // 2, n - 1]] - b).abs().max()) < 1e-4  # another split of the same sums


def test_logprobs_equal_calls_streams_and_workspaces(q):
    import torch
    g = np.random.default_rng(5800)
    for n, v, top in ((2, 100000, 20), (1, 131072, 64), (700, 3000, 5), (3, 500, 0)):
        x, _ = rand_logits(g, n, v, "bf16")
        t = torch.from_numpy(g.integers(0, v, n)).cuda()
        want = q.token_logprobs(x, t, top=top)
        need = q.logprobs_workspace_bytes(n, v, torch.bfloat16, top)
        room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = q.token_logprobs(x, t, top=top, workspace=room)
        side.synchronize()
        for a, b in zip(got, want):
            assert a is b or torch.equal(a, b)
        assert bool((room[need:] == 0xA5).all())
        if need:
            with pytest.raises(ValueError):
                q.token_logprobs(x, t, top=top, workspace=room[:need - 1])


def test_captured_calls_replay(q):
    """add_norm and token_logprobs in two graphs that share a workspace, replayed in turn on new inputs."""
    import torch
    g = np.random.default_rng(5900)
    sizes = ((4, 60000, 20), (500, 2500, 3))
    room = torch.empty(max([16] + [q.logprobs_workspace_bytes(n, v, torch.bfloat16, k) for n, v, k in sizes]), dtype=torch.uint8, device="cuda")
    xs = [torch.zeros((n, v), dtype=torch.bfloat16, device="cuda") for n, v, _ in sizes]
    ts = [torch.zeros(n, dtype=torch.int64, device="cuda") for n, _, _ in sizes]
    hs = [torch.zeros((n, 1024), dtype=torch.bfloat16, device="cuda") for n, _, _ in sizes]

    def step(x, t, h, k, room):
        return q.token_logprobs(x, t, top=k, workspace=room) + q.add_norm(h, h, form="fp8", group=128)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i, (_, _, k) in enumerate(sizes):
            step(xs[i], ts[i], hs[i], k, room)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i, (_, _, k) in enumerate(sizes):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(xs[i], ts[i], hs[i], k, room))
        graphs.append(graph)
    for rep in range(4):
        print("graph replay %d" % rep, flush=True)
        for i in ((0, 1) if rep % 2 else (1, 0)):
            n, v, k = sizes[i]
            xs[i].copy_(rand_logits(g, n, v, "bf16", ruled=0.3 * rep)[0])
            ts[i].copy_(torch.from_numpy(g.integers(0, v, n)))
            hs[i].copy_(rand16(g, (n, 1024), "bf16")[0])
            graphs[i].replay()
            torch.cuda.synchronize()
            want = step(xs[i].clone(), ts[i].clone(), hs[i].clone(), k, None)
            torch.cuda.synchronize()
            for a, b in zip(outs[i], want):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (rep, i)


def test_logprobs_empty_and_refusals(q):
    import torch
    x = torch.zeros((3, 40), dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(3, dtype=torch.int64, device="cuda")
    lp, ent, ids, tops = q.token_logprobs(x[:0], t[:0], top=4)
    assert lp.shape == (0,) and ent.shape == (0,) and ids.shape == (0, 4) and tops.shape == (0, 4)
    for args, more, error in (
        ((x.cpu(),), {}, TypeError), ((x[0],), {}, TypeError), ((x.double(),), {}, TypeError), ((x.t(),), {}, ValueError), ((x, t[:2]), {}, ValueError),
        ((x, t.float()), {}, TypeError), ((x, t.cpu()), {}, TypeError), ((x,), dict(top=65), ValueError), ((x,), dict(top=-1), ValueError),
        ((x[:, :0],), {}, q.QembError), ((x,), dict(lse=torch.zeros(2, device="cuda")), ValueError), ((x,), dict(err_count=t[:1]), TypeError),
        ((x,), dict(workspace=torch.zeros(1 << 20, device="cuda")), TypeError),
    ):
        with pytest.raises(error):
            q.token_logprobs(*args, **more)


def test_logprobs_any_nan_is_passed_over(q):
    """NaN of every kind (quiet or not, of either sign) beside large logits: the ids stand."""
    import torch
    g = np.random.default_rng(6000)
    for v in (700, 20000):
        x = (g.standard_normal((4, v)) * 2).astype(np.float32)
        for dtype, kind, bits in ((torch.bfloat16, torch.int16, (0x7F81, -0x7F, 0x7FC0, -0x40)), (torch.float16, torch.int16, (0x7C01, -0x3FF, 0x7E00, -0x200)),
                                  (torch.float32, torch.int32, (0x7F800001, -0x7FFFFF, 0x7FC00000, -0x400000))):
            t = torch.from_numpy(x).to(dtype)
            places = g.choice(v, 60, replace=False)
            raw = t.view(kind)
            for i, at in enumerate(places):
                raw[i % 4, int(at)] = bits[i // 4 % 4]
            xv = t.double().numpy()
            assert np.isnan(xv).sum() == 60
            _, ent, ids, tops = q.token_logprobs(t.cuda(), top=12)
            assert np.isnan(f64(ent)).all() and np.isnan(f64(tops)).all()
            for i in range(4):
                order = np.lexsort((np.arange(v), -np.where(np.isnan(xv[i]), -np.inf, xv[i])))[:12]
                assert np.array_equal(host(ids)[i], order), (dtype, v, i)


def test_logprobs_largest_at_every_place(q):
    """One logit above all others, at every border of vectors, slices, chunks and parts."""
    import torch
    v = 40001
    for dtype in (torch.bfloat16, torch.float32):
        each = 8 if dtype is torch.bfloat16 else 4
        places = sorted({p for base in (0, each, 64 * each, 256 * each, 512 * each, 1024 * each, 2048 * each, v) for p in (base - 1, base, base + 1) if 0 <= p < v})
        x = torch.zeros((len(places), v), dtype=dtype, device="cuda")
        at = torch.tensor(places, device="cuda")
        x[torch.arange(len(places)), at] = 9.0
        lp, ent, ids, tops = q.token_logprobs(x, at, top=2)
        want = 9.0 - np.log(np.exp(9.0) + v - 1)
        assert torch.equal(ids[:, 0], at.int()) and ids[:, 1].tolist() == [1 if p == 0 else 0 for p in places]
        assert float((lp - want).abs().max()) < 1e-4 and torch.equal(lp, tops[:, 0])


def test_logprobs_rising_and_falling_rows(q):
    """Rows whose largest logits come last, or all in one thread's vectors, so that bounds keep moving."""
    g = np.random.default_rng(6100)
    import torch
    v = 60000
    x = np.stack([np.arange(v) * 1e-3, np.arange(v)[::-1] * 1e-3, np.where(np.arange(v) % 2048 < 8, 5.0, 0.0) + np.arange(v) * 1e-6,
                  np.repeat(np.arange(v // 100), 100) * 0.05]).astype(np.float32)
    for top in (1, 20, 64):
        t = torch.from_numpy(x)
        check_logprobs(q, t.cuda(), t.double().numpy(), [int(i) for i in g.integers(0, v, 4)], top, "rising")
        t = t.bfloat16()
        check_logprobs(q, t.cuda(), t.double().numpy(), [int(i) for i in g.integers(0, v, 4)], top, "rising, 16 bits")
