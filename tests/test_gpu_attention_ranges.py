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
