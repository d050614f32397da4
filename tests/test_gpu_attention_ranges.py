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
