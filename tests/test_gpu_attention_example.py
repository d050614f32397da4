"""The serving example runs its whole path on the GPU: lookup, norm + rotation
+ append, prompt attention, one-token attention over INT8 pages, eviction."""
from __future__ import annotations

import importlib.util
import os

import pytest

from tests.gpu_common import require_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_serving_example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("cached_attention", os.path.join(ROOT, "examples", "cached_attention.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.main(verbose=False)
    # prompts: two bfloat16 roundings; steps: an INT8 row's half step (range / 510 of values about range / 5)
    # on keys and values
    assert r["errors"]["prompt"] < 2 * 2.0 ** -8 and r["errors"]["step"] < 0.05
    assert r["cuts"] >= 1 and r["finite"] and max(r["lens"]) <= example.BUDGET
    assert r["mass"] > 0
