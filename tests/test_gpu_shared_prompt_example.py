"""The example that draws many answers to one prompt runs its whole path on the
GPU: residual addition + norm, rotation by several axes + append, prompt
attention, attention over the shared prefix, log probabilities."""
from __future__ import annotations

import importlib.util
import os

import pytest

from tests.gpu_common import require_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("answers,steps", [(12, 6), (1, 20), (40, 2)])
def test_shared_prompt_example(answers, steps):
    require_gpu()
    spec = importlib.util.spec_from_file_location("shared_prompt", os.path.join(ROOT, "examples", "shared_prompt.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.main(answers=answers, steps=steps, verbose=False)
    # bfloat16 roundings of the turned queries and keys (which move the weights), of the weights and of the output
    assert r["errors"]["prompt"] < 4 * 2.0 ** -8 and r["errors"]["step"] < 4 * 2.0 ** -8
    # sums of 4000 terms in 32 bits, twice, of values around 10
    assert r["errors"]["logprob"] < 1e-4
    assert len(r["scores"]) == answers and all(-1e3 < s < 0 for s in r["scores"]) and len(r["top"][0]) == 4
