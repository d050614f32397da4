"""libqemb_attention at the ends of its arguments' ranges: what the host refuses
because the kernels' 32-bit counts do not hold it (no compute call here)."""
from __future__ import annotations

import pytest

from tests.test_attention_abi_cpu import DECODE, EVICT, NORM, PROMPT, call, lib  # noqa: F401

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("change", [
    dict(nq=MOST), dict(nq=MOST - 100), dict(nk=MOST), dict(nk=MOST - 100),
    dict(nq=MOST // 4, hq=4, hkv=1),  # (token, head of the group) rows
    dict(nq=MOST // 2, hq=4, hkv=2, window=7, sinks=MOST),
])
def test_prompt_rows_and_keys_near_2_31_are_refused(lib, change):  # noqa: F811
    assert call(lib.qemb_prompt_attention, PROMPT, **change) == -3
