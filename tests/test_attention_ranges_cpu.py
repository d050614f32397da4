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


@pytest.mark.parametrize("page,width", [(1, MOST), (16, 2 ** 27 - 1), (512, 2 ** 22 - 1)])
def test_decode_tables_near_2_31_slots_are_refused(lib, page, width):  # noqa: F811
    assert call(lib.qemb_decode_attention, DECODE, page=page, width=width, mass=None) == -3
    assert call(lib.qemb_decode_attention, DECODE, page=page, width=width, window=100) == -3
    assert lib.qemb_decode_workspace_bytes(2, 4, 2, 64, width, page, 0, 0, 1) == 0
    assert lib.qemb_decode_workspace_bytes(2, 4, 2, 64, (2 ** 31 - 1024) // page, page, 0, 0, 1) > 0


@pytest.mark.parametrize("change", [
    dict(page=1, width=MOST, mass_len=MOST, new_width=20), dict(page=16, width=2 ** 27 - 1, mass_len=MOST - 15),
    dict(page=512, width=2 ** 22 - 1, mass_len=MOST - 1022),
])
def test_evict_slots_near_2_31_are_refused(lib, change):  # noqa: F811
    assert call(lib.qemb_evict, EVICT, **change) == -3


@pytest.mark.parametrize("change", [
    dict(hq=2 ** 30, hkv=2 ** 29), dict(hq=MOST), dict(hq=MOST - 1030, hkv=8), dict(hkv=MOST),
    dict(hq=2 ** 30, hkv=2 ** 30, v=None, k_pages=None, v_pages=None),
])
def test_norm_rope_heads_near_2_31_are_refused(lib, change):  # noqa: F811
    assert call(lib.qemb_norm_rope, NORM, **change) == -3


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_scales_that_are_not_finite_are_refused(lib, scale):  # noqa: F811
    assert call(lib.qemb_prompt_attention, PROMPT, scale=scale) == -1
    assert call(lib.qemb_decode_attention, DECODE, scale=scale) == -1
