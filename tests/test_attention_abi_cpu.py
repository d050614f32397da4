"""libqemb_attention: the exports that include/qemb_attention.h declares, and
the refusals of bad arguments on the host (no compute call here)."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

from int4_row_wise_amd import attention
from int4_row_wise_amd import build as qbuild

FAKE = 1 << 20   # never dereferenced: validation fails first
MIS = FAKE + 2   # aligned for 16-bit values only


@pytest.fixture(scope="module")
def lib():
    qbuild.ensure_built()
    return attention.load_attention_library()


def test_every_declared_symbol_is_exported(lib):
    with open(qbuild.ATTN_HEADER) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    syms = sorted(set(re.findall(r"\b(qemb_[a-z0-9_]+)\s*\(", src)))
    assert syms == sorted(attention.EXPORTED)
    for s in syms:
        assert hasattr(lib, s), s


def call(fn, defaults, **change):
    assert not set(change) - set(defaults)
    return fn(*(defaults | change).values())


NORM = dict(q=FAKE, k=FAKE, v=FAKE, tokens=4, hq=4, hkv=2, dim=64, dtype=0, qt=256, qh=64, kt=128, kh=64, vt=128, vh=64,
            positions=FAKE, itype=0, cos_sin=FAKE, places=50, rot=64, inter=0, wq=None, wk=None, eps=1e-6, q_out=FAKE, k_out=FAKE,
            k_pages=FAKE, v_pages=FAKE, slots=FAKE, pages=3, page=16, bits=16, err=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(tokens=-1), -1), (dict(hq=0), -1), (dict(hkv=0), -1), (dict(dim=0), -1), (dict(dtype=2), -1), (dict(itype=2), -1),
    (dict(dim=264, rot=64), -3), (dict(dim=60, rot=16), -3), (dict(rot=24), -3), (dict(rot=80), -1), (dict(rot=-16), -1),
    (dict(places=-1), -1), (dict(pages=-1), -1), (dict(page=0), -1), (dict(page=12), -1), (dict(bits=2), -1), (dict(bits=32), -1),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(q_out=None), -1), (dict(positions=None), -1),
    (dict(cos_sin=None), -1), (dict(slots=None), -1), (dict(k_pages=None), -1), (dict(v_pages=None), -1),
    (dict(k_pages=None, v_pages=None, k_out=None), -1),
    (dict(q=MIS), -2), (dict(k=MIS), -2), (dict(v=MIS), -2), (dict(q_out=MIS), -2), (dict(k_out=MIS), -2), (dict(wq=MIS), -2),
    (dict(wk=MIS), -2), (dict(k_pages=MIS), -2), (dict(cos_sin=MIS), -2), (dict(slots=MIS), -2), (dict(positions=MIS), -2),
    (dict(qt=260), -2), (dict(kh=4), -2), (dict(vt=-8), -2), (dict(tokens=0, q=None), 0),
])
def test_norm_rope_refusals(lib, change, rc):
    assert call(lib.qemb_norm_rope, NORM, **change) == rc


PROMPT = dict(q=FAKE, k=FAKE, v=FAKE, nq=100, nk=100, batch=2, hq=4, hkv=2, dim=64, dtype=1, qt=256, qh=64, kt=128, kh=64, vt=128, vh=64,
              qo=FAKE, ko=FAKE, max_q=50, window=0, sinks=0, scale=0.125, out=FAKE, lse=FAKE, err=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(nq=-1), -1), (dict(nk=-1), -1), (dict(batch=-1), -1), (dict(hq=5), -1), (dict(dtype=3), -1), (dict(window=-1), -1),
    (dict(sinks=-1), -1), (dict(max_q=-1), -1), (dict(dim=512), -3), (dict(dim=20), -3), (dict(nq=2 ** 31), -3), (dict(nk=2 ** 31), -3),
    (dict(q=None), -1), (dict(k=None), -1), (dict(out=None), -1), (dict(qo=None), -1), (dict(ko=None), -1),
    (dict(q=MIS), -2), (dict(v=MIS), -2), (dict(out=MIS), -2), (dict(lse=MIS), -2), (dict(qo=MIS), -2), (dict(kt=4), -2), (dict(qh=-64), -2),
    (dict(nq=0, q=None), 0), (dict(batch=0), 0),
])
def test_prompt_refusals(lib, change, rc):
    assert call(lib.qemb_prompt_attention, PROMPT, **change) == rc


DECODE = dict(q=FAKE, k=FAKE, v=FAKE, pages=9, page=16, bits=16, batch=2, hq=4, hkv=2, dim=64, dtype=0, table=FAKE, width=4, lens=FAKE,
              window=0, sinks=0, scale=0.125, mass=FAKE, mass_len=64, out=FAKE, lse=FAKE, ws=FAKE, err=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(batch=-1), -1), (dict(width=-1), -1), (dict(pages=-1), -1), (dict(page=24), -1), (dict(page=0), -1), (dict(bits=2), -1),
    (dict(hq=3), -1), (dict(dtype=-1), -1), (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(mass_len=-1), -1),
    (dict(dim=300), -3), (dict(dim=257), -3), (dict(dim=36), -3), (dict(page=1024, width=2 ** 21), -3),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(out=None), -1), (dict(lens=None), -1), (dict(table=None), -1),
    (dict(ws=None), -1), (dict(q=MIS), -2), (dict(k=MIS), -2), (dict(out=MIS), -2), (dict(ws=MIS), -2), (dict(mass=MIS), -2),
    (dict(table=MIS), -2), (dict(lens=MIS), -2), (dict(batch=0, q=None), 0),
])
def test_decode_refusals(lib, change, rc):
    assert call(lib.qemb_decode_attention, DECODE, **change) == rc


def test_decode_workspace(lib):
    w = lib.qemb_decode_workspace_bytes
    #      batch hq hkv dim width page window sinks mass
    assert w(2, 4, 2, 64, 4, 16, 0, 0, 1) > 0
    assert w(2, 4, 2, 64, 4, 16, 8, 2, 1) <= w(2, 4, 2, 64, 4, 16, 0, 0, 1)
    for bad in ((0, 4, 2, 64, 4, 16, 0, 0, 1), (2, 5, 2, 64, 4, 16, 0, 0, 1), (2, 4, 2, 64, 4, 15, 0, 0, 1), (2, 4, 2, 64, 0, 16, 0, 0, 1)):
        assert w(*bad) == 0


EVICT = dict(k=FAKE, v=FAKE, pages=9, page=16, row=128, batch=2, hkv=2, table=FAKE, width=4, lens=FAKE, mass=FAKE, mass_len=64, keep=20,
             sinks=2, recent=4, nk=FAKE, nv=FAKE, new_pages=5, new_table=FAKE, new_width=2, kept=FAKE, new_mass=FAKE, new_mass_len=20,
             new_lens=FAKE, err=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(batch=-1), -1), (dict(hkv=0), -1), (dict(pages=-1), -1), (dict(new_pages=-1), -1), (dict(width=-1), -1), (dict(page=3), -1),
    (dict(mass_len=-1), -1), (dict(keep=0), -1), (dict(sinks=-1), -1), (dict(recent=-1), -1), (dict(sinks=17), -1), (dict(row=8), -1),
    (dict(keep=33), -1), (dict(new_mass_len=19), -1), (dict(row=136), -2), (dict(row=1 << 17), -3),
    (dict(lens=None), -1), (dict(new_table=None), -1), (dict(kept=None), -1), (dict(new_mass=None), -1), (dict(new_lens=None), -1),
    (dict(table=None), -1), (dict(mass=None), -1), (dict(k=None), -1), (dict(nv=None), -1), (dict(k=MIS), -2), (dict(nk=MIS), -2),
    (dict(mass=MIS), -2), (dict(kept=MIS), -2), (dict(batch=0, lens=None), 0),
])
def test_evict_refusals(lib, change, rc):
    assert call(lib.qemb_evict, EVICT, **change) == rc


def test_cpu_tensors_are_refused(lib):
    t = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        attention.prompt_attention(t, t, t, i, i)
    with pytest.raises(TypeError):
        attention.norm_rope(t, t, i, torch.zeros((4, 64)))
    with pytest.raises(TypeError):
        attention.decode_attention(t, t, t, i, i)
    with pytest.raises(TypeError):
        attention.evict(t, t, i, i, t, 4, t, t, i)


def test_library_from_other_sources_is_refused(lib, tmp_path, monkeypatch):
    """A library whose recorded source hash differs is refused before it loads."""
    import shutil
    stale = tmp_path / "libqemb_attention.so"
    shutil.copy(qbuild.ATTN_LIB, stale)
    with open(str(stale) + ".srchash", "w") as f:
        f.write("0" * 64 + "\n")
    monkeypatch.setattr(attention, "_lib", None)
    with pytest.raises(attention.QembError, match="other kernel sources"):
        attention.load_attention_library(str(stale))
    os.remove(str(stale))
    with pytest.raises(attention.QembError, match="not built"):
        attention.load_attention_library(str(stale))
    assert isinstance(attention.load_attention_library(), ctypes.CDLL)
