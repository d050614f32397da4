"""libqemb_serving, and the attention library's rotation by several axes and
attention over shared prefixes: exports, and the refusals of bad arguments on
the host (no compute call here)."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

from int4_row_wise_amd import build as qbuild
from int4_row_wise_amd import serving
from tests.test_attention_abi_cpu import FAKE, MIS, NORM, call
from tests.test_attention_abi_cpu import lib as attention_lib  # noqa: F401

MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    qbuild.ensure_built()
    return serving.load_serving_library()


def test_every_declared_symbol_is_exported(lib):
    with open(qbuild.SERVING_HEADER) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    syms = sorted(set(re.findall(r"\b(qemb_[a-z0-9_]+)\s*\(", src)))
    assert syms == sorted(serving.EXPORTED)
    for s in syms:
        assert hasattr(lib, s), s


ADD_NORM = dict(x=FAKE, residual=FAKE, weight=FAKE, rows=4, dim=256, dtype=0, xs=256, rs=256, ss=256, eps=1e-6, form=0, group=0, out=FAKE,
                scales=None, sum_out=FAKE, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(rows=-1), -1), (dict(dim=0), -1), (dict(dtype=2), -1), (dict(dtype=-1), -1), (dict(form=4), -1), (dict(form=-1), -1),
    (dict(group=128), -1), (dict(form=3, group=128), -1), (dict(form=1, group=48, scales=FAKE), -1), (dict(form=1, group=16, scales=FAKE), -1),
    (dict(form=1, group=1024, dim=1024, scales=FAKE), -1), (dict(form=2, group=-32, scales=FAKE), -1), (dict(form=1, group=128, dim=192, scales=FAKE), -1),
    (dict(form=1), -1), (dict(form=2), -1), (dict(dim=252), -3), (dict(dim=32776), -3), (dict(form=3, dim=1032), -3), (dict(rows=2 ** 24), -3),
    (dict(xs=252), -2), (dict(xs=-256), -2), (dict(rs=260), -2), (dict(ss=248), -2), (dict(ss=252), -2), (dict(ss=260), -2),
    (dict(x=None), -1), (dict(out=None), -1), (dict(x=MIS), -2), (dict(residual=MIS), -2), (dict(weight=MIS), -2), (dict(out=MIS), -2),
    (dict(sum_out=MIS), -2), (dict(form=1, scales=MIS), -2), (dict(rows=0, x=None), 0), (dict(rows=0, form=1, scales=FAKE, out=None), 0),
])
def test_add_norm_refusals(lib, change, rc):
    assert call(lib.qemb_add_norm, ADD_NORM, **change) == rc


LOGPROBS = dict(logits=FAKE, rows=4, vocab=1000, dtype=0, stride=1000, targets=FAKE, itype=1, top=5, logprobs=FAKE, entropy=FAKE, lse=FAKE,
                ids=FAKE, tops=FAKE, ws=FAKE, err=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(rows=-1), -1), (dict(vocab=0), -1), (dict(vocab=-5), -1), (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(top=-1), -1), (dict(top=65), -1),
    (dict(itype=2), -1), (dict(stride=-1), -1), (dict(vocab=2 ** 30 + 1), -3), (dict(rows=2 ** 24), -3), (dict(logits=None), -1), (dict(targets=None), -1),
    (dict(logprobs=None), -1), (dict(ids=None), -1), (dict(tops=None), -1), (dict(logits=FAKE + 1), -2), (dict(logits=MIS, dtype=2), -2),
    (dict(targets=FAKE + 4), -2), (dict(targets=MIS, itype=0), -2), (dict(logprobs=MIS), -2), (dict(entropy=MIS), -2), (dict(lse=MIS), -2),
    (dict(ids=MIS), -2), (dict(tops=MIS), -2), (dict(ws=FAKE + 8), -2), (dict(rows=0, logits=None), 0),
    (dict(rows=1, vocab=200000, ws=None), -1),
])
def test_logprobs_refusals(lib, change, rc):
    assert call(lib.qemb_token_logprobs, LOGPROBS, **change) == rc


def test_logprobs_workspace(lib):
    w = lib.qemb_logprobs_workspace_bytes
    assert w(1, 200000, 0, 20) > 0
    for bad in ((0, 1000, 0, 5), (4, 0, 0, 5), (4, 2 ** 30 + 1, 0, 5), (4, 1000, 3, 5), (4, 1000, 0, 65), (4, 1000, 0, -1)):
        assert w(*bad) == 0
    assert w(2 ** 24 - 1, 2 ** 30, 2, 64) < 2 ** 50  # no overflow at the largest sizes


AXES = {k: v for k, v in NORM.items()}
AXES = dict(list(AXES.items())[:15] + [("axes", 3), ("pair_axes", FAKE)] + list(AXES.items())[15:20] + [("norm", 1)] + list(AXES.items())[20:])


@pytest.mark.parametrize("change,rc", [
    (dict(axes=0), -1), (dict(axes=-1), -1), (dict(axes=5), -1), (dict(pair_axes=None), -1), (dict(pair_axes=MIS), -2), (dict(norm=0, wq=FAKE), -1),
    (dict(norm=0, wk=FAKE), -1), (dict(rot=24), -3), (dict(rot=80), -1), (dict(positions=None), -1), (dict(tokens=-1), -1), (dict(cos_sin=None), -1),
    (dict(tokens=0, q=None), 0), (dict(tokens=0, axes=1, pair_axes=None, norm=0), 0), (dict(tokens=0, axes=4, pair_axes=None, rot=0), 0),
])
def test_norm_rope_axes_refusals(attention_lib, change, rc):  # noqa: F811
    assert call(attention_lib.qemb_norm_rope_axes, AXES, **change) == rc


SHARED = dict(q=FAKE, k=FAKE, v=FAKE, pages=9, page=16, bits=16, batch=3, hq=4, hkv=2, dim=64, dtype=0, prefix=FAKE, prefix_width=8, prefix_lens=FAKE,
              offsets=FAKE, groups=2, table=FAKE, width=4, lens=FAKE, scale=0.125, out=FAKE, lse=FAKE, ws=FAKE, err=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(batch=-1), -1), (dict(width=-1), -1), (dict(prefix_width=-1), -1), (dict(pages=-1), -1), (dict(groups=0), -1), (dict(page=24), -1), (dict(page=0), -1),
    (dict(bits=2), -1), (dict(hq=3), -1), (dict(dtype=2), -1), (dict(offsets=None), -1), (dict(dim=300), -3), (dict(dim=36), -3),
    (dict(page=1024, width=2 ** 21), -3), (dict(page=1024, prefix_width=2 ** 21), -3), (dict(page=1, prefix_width=MOST), -3), (dict(batch=MOST, hq=2, hkv=1), -3),
    (dict(page=2 ** 26, width=1, prefix_width=1), -3), (dict(scale=float("nan")), -1), (dict(scale=-float("inf")), -1),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(out=None), -1), (dict(lens=None), -1), (dict(prefix_lens=None), -1),
    (dict(table=None), -1), (dict(prefix=None), -1), (dict(ws=None), -1), (dict(q=MIS), -2), (dict(k=MIS), -2), (dict(out=MIS), -2), (dict(ws=MIS), -2),
    (dict(table=MIS), -2), (dict(prefix=MIS), -2), (dict(prefix_lens=MIS), -2), (dict(offsets=MIS), -2), (dict(lens=MIS), -2), (dict(lse=MIS), -2),
    (dict(batch=0, q=None), 0),
])
def test_shared_refusals(attention_lib, change, rc):  # noqa: F811
    assert call(attention_lib.qemb_shared_attention, SHARED, **change) == rc


def test_shared_workspace(attention_lib):  # noqa: F811
    w = attention_lib.qemb_shared_workspace_bytes
    #      batch hq hkv dim groups prefix_width width page bits
    assert w(3, 4, 2, 64, 2, 8, 4, 16, 16) > 0
    for bad in ((0, 4, 2, 64, 1, 8, 4, 16, 16), (3, 5, 2, 64, 1, 8, 4, 16, 16), (3, 4, 2, 64, 0, 8, 4, 16, 16), (3, 4, 2, 64, 1, -1, 4, 16, 16),
                (3, 4, 2, 64, 1, 8, -1, 16, 16), (3, 4, 2, 64, 1, 8, 4, 15, 16), (3, 4, 2, 64, 1, 2 ** 27, 4, 16, 16), (3, 4, 2, 64, 1, 8, 4, 16, 5)):
        assert w(*bad) == 0


def test_cpu_tensors_are_refused(lib):
    import int4_row_wise_amd as q
    t = torch.zeros((2, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 3), dtype=torch.int32)
    with pytest.raises(TypeError):
        q.add_norm(t)
    with pytest.raises(TypeError):
        q.token_logprobs(t)
    with pytest.raises(TypeError):
        q.shared_attention(t[None], t, t, i, i[0], i, i[0])


def test_library_from_other_sources_is_refused(lib, tmp_path, monkeypatch):
    """A library whose recorded source hash differs is refused before it loads."""
    import shutil
    stale = tmp_path / "libqemb_serving.so"
    shutil.copy(qbuild.SERVING_LIB, stale)
    with open(str(stale) + ".srchash", "w") as f:
        f.write("0" * 64 + "\n")
    monkeypatch.setattr(serving, "_lib", None)
    with pytest.raises(serving.QembError, match="other kernel sources"):
        serving.load_serving_library(str(stale))
    os.remove(str(stale))
    with pytest.raises(serving.QembError, match="not built"):
        serving.load_serving_library(str(stale))
    assert isinstance(serving.load_serving_library(), ctypes.CDLL)


def test_launches_make_the_tensors_gpu_current(monkeypatch):
    """A call for another GPU than the current one runs with that one current, and only such a call."""
    import contextlib

    from int4_row_wise_amd import attention
    entered = []

    @contextlib.contextmanager
    def device(index):
        entered.append(index)
        yield

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    assert attention._launch(0, lambda *a: sum(a), 1, 2) == 3 and entered == []
    assert attention._launch(2, lambda *a: sum(a), 1, 2) == 3 and entered == [2]


@pytest.mark.parametrize("scale,rc", [(3e38, -1), (-3e38, -1), (2.36e38, -1), (2.35e38, 0), (-2.35e38, 0), (0.0, 0), (1e-45, 0)])
def test_scales_whose_powers_of_two_overflow_are_refused(attention_lib, scale, rc):  # noqa: F811
    """Scores are taken as powers of two: a scale times log2 e past binary32 would make even scores of 0 a NaN."""
    from tests.test_attention_abi_cpu import DECODE, PROMPT
    assert call(attention_lib.qemb_prompt_attention, PROMPT, scale=scale, batch=0) == rc
    assert call(attention_lib.qemb_decode_attention, DECODE, scale=scale, batch=0) == rc
    assert call(attention_lib.qemb_shared_attention, SHARED, scale=scale, batch=0) == rc
