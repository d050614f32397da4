"""Every call runs with its tensors' GPU as the current one (CPU only: the
library and the tensors' place are stood in for, nothing is computed)."""
from __future__ import annotations

import contextlib

import pytest
import torch

import int4_row_wise_amd as q
from int4_row_wise_amd import attention, serving

FAR = 2  # the tensors' GPU; the current one is 0


class Far(torch.Tensor):
    """A tensor that says that it is on GPU FAR."""
    is_cuda = True

    def get_device(self):
        return FAR


def far(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(Far)


def ints(*shape):
    return far(*shape, dtype=torch.int32)


@pytest.fixture
def calls(monkeypatch):
    """(entry point, the GPU that is current) of every call that enqueues work."""
    seen, current = [], [0]

    @contextlib.contextmanager
    def device(index):
        was, current[0] = current[0], index if isinstance(index, int) else index.index
        yield
        current[0] = was

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                if name.endswith("_bytes"):
                    return 64
                seen.append((name, current[0]))
                return 0
            return entry

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    for module in (attention, serving):
        monkeypatch.setattr(module, "_lib", Library())
        monkeypatch.setattr(module, "_raw_stream", lambda index: 0)
    return seen


def heads():
    return far(5, 4, 64), far(5, 2, 64), far(5, 2, 64)


def pool(n=6):
    return far(n, 2, 16, 64), far(n, 2, 16, 64)


def test_norm_rope(calls):
    x, k, v = heads()
    pages = pool()
    table, slots = far(50, 64, dtype=torch.float32), far(5, dtype=torch.int64)
    q.norm_rope(x, k, ints(5), table, k_out=far(5, 2, 64))
    q.norm_rope(x, k, ints(5), table, v=v, k_pages=pages[0], v_pages=pages[1], slots=slots)
    q.norm_rope(x, k, ints(5), table, norm=False, k_out=far(5, 2, 64))
    q.norm_rope(x, k, ints(3, 5), table, pair_axes=far(32, dtype=torch.uint8), k_out=far(5, 2, 64))
    assert calls == [("qemb_norm_rope", FAR)] * 2 + [("qemb_norm_rope_axes", FAR)] * 2


def test_attention(calls):
    x, k, v = heads()
    pages = pool()
    q.prompt_attention(x, k, v, ints(3), ints(3))
    q.decode_attention(x, *pages, ints(5, 2), ints(5))
    q.shared_attention(x, *pages, ints(1, 2), ints(1), ints(5, 2), ints(5))
    assert calls == [(n, FAR) for n in ("qemb_prompt_attention", "qemb_decode_attention", "qemb_shared_attention")]


def test_evict(calls):
    q.evict(*pool(), ints(3, 2), ints(3), far(3, 2, 32, dtype=torch.float32), 16, *pool(), ints(3, 1))
    assert calls == [("qemb_evict", FAR)]


def test_serving(calls):
    q.add_norm(far(4, 64), far(4, 64))
    q.token_logprobs(far(4, 100), far(4, dtype=torch.int64), top=2)
    assert calls == [("qemb_add_norm", FAR), ("qemb_token_logprobs", FAR)]


@pytest.fixture
def tables(calls, monkeypatch):
    """The table library stood in for, too: a row of 64 elements has 48 bytes."""
    from int4_row_wise_amd import qemb

    class Library:
        def __getattr__(self, name):
            if name.endswith("_stride"):
                return lambda *args: 48
            if name.endswith(("_bound", "_bytes", "_width")):
                return lambda *args: 64
            return getattr(attention._lib, name)

    monkeypatch.setattr(qemb, "_lib", Library())
    monkeypatch.setattr(qemb, "_stream", lambda t: 0)
    return calls


def test_tables(tables):
    f32, u8, i64 = torch.float32, torch.uint8, torch.int64
    x, rows = far(3, 64, dtype=f32), far(3, 48, dtype=u8)
    q.quantize_rowwise(x, 4, out=rows)
    q.quantize_baseline(x, 4, out=rows)
    q.dequantize(rows, 64, 4, out=x)
    q.quantize_codebook(x, out=rows)
    q.dequantize_codebook(rows, 64, out=x)
    ids, spans, pooled = far(4, dtype=i64), far(3, dtype=i64), far(2, 1, 64, dtype=f32)
    q.bag_forward(rows, far(2, dtype=i64), 2, 64, 4, ids, spans, out=pooled)
    q.bag_forward_codebook(rows, far(2, dtype=i64), 2, 64, ids, spans, out=pooled)
    room4 = dict(workspace=far(64, dtype=u8), out4=far(4, dtype=torch.float64))
    q.l2_error(x, rows, 4, **room4)
    q.l2_error_codebook(x, rows, **room4)
    q.dot_interaction(far(3, 64, dtype=f32), far(3, 2, 64, dtype=f32), out=far(3, 64, dtype=f32))
    eb, offs, room = far(1, dtype=f32), far(4, dtype=i64), far(64, dtype=u8)
    q.compress_pooled(x, eb, T=1, out=room, offs=offs, workspace=room)
    q.compress_pooled_noalloc(x, eb, room, offs, T=1)
    q.decompress_pooled(room, offs, 64, eb, y=x)
    assert [place for _, place in tables] == [FAR] * 13 and len({name for name, _ in tables}) == 13


def test_tables_refuse_arrays_too_small(tables):
    """What a kernel would write past is refused before anything is enqueued."""
    f32, u8, i32, i64 = torch.float32, torch.uint8, torch.int32, torch.int64
    x, rows, small = far(3, 64, dtype=f32), far(3, 48, dtype=u8), far(2, 64, dtype=f32)
    bag = (far(2, dtype=i64), 4, 64)
    ids, spans = far(4, dtype=i64), far(5, dtype=i64)
    none, offs, eb = far(0, dtype=i32), far(4, dtype=i64), far(1, dtype=f32)
    for call in (
        lambda: q.dequantize(rows, 64, 4, out=small),
        lambda: q.dequantize_codebook(rows, 64, out=small),
        lambda: q.bag_forward(rows, *bag, 4, ids, spans, out=x),
        lambda: q.bag_forward(rows, *bag, 4, ids, spans, out=far(4, 1, 64, dtype=f32), err_count=none),
        lambda: q.bag_forward_codebook(rows, *bag, ids, spans, out=x),
        lambda: q.l2_error(x, rows, 4, workspace=far(63, dtype=u8)),
        lambda: q.l2_error(x, rows, 4, out4=far(3, dtype=torch.float64)),
        lambda: q.l2_error_codebook(x, rows, workspace=far(63, dtype=u8)),
        lambda: q.l2_error_codebook(x, rows, out4=far(3, dtype=torch.float64)),
        lambda: q.decompress_pooled(far(64, dtype=u8), offs, 64, eb, y=x, err_count=none),
    ):
        with pytest.raises(ValueError):
            call()
    assert tables == []


def test_tables_refuse_tensors_of_several_gpus(tables):
    f32, u8, i64 = torch.float32, torch.uint8, torch.int64

    class Elsewhere(Far):
        def get_device(self):
            return FAR + 1

    def other(*shape, dtype):
        return torch.zeros(shape, dtype=dtype).as_subclass(Elsewhere)

    x, rows = far(3, 64, dtype=f32), far(3, 48, dtype=u8)
    ids, spans, pooled = far(4, dtype=i64), far(3, dtype=i64), far(2, 1, 64, dtype=f32)
    eb, offs, room = far(1, dtype=f32), far(4, dtype=i64), far(64, dtype=u8)
    bag = dict(B=2, dim=64, indices=ids, offsets=spans, out=pooled)
    for call in (
        lambda: q.quantize_rowwise(x, 4, out=other(3, 48, dtype=u8)),
        lambda: q.quantize_baseline(x, 4, out=other(3, 48, dtype=u8)),
        lambda: q.dequantize(rows, 64, 4, out=other(3, 64, dtype=f32)),
        lambda: q.quantize_codebook(x, out=other(3, 48, dtype=u8)),
        lambda: q.dequantize_codebook(rows, 64, out=other(3, 64, dtype=f32)),
        lambda: q.bag_forward(rows, other(2, dtype=i64), bits=4, **bag),
        lambda: q.bag_forward(rows, far(2, dtype=i64), bits=4, **bag | dict(indices=other(4, dtype=i64))),
        lambda: q.bag_forward(rows, far(2, dtype=i64), bits=4, weights=other(4, dtype=f32), **bag),
        lambda: q.bag_forward(rows, far(2, dtype=i64), bits=4, err_count=other(1, dtype=torch.int32), **bag),
        lambda: q.bag_forward_codebook(rows, far(2, dtype=i64), **bag | dict(offsets=other(3, dtype=i64))),
        lambda: q.l2_error(x, other(3, 48, dtype=u8), 4),
        lambda: q.l2_error_codebook(x, other(3, 48, dtype=u8)),
        lambda: q.dot_interaction(far(3, 64, dtype=f32), other(3, 2, 64, dtype=f32), out=far(3, 64, dtype=f32)),
        lambda: q.compress_pooled(x, other(1, dtype=f32), T=1, out=room, offs=offs, workspace=room),
        lambda: q.compress_pooled_noalloc(x, eb, room, other(4, dtype=i64), T=1),
        lambda: q.decompress_pooled(room, offs, 64, eb, y=other(3, 64, dtype=f32)),
    ):
        with pytest.raises(ValueError):
            call()
    assert tables == []
