"""Thin ctypes binding over libqemb_attention.so (include/qemb_attention.h):
attention over a paged key-value cache.

The cache is two tensors of pages, ``[pages, kv_heads, page_size, row]``: rows
of 16-bit values (``bits=16``, the queries' dtype, row = head dim) or packed
INT8 / INT4 rows (uint8, row = ``row_stride(dim, bits)``), the rows that
``quantize_rowwise`` writes.  ``block_table[b, i]`` is the page of slots
``[i * page_size, (i + 1) * page_size)`` of sequence b.

Argument marshalling only: the kernels run behind the C ABI, on the current
stream, and nothing synchronizes.  Outputs and workspaces are torch tensors,
allocated here unless given.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple

import torch

from .qemb import INDEX_INT32, INDEX_INT64, QembError, _launch, _ptr, _raw_stream

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqemb_attention.so")

MAX_HEAD_DIM = 256
MAX_AXES = 4

EXPORTED = (
    "qemb_norm_rope", "qemb_norm_rope_axes", "qemb_prompt_attention", "qemb_decode_workspace_bytes",
    "qemb_decode_attention", "qemb_shared_workspace_bytes", "qemb_shared_attention", "qemb_evict",
)

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_REASONS = {-1: "invalid argument", -2: "array not aligned", -3: "unsupported size", -4: "kernel launch failed"}

_lib = None


def load_attention_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """The loaded library; raises if it is not built, or from other sources."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise QembError("load_attention_library", -100,
                        "%s is not built (run `python -m int4_row_wise_amd.build`)" % path)
    from . import build as qbuild
    if qbuild.recorded_hash(path) != qbuild.attention_source_sha256():
        raise QembError("load_attention_library", -101,
                        "%s was built from other kernel sources; rebuild with "
                        "`python -m int4_row_wise_amd.build`" % path)
    L = ctypes.CDLL(path)
    p, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    L.qemb_norm_rope.argtypes = [p, p, p, i64, i32, i32, i32, i32, i64, i64, i64, i64, i64, i64, p, i32, p, i64,
                                 i32, i32, p, p, f32, p, p, p, p, p, i64, i32, i32, p, p]
    L.qemb_norm_rope.restype = ctypes.c_int
    L.qemb_norm_rope_axes.argtypes = [p, p, p, i64, i32, i32, i32, i32, i64, i64, i64, i64, i64, i64, p, i32, p, i32, p,
                                      i64, i32, i32, i32, p, p, f32, p, p, p, p, p, i64, i32, i32, p, p]
    L.qemb_norm_rope_axes.restype = ctypes.c_int
    L.qemb_prompt_attention.argtypes = [p, p, p, i64, i64, i32, i32, i32, i32, i32, i64, i64, i64, i64, i64, i64,
                                        p, p, i64, i32, i32, f32, p, p, p, p]
    L.qemb_prompt_attention.restype = ctypes.c_int
    L.qemb_decode_workspace_bytes.argtypes = [i32] * 9
    L.qemb_decode_workspace_bytes.restype = ctypes.c_size_t
    L.qemb_decode_attention.argtypes = [p, p, p, i64, i32, i32, i32, i32, i32, i32, i32, p, i32, p, i32, i32, f32,
                                        p, i64, p, p, p, p, p]
    L.qemb_decode_attention.restype = ctypes.c_int
    L.qemb_shared_workspace_bytes.argtypes = [i32] * 9
    L.qemb_shared_workspace_bytes.restype = ctypes.c_size_t
    L.qemb_shared_attention.argtypes = [p, p, p, i64, i32, i32, i32, i32, i32, i32, i32, p, i32, p, p, i32, p, i32, p,
                                        f32, p, p, p, p, p]
    L.qemb_shared_attention.restype = ctypes.c_int
    L.qemb_evict.argtypes = [p, p, i64, i32, i64, i32, i32, p, i32, p, p, i64, i32, i32, i32, p, p, i64, p, i32,
                             p, p, i64, p, p, p]
    L.qemb_evict.restype = ctypes.c_int
    _lib = L
    return L


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        raise QembError(fn, rc, _REASONS.get(rc, "unknown error"))


def _device(name: str, t: torch.Tensor) -> int:
    """The GPU index of the tensor that decides where a call runs."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    return t.get_device()


def _int32(name: str, value: int) -> None:
    """Refuses a number that the C ABI's 32 bits would cut."""
    if not -1 << 31 <= value < 1 << 31:
        raise ValueError("%s must fit 32 bits, got %d" % (name, value))


def _want(name: str, t: torch.Tensor, shape: tuple, dtype, dev: int) -> None:
    """A contiguous tensor of a given shape and type on a given GPU."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if t.get_device() != dev:
        raise ValueError("%s must be on cuda:%d, got %s" % (name, dev, t.device))
    raise ValueError("%s must be contiguous" % name)


def _heads(name: str, t: torch.Tensor, dtype, dev: int) -> tuple:
    """A [tokens, heads, dim] tensor whose last dimension is contiguous: its strides."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise TypeError("%s must be a CUDA (HIP) tensor on cuda:%d" % (name, dev))
    if t.dtype is not dtype or dtype not in _DTYPES:
        raise TypeError("%s must be %s, got %s" % (name, dtype if dtype in _DTYPES else "bfloat16 or float16", t.dtype))
    stride = t.stride()
    if len(stride) != 3 or (stride[2] != 1 and t.shape[2] > 1):
        raise ValueError("%s must be [tokens, heads, dim] with dim contiguous" % name)
    return stride


def _cache(k_pages: torch.Tensor, v_pages: torch.Tensor, dim: int, bits: int, dtype, dev: int) -> tuple:
    """(pages, kv heads, page size) of a cache of rows of `dim` elements."""
    if bits == 16:
        row = dim
    elif bits == 8 or bits == 4:
        row, dtype = (dim * bits // 8 + 4 + 15) // 16 * 16, torch.uint8
    else:
        raise ValueError("bits must be 16, 8 or 4")
    if not isinstance(k_pages, torch.Tensor) or not k_pages.is_cuda:
        raise TypeError("k_pages must be a CUDA (HIP) tensor")
    shape = k_pages.shape
    if len(shape) != 4 or shape[3] != row:
        raise ValueError("k_pages must be [pages, kv_heads, page_size, %d], got %s" % (row, list(shape)))
    size = shape[2]
    if size < 1 or size & (size - 1):
        raise ValueError("page_size must be a power of two, got %d" % size)
    _want("k_pages", k_pages, shape, dtype, dev)
    _want("v_pages", v_pages, shape, dtype, dev)
    return shape[0], shape[1], size


def norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
              q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, *,
              eps: float = 1e-6, interleaved: bool = False, v: Optional[torch.Tensor] = None,
              k_pages: Optional[torch.Tensor] = None, v_pages: Optional[torch.Tensor] = None,
              slots: Optional[torch.Tensor] = None, bits: int = 16, q_out: Optional[torch.Tensor] = None,
              k_out: Optional[torch.Tensor] = None, err_count: Optional[torch.Tensor] = None,
              pair_axes: Optional[torch.Tensor] = None, norm: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Norm of each head of q [N, Hq, d] and k [N, Hkv, d] (any strides between
    tokens and heads), then rotation by cos_sin[positions] ([places, R] float32:
    R/2 cosines, R/2 sines).  With k_pages and v_pages, k's result and v are
    written to the flat `slots` [N] int64 (page * page_size + offset; negative:
    not written).  Returns (q_out, k_out); k_out is None with pages unless it is
    given.

    With pair_axes [R/2] uint8 (see rotary_axes), positions is [axes, N] (at most
    4 axes) and pair i turns by the position on axis pair_axes[i]; a pair whose
    number is no axis is not turned.  norm=False leaves the norm out (and takes no
    weights)."""
    dev, dtype = _device("q", q), q.dtype
    qs, ks, vs = _heads("q", q, dtype, dev), _heads("k", k, dtype, dev), (0, 0)
    n, hq, d = q.shape
    hkv = k.shape[1]
    if k.shape[0] != n or k.shape[2] != d:
        raise ValueError("q and k must have the same tokens and head dim")
    wide = isinstance(positions, torch.Tensor) and positions.dtype is torch.int64
    axes = 1
    if pair_axes is None:
        _want("positions", positions, (n,), torch.int64 if wide else torch.int32, dev)
    else:
        if not isinstance(positions, torch.Tensor) or positions.dim() != 2 or not 1 <= positions.shape[0] <= MAX_AXES:
            raise ValueError("positions must be [axes, %d] with at most %d axes" % (n, MAX_AXES))
        axes = positions.shape[0]
        _want("positions", positions, (axes, n), torch.int64 if wide else torch.int32, dev)
    if not norm and (q_weight is not None or k_weight is not None):
        raise ValueError("weights belong to the norm")
    if not isinstance(cos_sin, torch.Tensor) or cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [places, rot_dim]")
    places, rot = cos_sin.shape
    _want("cos_sin", cos_sin, (places, rot), torch.float32, dev)
    if pair_axes is not None:
        _want("pair_axes", pair_axes, (rot // 2,), torch.uint8, dev)
    if q_weight is not None:
        _want("q_weight", q_weight, (d,), dtype, dev)
    if k_weight is not None:
        _want("k_weight", k_weight, (d,), dtype, dev)
    pages = size = 0
    if k_pages is not None:
        if v_pages is None or slots is None or v is None:
            raise ValueError("v, k_pages, v_pages and slots come together")
        vs = _heads("v", v, dtype, dev)
        if v.shape != k.shape:
            raise ValueError("v must have k's shape")
        pages, heads, size = _cache(k_pages, v_pages, d, bits, dtype, dev)
        if heads != hkv:
            raise ValueError("the cache has %d kv heads, k has %d" % (heads, hkv))
        _want("slots", slots, (n,), torch.int64, dev)
    elif v_pages is not None or slots is not None or v is not None:
        raise ValueError("v, k_pages, v_pages and slots come together")
    elif k_out is None:
        k_out = torch.empty((n, hkv, d), dtype=dtype, device=q.device)
    if q_out is None:
        q_out = torch.empty((n, hq, d), dtype=dtype, device=q.device)
    else:
        _want("q_out", q_out, (n, hq, d), dtype, dev)
    if k_out is not None:
        _want("k_out", k_out, (n, hkv, d), dtype, dev)
    if err_count is not None:
        _want("err_count", err_count, (1,), torch.int32, dev)
    index = INDEX_INT64 if wide else INDEX_INT32
    if pair_axes is None and norm:
        _check("qemb_norm_rope", _launch(
            dev, load_attention_library().qemb_norm_rope,
            q.data_ptr(), k.data_ptr(), _ptr(v), n, hq, hkv, d, _DTYPES[dtype], qs[0], qs[1], ks[0], ks[1], vs[0], vs[1],
            positions.data_ptr(), index, cos_sin.data_ptr(), places, rot, int(interleaved),
            _ptr(q_weight), _ptr(k_weight), eps, q_out.data_ptr(), _ptr(k_out), _ptr(k_pages), _ptr(v_pages), _ptr(slots),
            pages, size, bits, _ptr(err_count), _raw_stream(dev)))
    else:
        _check("qemb_norm_rope_axes", _launch(
            dev, load_attention_library().qemb_norm_rope_axes,
            q.data_ptr(), k.data_ptr(), _ptr(v), n, hq, hkv, d, _DTYPES[dtype], qs[0], qs[1], ks[0], ks[1], vs[0], vs[1],
            positions.data_ptr(), axes, _ptr(pair_axes), index, cos_sin.data_ptr(), places, rot, int(interleaved), int(norm),
            _ptr(q_weight), _ptr(k_weight), eps, q_out.data_ptr(), _ptr(k_out), _ptr(k_pages), _ptr(v_pages), _ptr(slots),
            pages, size, bits, _ptr(err_count), _raw_stream(dev)))
    return q_out, k_out


def rotary_axes(sections: Sequence[int], *, in_turn: bool = False, device="cuda") -> torch.Tensor:
    """The axis of each pair, for norm_rope's pair_axes: sections[a] pairs turn by
    axis a, one axis after the other, or (in_turn) in turn as long as an axis has
    pairs left: sections (3, 2, 2) give 0 0 0 1 1 2 2, or 0 1 2 0 1 2 0."""
    if not 1 <= len(sections) <= MAX_AXES or any(n < 0 for n in sections):
        raise ValueError("sections must be the pairs of 1 .. %d axes" % MAX_AXES)
    pairs = [(i, a) if in_turn else (a, i) for a, n in enumerate(sections) for i in range(n)]
    pairs.sort()
    return torch.tensor([p[1] if in_turn else p[0] for p in pairs], dtype=torch.uint8, device=device)


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor,
                     k_offsets: torch.Tensor, *, max_q: int = 0, window: int = 0, sinks: int = 0,
                     scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, err_count: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention of packed prompts: q [Nq, Hq, d], k and v [Nk, Hkv, d]
    (any strides between tokens and heads), sequence b in rows
    [offsets[b], offsets[b + 1]); its last query stands at its last key.  With a
    window, a query sees the last `window` keys up to its own and the first
    `sinks` keys.  max_q (the longest run of queries) only shapes the grid; left
    at 0, every sequence gets workgroups for all queries.
    scale: 1 / sqrt(d) unless given.  Returns out [Nq, Hq, d]; lse [Nq, Hq]
    float32 is filled if given."""
    dev, dtype = _device("q", q), q.dtype
    qs, ks, vs = _heads("q", q, dtype, dev), _heads("k", k, dtype, dev), _heads("v", v, dtype, dev)
    n, hq, d = q.shape
    if k.shape != v.shape or k.shape[2] != d:
        raise ValueError("k and v must be [tokens, kv_heads, %d] alike" % d)
    _int32("window", window)
    _int32("sinks", sinks)
    if not isinstance(q_offsets, torch.Tensor) or q_offsets.numel() < 1:
        raise ValueError("q_offsets must have batch + 1 entries")
    batch = q_offsets.numel() - 1
    _want("q_offsets", q_offsets, (batch + 1,), torch.int32, dev)
    _want("k_offsets", k_offsets, (batch + 1,), torch.int32, dev)
    if out is None:
        out = torch.empty((n, hq, d), dtype=dtype, device=q.device)
    else:
        _want("out", out, (n, hq, d), dtype, dev)
    if lse is not None:
        _want("lse", lse, (n, hq), torch.float32, dev)
    if err_count is not None:
        _want("err_count", err_count, (1,), torch.int32, dev)
    _check("qemb_prompt_attention", _launch(
        dev, load_attention_library().qemb_prompt_attention,
        q.data_ptr(), k.data_ptr(), v.data_ptr(), n, k.shape[0], batch, hq, k.shape[1], d, _DTYPES[dtype], qs[0], qs[1],
        ks[0], ks[1], vs[0], vs[1], q_offsets.data_ptr(), k_offsets.data_ptr(), max_q, window, sinks,
        d ** -0.5 if scale is None else scale, out.data_ptr(), _ptr(lse), _ptr(err_count), _raw_stream(dev)))
    return out


def decode_workspace_bytes(batch: int, q_heads: int, kv_heads: int, dim: int, width: int, page_size: int,
                           window: int = 0, sinks: int = 0, with_mass: bool = False) -> int:
    """Bytes of workspace that decode_attention needs for these sizes."""
    for name, value in (("batch", batch), ("q_heads", q_heads), ("kv_heads", kv_heads), ("dim", dim), ("width", width),
                        ("page_size", page_size), ("window", window), ("sinks", sinks)):
        _int32(name, value)
    return int(load_attention_library().qemb_decode_workspace_bytes(
        batch, q_heads, kv_heads, dim, width, page_size, window, sinks, int(with_mass)))


def decode_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                     seq_lens: torch.Tensor, *, bits: int = 16, window: int = 0, sinks: int = 0,
                     scale: Optional[float] = None, mass: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     err_count: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of one new token for each sequence, q [B, Hq, d], over the
    seq_lens[b] rows of its pages block_table[b] (int32; the token's own row is
    the last).  window and sinks as in prompt_attention.  mass [B, Hkv, M]
    float32 (M >= every length) grows by each key's softmax weight, summed over
    the query heads of its kv head.  The table's width (not the lengths) sets how
    the work is split and the workspace, so it is best kept near the longest
    sequence.  Returns out [B, Hq, d]; lse [B, Hq] float32
    is filled if given."""
    dev, dtype = _device("q", q), q.dtype
    if q.dim() != 3 or dtype not in _DTYPES or not q.is_contiguous():
        raise TypeError("q must be [batch, heads, dim] of bfloat16 or float16, contiguous")
    _int32("window", window)
    _int32("sinks", sinks)
    b, hq, d = q.shape
    pages, hkv, size = _cache(k_pages, v_pages, d, bits, dtype, dev)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [%d, width]" % b)
    width = block_table.shape[1]
    _want("block_table", block_table, (b, width), torch.int32, dev)
    _want("seq_lens", seq_lens, (b,), torch.int32, dev)
    mass_len = 0
    if mass is not None:
        mass_len = mass.shape[-1]
        _want("mass", mass, (b, hkv, mass_len), torch.float32, dev)
    if out is None:
        out = torch.empty((b, hq, d), dtype=dtype, device=q.device)
    else:
        _want("out", out, (b, hq, d), dtype, dev)
    if lse is not None:
        _want("lse", lse, (b, hq), torch.float32, dev)
    if err_count is not None:
        _want("err_count", err_count, (1,), torch.int32, dev)
    L = load_attention_library()
    need = L.qemb_decode_workspace_bytes(b, hq, hkv, d, width, size, window, sinks, mass is not None)
    if workspace is not None:
        if workspace.numel() < need:
            raise ValueError("workspace must have at least %d bytes" % need)
        _want("workspace", workspace, workspace.shape, torch.uint8, dev)
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check("qemb_decode_attention", _launch(
        dev, L.qemb_decode_attention,
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), pages, size, bits, b, hq, hkv, d, _DTYPES[dtype],
        block_table.data_ptr(), width, seq_lens.data_ptr(), window, sinks, d ** -0.5 if scale is None else scale,
        _ptr(mass), mass_len, out.data_ptr(), _ptr(lse), _ptr(workspace), _ptr(err_count), _raw_stream(dev)))
    return out


def shared_workspace_bytes(batch: int, q_heads: int, kv_heads: int, dim: int, groups: int, prefix_width: int, width: int,
                           page_size: int, bits: int = 16) -> int:
    """Bytes of workspace that shared_attention needs for these sizes."""
    for name, value in (("batch", batch), ("q_heads", q_heads), ("kv_heads", kv_heads), ("dim", dim), ("groups", groups),
                        ("prefix_width", prefix_width), ("width", width), ("page_size", page_size),
                        ("bits", bits)):
        _int32(name, value)
    return int(load_attention_library().qemb_shared_workspace_bytes(
        batch, q_heads, kv_heads, dim, groups, prefix_width, width, page_size, bits))


def shared_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, prefix_table: torch.Tensor,
                     prefix_lens: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, *,
                     group_offsets: Optional[torch.Tensor] = None, bits: int = 16, scale: Optional[float] = None,
                     out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     err_count: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of one new token for each sequence, q [B, Hq, d], where groups of
    sequences share a prefix: sequences group_offsets[g] .. group_offsets[g + 1] - 1
    (int32 [G + 1]; None: one group of all) see the prefix_lens[g] rows of the pages
    prefix_table[g] (int32 [G, P]), read once for the group, and then the seq_lens[b]
    rows of their own pages block_table[b] (int32 [B, W]; the token's own row is the
    last; 0 rows are fine).  The tables' widths (not the lengths) set how the work is
    split and the workspace, so they are best kept near the longest.  Returns out
    [B, Hq, d]; lse [B, Hq] float32 is filled if given."""
    dev, dtype = _device("q", q), q.dtype
    if q.dim() != 3 or dtype not in _DTYPES or not q.is_contiguous():
        raise TypeError("q must be [batch, heads, dim] of bfloat16 or float16, contiguous")
    b, hq, d = q.shape
    pages, hkv, size = _cache(k_pages, v_pages, d, bits, dtype, dev)
    if not isinstance(prefix_table, torch.Tensor) or prefix_table.dim() != 2 or prefix_table.shape[0] < 1:
        raise ValueError("prefix_table must be [groups, width]")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be [%d, width]" % b)
    groups, prefix_width = prefix_table.shape
    width = block_table.shape[1]
    _want("prefix_table", prefix_table, (groups, prefix_width), torch.int32, dev)
    _want("prefix_lens", prefix_lens, (groups,), torch.int32, dev)
    _want("block_table", block_table, (b, width), torch.int32, dev)
    _want("seq_lens", seq_lens, (b,), torch.int32, dev)
    if group_offsets is not None:
        _want("group_offsets", group_offsets, (groups + 1,), torch.int32, dev)
    elif groups != 1:
        raise ValueError("%d prefixes need group_offsets" % groups)
    if out is None:
        out = q.new_empty((b, hq, d))
    else:
        _want("out", out, (b, hq, d), dtype, dev)
    if lse is not None:
        _want("lse", lse, (b, hq), torch.float32, dev)
    if err_count is not None:
        _want("err_count", err_count, (1,), torch.int32, dev)
    L = load_attention_library()
    need = L.qemb_shared_workspace_bytes(b, hq, hkv, d, groups, prefix_width, width, size, bits)
    if workspace is not None:
        if workspace.numel() < need:
            raise ValueError("workspace must have at least %d bytes" % need)
        _want("workspace", workspace, workspace.shape, torch.uint8, dev)
    elif need:
        workspace = q.new_empty(need, dtype=torch.uint8)
    _check("qemb_shared_attention", _launch(
        dev, L.qemb_shared_attention,
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), pages, size, bits, b, hq, hkv, d, _DTYPES[dtype],
        prefix_table.data_ptr(), prefix_width, prefix_lens.data_ptr(), _ptr(group_offsets), groups,
        block_table.data_ptr(), width, seq_lens.data_ptr(), d ** -0.5 if scale is None else scale, out.data_ptr(),
        _ptr(lse), _ptr(workspace), _ptr(err_count), _raw_stream(dev)))
    return out


def evict(k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
          mass: torch.Tensor, keep: int, new_k_pages: torch.Tensor, new_v_pages: torch.Tensor,
          new_block_table: torch.Tensor, *, sinks: int = 0, recent: int = 0, kept: Optional[torch.Tensor] = None,
          new_mass: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
          err_count: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Cuts every (sequence, kv head) to at most `keep` slots: the first `sinks`,
    the last `recent` and the largest mass [B, Hkv, M] between (ties to the lower
    slot), copied in slot order to the pages of new_block_table (pages of
    new_k_pages / new_v_pages that overlap none of the old ones; the arrays may
    be the same).  Returns (kept [B, Hkv, keep] int32 with -1 past the end,
    new_mass [B, Hkv, >= keep], new_lens [B])."""
    dev = _device("k_pages", k_pages)
    if k_pages.dim() != 4:
        raise ValueError("k_pages must be [pages, kv_heads, page_size, row]")
    kind = k_pages.dtype
    pages, hkv, size, row = k_pages.shape
    if size < 1 or size & (size - 1):
        raise ValueError("page_size must be a power of two, got %d" % size)
    _want("k_pages", k_pages, k_pages.shape, kind, dev)
    _want("v_pages", v_pages, k_pages.shape, kind, dev)
    if not isinstance(new_k_pages, torch.Tensor) or new_k_pages.dim() != 4:
        raise ValueError("new_k_pages must be [pages, kv_heads, page_size, row] like k_pages")
    new_pages = new_k_pages.shape[0]
    _want("new_k_pages", new_k_pages, (new_pages, hkv, size, row), kind, dev)
    _want("new_v_pages", new_v_pages, (new_pages, hkv, size, row), kind, dev)
    b = seq_lens.numel()
    _want("seq_lens", seq_lens, (b,), torch.int32, dev)
    if block_table.dim() != 2 or new_block_table.dim() != 2 or mass.dim() != 3:
        raise ValueError("block tables must be [%d, width], mass [%d, %d, slots]" % (b, b, hkv))
    width, new_width, mass_len = block_table.shape[1], new_block_table.shape[1], mass.shape[2]
    _want("block_table", block_table, (b, width), torch.int32, dev)
    _want("new_block_table", new_block_table, (b, new_width), torch.int32, dev)
    _want("mass", mass, (b, hkv, mass_len), torch.float32, dev)
    _int32("keep", keep)
    if keep < 1 or sinks < 0 or recent < 0 or sinks + recent > keep or new_width * size < keep:
        raise ValueError("keep must be at least 1 and sinks + recent, and fit the new pages")
    if kept is None:
        kept = torch.empty((b, hkv, keep), dtype=torch.int32, device=mass.device)
    else:
        _want("kept", kept, (b, hkv, keep), torch.int32, dev)
    if new_mass is None:
        new_mass = torch.empty((b, hkv, keep), dtype=torch.float32, device=mass.device)
    else:
        if new_mass.dim() != 3 or new_mass.shape[2] < keep:
            raise ValueError("new_mass must be [%d, %d, >= %d]" % (b, hkv, keep))
        _want("new_mass", new_mass, (b, hkv, new_mass.shape[2]), torch.float32, dev)
    if new_lens is None:
        new_lens = torch.empty(b, dtype=torch.int32, device=mass.device)
    else:
        _want("new_lens", new_lens, (b,), torch.int32, dev)
    if err_count is not None:
        _want("err_count", err_count, (1,), torch.int32, dev)
    _check("qemb_evict", _launch(
        dev, load_attention_library().qemb_evict,
        k_pages.data_ptr(), v_pages.data_ptr(), pages, size, row * k_pages.element_size(), b, hkv,
        block_table.data_ptr(), width, seq_lens.data_ptr(), mass.data_ptr(), mass_len, keep, sinks,
        recent, new_k_pages.data_ptr(), new_v_pages.data_ptr(), new_pages, new_block_table.data_ptr(),
        new_width, kept.data_ptr(), new_mass.data_ptr(), new_mass.shape[2], new_lens.data_ptr(),
        _ptr(err_count), _raw_stream(dev)))
    return kept, new_mass, new_lens
