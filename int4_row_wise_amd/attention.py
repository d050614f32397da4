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
from typing import Optional, Tuple

import torch

from .qemb import INDEX_INT32, INDEX_INT64, QembError, _dev, _ptr, _stream

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqemb_attention.so")

MAX_HEAD_DIM = 256

EXPORTED = (
    "qemb_norm_rope", "qemb_prompt_attention", "qemb_decode_workspace_bytes",
    "qemb_decode_attention", "qemb_evict",
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
    L.qemb_prompt_attention.argtypes = [p, p, p, i64, i64, i32, i32, i32, i32, i32, i64, i64, i64, i64, i64, i64,
                                        p, p, i64, i32, i32, f32, p, p, p, p]
    L.qemb_prompt_attention.restype = ctypes.c_int
    L.qemb_decode_workspace_bytes.argtypes = [i32] * 9
    L.qemb_decode_workspace_bytes.restype = ctypes.c_size_t
    L.qemb_decode_attention.argtypes = [p, p, p, i64, i32, i32, i32, i32, i32, i32, i32, p, i32, p, i32, i32, f32,
                                        p, i64, p, p, p, p, p]
    L.qemb_decode_attention.restype = ctypes.c_int
    L.qemb_evict.argtypes = [p, p, i64, i32, i64, i32, i32, p, i32, p, p, i64, i32, i32, i32, p, p, i64, p, i32,
                             p, p, i64, p, p, p]
    L.qemb_evict.restype = ctypes.c_int
    _lib = L
    return L


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        raise QembError(fn, rc, _REASONS.get(rc, "unknown error"))


def _heads(name: str, t: torch.Tensor, dtype=None) -> None:
    """A [tokens, heads, dim] tensor whose last dimension is contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    if t.dim() != 3 or (t.stride(2) != 1 and t.shape[2] > 1):
        raise ValueError("%s must be [tokens, heads, dim] with dim contiguous" % name)
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError("%s must be %s, got %s" % (name, dtype or "bfloat16 or float16", t.dtype))


def _exact(name: str, t: Optional[torch.Tensor], shape: tuple, dtype) -> None:
    """An optional contiguous tensor of a given shape and type."""
    if t is None:
        return
    _dev(name, t, dtype)
    if tuple(t.shape) != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))


def _same_device(first: torch.Tensor, *others: Optional[torch.Tensor]) -> None:
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError("all tensors must be on %s, got one on %s" % (first.device, t.device))


def _cache(k_pages: torch.Tensor, v_pages: torch.Tensor, dim: int, bits: int, dtype) -> Tuple[int, int, int]:
    """(pages, kv heads, page size) of a cache of rows of `dim` elements."""
    if bits not in (16, 8, 4):
        raise ValueError("bits must be 16, 8 or 4")
    kind = dtype if bits == 16 else torch.uint8
    row = dim if bits == 16 else (dim * bits // 8 + 4 + 15) // 16 * 16
    _dev("k_pages", k_pages, kind)
    _dev("v_pages", v_pages, kind)
    if k_pages.dim() != 4 or k_pages.shape[3] != row or k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must both be [pages, kv_heads, page_size, %d]" % row)
    pages, heads, size, _ = k_pages.shape
    if size < 1 or size & (size - 1):
        raise ValueError("page_size must be a power of two, got %d" % size)
    return pages, heads, size


def norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
              q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, *,
              eps: float = 1e-6, interleaved: bool = False, v: Optional[torch.Tensor] = None,
              k_pages: Optional[torch.Tensor] = None, v_pages: Optional[torch.Tensor] = None,
              slots: Optional[torch.Tensor] = None, bits: int = 16, q_out: Optional[torch.Tensor] = None,
              k_out: Optional[torch.Tensor] = None,
              err_count: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Norm of each head of q [N, Hq, d] and k [N, Hkv, d] (any strides between
    tokens and heads), then rotation by cos_sin[positions] ([places, R] float32:
    R/2 cosines, R/2 sines).  With k_pages and v_pages, k's result and v are
    written to the flat `slots` [N] int64 (page * page_size + offset; negative:
    not written).  Returns (q_out, k_out); k_out is None with pages unless it is
    given."""
    _heads("q", q)
    _heads("k", k, q.dtype)
    n, hq, d = q.shape
    hkv = k.shape[1]
    if k.shape[0] != n or k.shape[2] != d:
        raise ValueError("q and k must have the same tokens and head dim")
    _exact("positions", positions, (n,), positions.dtype)
    if positions.dtype not in (torch.int32, torch.int64):
        raise TypeError("positions must be int32 or int64")
    _dev("cos_sin", cos_sin, torch.float32)
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [places, rot_dim]")
    _exact("q_weight", q_weight, (d,), q.dtype)
    _exact("k_weight", k_weight, (d,), q.dtype)
    pages = size = 0
    if (k_pages is None) != (v_pages is None) or (k_pages is None) != (slots is None) or (k_pages is None) != (v is None):
        raise ValueError("v, k_pages, v_pages and slots come together")
    if k_pages is not None:
        _heads("v", v, q.dtype)
        if v.shape != k.shape:
            raise ValueError("v must have k's shape")
        pages, heads, size = _cache(k_pages, v_pages, d, bits, q.dtype)
        if heads != hkv:
            raise ValueError("the cache has %d kv heads, k has %d" % (heads, hkv))
        _exact("slots", slots, (n,), torch.int64)
    elif k_out is None:
        k_out = torch.empty((n, hkv, d), dtype=q.dtype, device=q.device)
    if q_out is None:
        q_out = torch.empty((n, hq, d), dtype=q.dtype, device=q.device)
    _exact("q_out", q_out, (n, hq, d), q.dtype)
    _exact("k_out", k_out, (n, hkv, d), q.dtype)
    _exact("err_count", err_count, (1,), torch.int32)
    _same_device(q, k, v, positions, cos_sin, q_weight, k_weight, k_pages, v_pages, slots, q_out, k_out, err_count)
    vt, vh = (v.stride(0), v.stride(1)) if v is not None else (0, 0)
    _check("qemb_norm_rope", load_attention_library().qemb_norm_rope(
        q.data_ptr(), k.data_ptr(), _ptr(v), n, hq, hkv, d, _DTYPES[q.dtype], q.stride(0), q.stride(1), k.stride(0),
        k.stride(1), vt, vh, positions.data_ptr(), INDEX_INT64 if positions.dtype == torch.int64 else INDEX_INT32,
        cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1], int(interleaved), _ptr(q_weight), _ptr(k_weight), eps,
        q_out.data_ptr(), _ptr(k_out), _ptr(k_pages), _ptr(v_pages), _ptr(slots), pages, size, bits, _ptr(err_count),
        _stream(q)))
    return q_out, k_out


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor,
                     k_offsets: torch.Tensor, *, max_q: int = 0, window: int = 0, sinks: int = 0,
                     scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, err_count: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention of packed prompts: q [Nq, Hq, d], k and v [Nk, Hkv, d]
    (any strides between tokens and heads), sequence b in rows
    [offsets[b], offsets[b + 1]); its last query stands at its last key.  With a
    window, a query sees the last `window` keys up to its own and the first
    `sinks` keys.  max_q (the longest run of queries) only shapes the grid.
    scale: 1 / sqrt(d) unless given.  Returns out [Nq, Hq, d]; lse [Nq, Hq]
    float32 is filled if given."""
    _heads("q", q)
    _heads("k", k, q.dtype)
    _heads("v", v, q.dtype)
    n, hq, d = q.shape
    if k.shape != v.shape or k.shape[2] != d:
        raise ValueError("k and v must be [tokens, kv_heads, %d] alike" % d)
    batch = q_offsets.numel() - 1
    if batch < 0:
        raise ValueError("q_offsets must have batch + 1 entries")
    _exact("q_offsets", q_offsets, (batch + 1,), torch.int32)
    _exact("k_offsets", k_offsets, (batch + 1,), torch.int32)
    if out is None:
        out = torch.empty((n, hq, d), dtype=q.dtype, device=q.device)
    _exact("out", out, (n, hq, d), q.dtype)
    _exact("lse", lse, (n, hq), torch.float32)
    _exact("err_count", err_count, (1,), torch.int32)
    _same_device(q, k, v, q_offsets, k_offsets, out, lse, err_count)
    _check("qemb_prompt_attention", load_attention_library().qemb_prompt_attention(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), n, k.shape[0], batch, hq, k.shape[1], d, _DTYPES[q.dtype], q.stride(0),
        q.stride(1), k.stride(0), k.stride(1), v.stride(0), v.stride(1), q_offsets.data_ptr(), k_offsets.data_ptr(),
        max_q, window, sinks, d ** -0.5 if scale is None else scale, out.data_ptr(), _ptr(lse), _ptr(err_count),
        _stream(q)))
    return out


def decode_workspace_bytes(batch: int, q_heads: int, kv_heads: int, dim: int, width: int, page_size: int,
                           window: int = 0, sinks: int = 0, with_mass: bool = False) -> int:
    """Bytes of workspace that decode_attention needs for these sizes."""
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
    the query heads of its kv head.  Returns out [B, Hq, d]; lse [B, Hq] float32
    is filled if given."""
    _dev("q", q)
    if q.dim() != 3 or q.dtype not in _DTYPES:
        raise TypeError("q must be [batch, heads, dim] of bfloat16 or float16")
    b, hq, d = q.shape
    pages, hkv, size = _cache(k_pages, v_pages, d, bits, q.dtype)
    _dev("block_table", block_table, torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] != b:
        raise ValueError("block_table must be [%d, width]" % b)
    _exact("seq_lens", seq_lens, (b,), torch.int32)
    mass_len = 0
    if mass is not None:
        mass_len = mass.shape[-1]
        _exact("mass", mass, (b, hkv, mass_len), torch.float32)
    if out is None:
        out = torch.empty((b, hq, d), dtype=q.dtype, device=q.device)
    _exact("out", out, (b, hq, d), q.dtype)
    _exact("lse", lse, (b, hq), torch.float32)
    _exact("err_count", err_count, (1,), torch.int32)
    L = load_attention_library()
    width = block_table.shape[1]
    need = int(L.qemb_decode_workspace_bytes(b, hq, hkv, d, width, size, window, sinks, mass is not None))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    else:
        _dev("workspace", workspace, torch.uint8)
        if workspace.numel() < need:
            raise ValueError("workspace must have at least %d bytes" % need)
    _same_device(q, k_pages, v_pages, block_table, seq_lens, mass, out, lse, workspace, err_count)
    _check("qemb_decode_attention", L.qemb_decode_attention(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), pages, size, bits, b, hq, hkv, d, _DTYPES[q.dtype],
        block_table.data_ptr(), width, seq_lens.data_ptr(), window, sinks, d ** -0.5 if scale is None else scale,
        _ptr(mass), mass_len, out.data_ptr(), _ptr(lse), _ptr(workspace), _ptr(err_count), _stream(q)))
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
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages), ("new_k_pages", new_k_pages), ("new_v_pages", new_v_pages)):
        _dev(name, t, k_pages.dtype)
        if t.dim() != 4 or t.shape[1:] != k_pages.shape[1:]:
            raise ValueError("%s must be [pages, kv_heads, page_size, row] like k_pages" % name)
    if v_pages.shape != k_pages.shape or new_v_pages.shape != new_k_pages.shape:
        raise ValueError("key and value pages must have the same shape")
    pages, hkv, size, row = k_pages.shape
    if size < 1 or size & (size - 1):
        raise ValueError("page_size must be a power of two, got %d" % size)
    _dev("seq_lens", seq_lens, torch.int32)
    b = seq_lens.numel()
    _dev("block_table", block_table, torch.int32)
    _dev("new_block_table", new_block_table, torch.int32)
    if block_table.dim() != 2 or new_block_table.dim() != 2 or block_table.shape[0] != b or new_block_table.shape[0] != b:
        raise ValueError("block tables must be [%d, width]" % b)
    _dev("mass", mass, torch.float32)
    if mass.dim() != 3 or mass.shape[0] != b or mass.shape[1] != hkv:
        raise ValueError("mass must be [%d, %d, slots]" % (b, hkv))
    if keep < 1 or sinks < 0 or recent < 0 or sinks + recent > keep or new_block_table.shape[1] * size < keep:
        raise ValueError("keep must be at least 1 and sinks + recent, and fit the new pages")
    if kept is None:
        kept = torch.empty((b, hkv, keep), dtype=torch.int32, device=mass.device)
    if new_mass is None:
        new_mass = torch.empty((b, hkv, keep), dtype=torch.float32, device=mass.device)
    if new_lens is None:
        new_lens = torch.empty(b, dtype=torch.int32, device=mass.device)
    _exact("kept", kept, (b, hkv, keep), torch.int32)
    if new_mass.dim() != 3 or new_mass.shape[2] < keep:
        raise ValueError("new_mass must be [%d, %d, >= %d]" % (b, hkv, keep))
    _exact("new_mass", new_mass, (b, hkv, new_mass.shape[2]), torch.float32)
    _exact("new_lens", new_lens, (b,), torch.int32)
    _exact("err_count", err_count, (1,), torch.int32)
    _same_device(k_pages, v_pages, block_table, seq_lens, mass, new_k_pages, new_v_pages, new_block_table, kept,
                 new_mass, new_lens, err_count)
    _check("qemb_evict", load_attention_library().qemb_evict(
        k_pages.data_ptr(), v_pages.data_ptr(), pages, size, row * k_pages.element_size(), b, hkv,
        block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(), mass.data_ptr(), mass.shape[2], keep, sinks,
        recent, new_k_pages.data_ptr(), new_v_pages.data_ptr(), new_k_pages.shape[0], new_block_table.data_ptr(),
        new_block_table.shape[1], kept.data_ptr(), new_mass.data_ptr(), new_mass.shape[2], new_lens.data_ptr(),
        _ptr(err_count), _stream(k_pages)))
    return kept, new_mass, new_lens
