"""Thin ctypes binding over libqemb_serving.so (include/qemb_serving.h): what
stands around the attention in a serving loop, the residual's addition with a
norm and the log probabilities of tokens.

Argument marshalling only: the kernels run behind the C ABI, on the current
stream of the tensors' GPU, and nothing synchronizes.  Outputs and workspaces are
torch tensors, allocated here where none can be or is given (token_logprobs takes
lse and a workspace; its other outputs are new ones).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

from .attention import _check, _device, _want
from .qemb import INDEX_INT32, INDEX_INT64, QembError, _launch, _ptr, _raw_stream

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqemb_serving.so")

MAX_NORM_DIM = 32768
MAX_TOP = 64

EXPORTED = ("qemb_add_norm", "qemb_logprobs_workspace_bytes", "qemb_token_logprobs")

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_FORMS = {"values": (0, None), "int8": (1, torch.int8), "fp8": (2, torch.float8_e4m3fn), "rows8": (3, torch.uint8)}

_lib = None


def load_serving_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """The loaded library; raises if it is not built, or from other sources."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise QembError("load_serving_library", -100,
                        "%s is not built (run `python -m int4_row_wise_amd.build`)" % path)
    from . import build as qbuild
    if qbuild.recorded_hash(path) != qbuild.serving_source_sha256():
        raise QembError("load_serving_library", -101,
                        "%s was built from other kernel sources; rebuild with "
                        "`python -m int4_row_wise_amd.build`" % path)
    L = ctypes.CDLL(path)
    p, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    L.qemb_add_norm.argtypes = [p, p, p, i64, i32, i32, i64, i64, i64, f32, i32, i32, p, p, p, p]
    L.qemb_add_norm.restype = ctypes.c_int
    L.qemb_logprobs_workspace_bytes.argtypes = [i64, i64, i32, i32]
    L.qemb_logprobs_workspace_bytes.restype = ctypes.c_size_t
    L.qemb_token_logprobs.argtypes = [p, i64, i64, i32, i64, p, i32, i32, p, p, p, p, p, p, p, p]
    L.qemb_token_logprobs.restype = ctypes.c_int
    _lib = L
    return L


def _rows(name: str, t: torch.Tensor, shape: tuple, dtype, dev: int) -> int:
    """A [rows, dim] tensor whose last dimension is contiguous: the stride between its rows."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != dev:
        raise TypeError("%s must be a CUDA (HIP) tensor on cuda:%d" % (name, dev))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    stride = t.stride()
    if stride[1] != 1 and shape[1] > 1:
        raise ValueError("%s must have contiguous rows" % name)
    return stride[0]


def add_norm(x: torch.Tensor, residual: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None, *,
             eps: float = 1e-6, form: str = "values", group: int = 0, out: Optional[torch.Tensor] = None,
             scales: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
             ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """h = x + residual (both [N, d], any stride between rows) and its root-mean-square
    norm times `weight` [d], from the unrounded sum.  form: "values" (x's dtype),
    "int8" or "fp8" (e4m3) codes with float32 scales a row (group=0) or a group of
    32 .. 512 elements, or "rows8" (the packed INT8 rows of quantize_rowwise, d at
    most 1024).  sum_out takes h rounded to x's dtype; it may be x or residual
    itself, and is allocated if there is a residual and none is given.  Returns
    (out, sum_out, scales); what a form or call does not have is None."""
    dev, dtype = _device("x", x), x.dtype
    if x.dim() != 2 or (dtype is not torch.bfloat16 and dtype is not torch.float16):
        raise TypeError("x must be [rows, dim] of bfloat16 or float16")
    shape = x.shape
    n, d = shape
    xs = _rows("x", x, shape, dtype, dev)
    rs = _rows("residual", residual, shape, dtype, dev) if residual is not None else 0
    if weight is not None:
        _want("weight", weight, (d,), dtype, dev)
    if form not in _FORMS:
        raise ValueError("form must be one of %s" % ", ".join(_FORMS))
    code, kind = _FORMS[form]
    if form == "rows8":
        want = (n, (d + 4 + 15) // 16 * 16)
    else:
        want, kind = (n, d), kind or dtype
    if out is None:
        out = x.new_empty(want, dtype=kind)
    else:
        _want("out", out, want, kind, dev)
    if code == 1 or code == 2:
        if group and (group < 0 or d % group):
            raise ValueError("group must divide the rows' %d elements, got %d" % (d, group))
        of_scales = (n, d // group) if group else (n,)
        if scales is None:
            scales = x.new_empty(of_scales, dtype=torch.float32)
        else:
            _want("scales", scales, of_scales, torch.float32, dev)
    elif scales is not None or group:
        raise ValueError("form %r has no scales" % form)
    if sum_out is not None:
        ss = _rows("sum_out", sum_out, shape, dtype, dev)
    elif residual is not None:
        sum_out, ss = x.new_empty(shape), d
    else:
        ss = 0
    _check("qemb_add_norm", _launch(
        dev, load_serving_library().qemb_add_norm,
        x.data_ptr(), _ptr(residual), _ptr(weight), n, d, _DTYPES[dtype], xs, rs, ss, eps, code, group, out.data_ptr(),
        _ptr(scales), _ptr(sum_out), _raw_stream(dev)))
    return out, sum_out, scales


def logprobs_workspace_bytes(rows: int, vocab: int, dtype: torch.dtype, top: int = 0) -> int:
    """Bytes of workspace that token_logprobs needs for these sizes."""
    if dtype not in _DTYPES:
        raise TypeError("dtype must be bfloat16, float16 or float32")
    return int(load_serving_library().qemb_logprobs_workspace_bytes(rows, vocab, _DTYPES[dtype], top))


def token_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, *, top: int = 0,
                   lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   err_count: Optional[torch.Tensor] = None,
                   ) -> Tuple[Optional[torch.Tensor], torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Of each row of logits [N, V] (16 or 32 bits, any stride between rows): the log
    probability of targets[n] (int32 or int64; 0 where it is not a token, e.g. -1),
    the entropy, and the `top` (at most 64) most likely tokens, the likeliest first
    and the lowest id of equals, with their log probabilities.  Returns (logprobs
    [N], entropy [N], top_ids [N, top] int32, top_logprobs [N, top]); what is not
    asked for is None.  lse [N] float32 is filled if given."""
    dev, dtype = _device("logits", logits), logits.dtype
    if logits.dim() != 2 or dtype not in _DTYPES:
        raise TypeError("logits must be [rows, vocab] of bfloat16, float16 or float32")
    n, v = logits.shape
    stride = _rows("logits", logits, logits.shape, dtype, dev)
    if not 0 <= top <= MAX_TOP:
        raise ValueError("top must be 0 .. %d, got %d" % (MAX_TOP, top))
    logprobs = ids = tops = None
    wide = False
    if targets is not None:
        wide = isinstance(targets, torch.Tensor) and targets.dtype is torch.int64
        _want("targets", targets, (n,), torch.int64 if wide else torch.int32, dev)
        logprobs = logits.new_empty(n, dtype=torch.float32)
    entropy = logits.new_empty(n, dtype=torch.float32)
    if top:
        ids = logits.new_empty((n, top), dtype=torch.int32)
        tops = logits.new_empty((n, top), dtype=torch.float32)
    if lse is not None:
        _want("lse", lse, (n,), torch.float32, dev)
    if err_count is not None:
        _want("err_count", err_count, (1,), torch.int32, dev)
    L = load_serving_library()
    need = L.qemb_logprobs_workspace_bytes(n, v, _DTYPES[dtype], top)
    if workspace is not None:
        if workspace.numel() < need:
            raise ValueError("workspace must have at least %d bytes" % need)
        _want("workspace", workspace, workspace.shape, torch.uint8, dev)
    elif need:
        workspace = logits.new_empty(need, dtype=torch.uint8)
    _check("qemb_token_logprobs", _launch(
        dev, L.qemb_token_logprobs,
        logits.data_ptr(), n, v, _DTYPES[dtype], stride, _ptr(targets), INDEX_INT64 if wide else INDEX_INT32, top,
        _ptr(logprobs), entropy.data_ptr(), _ptr(lse), _ptr(ids), _ptr(tops), _ptr(workspace), _ptr(err_count),
        _raw_stream(dev)))
    return logprobs, entropy, ids, tops
