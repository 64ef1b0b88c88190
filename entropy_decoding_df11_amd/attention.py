"""A paged cache of keys and values, and attention of new tokens over it.

What a step of generation does between a block's q, k and v products and its
output product (the C ABI's df11_append_kv and df11_tree_attention):

    q = append_kv(k, v, k_cache, v_cache, page_table, starts, lengths, q=q, rotary=table)
    o = tree_attention(q, k_cache, v_cache, page_table, starts, lengths, mask=tree)

The cache is two tensors (pages, page, kv_heads, head_dim) of any strides with
contiguous heads: (pages, kv_heads, page, head_dim) goes in transposed.  Of a
batch, sequence s has lengths[s] tokens in the cache, in the pages that
page_table[s] lists, and brings tokens starts[s] .. starts[s + 1] - 1; its i-th
new token belongs at place lengths[s] + i.  The new tokens are one for each
sequence when decoding, a piece of a prompt, or a tree of drafted tokens, whose
mask says which of its sequence's new tokens each one sees.

starts, lengths and page_table are int32 and stay on the GPU: no call waits for
the host, so that a captured step is replayed with other lengths and pages.
Tokens before starts[0] or behind starts[-1] (a captured batch's spare rows)
belong to no sequence, and their rows are left as they were.  What the arrays
hold is checked where it is used: places beyond the table and pages that do not
exist are neither read nor written.

As in operators.py the calls run on torch's current stream, or on the stream
given.  Serving's operators: they carry no gradients.
"""

from __future__ import annotations

import math
from typing import Optional, Tuple, Union

from . import _lib, operators
from .operators import _check_outputs, _dtype, _run, _same_device, _stream


def rotary_table(positions: int, dims: int, base: float = 10000.0, device="cuda") -> "torch.Tensor":  # noqa: F821
    """Cosines and sines for append_kv: float32 (positions, dims), row p with
    the cosines of p * base^(-2 i / dims), i < dims / 2, then their sines, from
    angles in 64 bits (float32 loses a far position's angle)."""
    import torch
    if positions < 0 or dims < 2 or dims % 2:
        raise ValueError("dims must be even and positive, positions not negative")
    i = torch.arange(dims // 2, dtype=torch.float64, device=device)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * float(base) ** (-2.0 * i / dims)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _check_heads(t, what, dim, heads=None):
    """Checks a (tokens, heads, head_dim) tensor."""
    if t.dim() != 3 or t.shape[2] != dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{what} must be (tokens, heads, head_dim), with the cache's heads and head_dim")
    if t.shape[2] > 1 and t.stride(2) != 1 and t.numel():
        raise ValueError(f"{what} must be contiguous along its last dimension")


def _strides(t, n):
    """The first n strides, 0 along dimensions of one element (theirs say nothing)."""
    shape, strides = t.shape, t.stride()
    return [strides[i] if shape[i] > 1 else 0 for i in range(n)]


def _check_cache(k_cache, v_cache, page_table, starts, lengths):
    torch = operators.torch
    dev = k_cache.device
    code = _dtype(k_cache, "k_cache")
    if code == _lib.FP32 or v_cache.dtype != k_cache.dtype or k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be (pages, page, kv_heads, head_dim), bfloat16 or float16, alike")
    pages, page, heads, dim = k_cache.shape
    if dim % 8 or not 8 <= dim <= _lib.MAX_HEAD_DIM or k_cache.stride(3) != 1 or v_cache.stride(3) != 1:
        raise ValueError("head_dim must be a multiple of 8, 8 to 256, and contiguous")
    if not pages or not page or not heads:
        raise ValueError("the cache must have a page, a place and a head")
    for name, t in (("page_table", page_table), ("starts", starts), ("lengths", lengths)):
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
        _same_device(dev, name, t)
    _same_device(dev, "v_cache", v_cache)
    if lengths.dim() != 1 or starts.dim() != 1 or page_table.dim() != 2 or not lengths.is_contiguous() or \
            not starts.is_contiguous() or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("starts and lengths must be contiguous vectors, page_table a matrix of contiguous rows")
    seqs = lengths.shape[0]
    if starts.shape[0] != seqs + 1 or page_table.shape[0] != seqs:
        raise ValueError("starts must have one element more than lengths, page_table one row for each")
    return dev, code


def _structs(k_cache, v_cache, page_table, starts, lengths, code, tokens):
    pages, page, heads, dim = k_cache.shape
    cache = _lib.KvCache(k_cache.data_ptr(), v_cache.data_ptr(), *_strides(k_cache, 3), *_strides(v_cache, 3), pages,
                         page, heads, dim, code)
    batch = _lib.KvBatch(starts.data_ptr(), lengths.data_ptr(), page_table.data_ptr(), page_table.stride(0),
                         page_table.shape[0], page_table.shape[1], tokens)
    return cache, batch


def _no_gradients(*tensors):
    if operators.torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError("the cache's operators carry no gradients: call them under torch.no_grad()")


def _launch_append(dev, k, v, q, k_cache, v_cache, page_table, starts, lengths, rotary, positions, interleaved, q_out,
                   code):
    cache, batch = _structs(k_cache, v_cache, page_table, starts, lengths, code, k.shape[0])
    ks, vs = _strides(k, 2), _strides(v, 2)
    a = _lib.Append(k=k.data_ptr(), v=v.data_ptr(), k_stride=ks[0], k_head_stride=ks[1], v_stride=vs[0],
                    v_head_stride=vs[1], dtype=operators._DTYPES[k.dtype])
    if q is not None:
        if q_out is None:
            q_out = operators.torch.empty(q.shape, dtype=k_cache.dtype, device=dev)
        a.q, (a.q_stride, a.q_head_stride), a.q_heads = q.data_ptr(), _strides(q, 2), q.shape[1]
        a.q_out, (a.q_out_stride, a.q_out_head_stride) = q_out.data_ptr(), _strides(q_out, 2)
    if rotary is not None:
        a.rotary, a.rotary_rows, a.rotary_dims, a.interleaved = rotary.data_ptr(), rotary.shape[0], rotary.shape[1], \
            interleaved
    if positions is not None:
        a.positions = positions.data_ptr()
    status = _lib.load().df11_append_kv(cache, batch, a, _stream(dev))
    if status:
        _lib.check(status, "df11_append_kv")
    return (q_out,)


def append_kv(k: "torch.Tensor", v: "torch.Tensor", k_cache: "torch.Tensor", v_cache: "torch.Tensor",  # noqa: F821
              page_table: "torch.Tensor", starts: "torch.Tensor", lengths: "torch.Tensor",  # noqa: F821
              q: Optional["torch.Tensor"] = None, rotary: Optional["torch.Tensor"] = None,  # noqa: F821
              positions: Optional["torch.Tensor"] = None, interleaved: bool = False,  # noqa: F821
              q_out: Optional["torch.Tensor"] = None, stream=None) -> Optional["torch.Tensor"]:  # noqa: F821
    """Writes the new tokens' keys and values to their places in the cache,
    rotated by their positions on the way, and returns their queries, rotated
    too, in the cache's type (df11_append_kv); None without q.

    k, v: (tokens, kv_heads, head_dim), q: (tokens, heads, head_dim), all of one
    type (bfloat16, float16 or float32: a product's sums), any strides with
    contiguous heads.  rotary: float32 (positions, dims) contiguous, dims even
    and at most head_dim, as rotary_table makes it (None: no rotation); a head's
    first dims elements are rotated in pairs (d, d + dims / 2), or with
    interleaved (2 d, 2 d + 1).  positions: int32, one for each token (None:
    each token's place; drafted trees have depths of their own); one beyond the
    table gives NaN.  q_out may be q itself.  Rotated in float32, rounded once."""
    if operators.torch is None:
        operators._import_torch()
    torch = operators.torch
    dev, code = _check_cache(k_cache, v_cache, page_table, starts, lengths)
    dim, heads = k_cache.shape[3], k_cache.shape[2]
    _dtype(k, "k")
    _check_heads(k, "k", dim, heads)
    _check_heads(v, "v", dim, heads)
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("v must have k's shape and dtype")
    for name, t in (("k", k), ("v", v), ("q", q), ("rotary", rotary), ("positions", positions), ("q_out", q_out)):
        _same_device(dev, name, t)
    if q is None:
        if q_out is not None:
            raise ValueError("q_out needs q")
    else:
        _check_heads(q, "q", dim)
        if q.shape[0] != k.shape[0] or q.dtype != k.dtype or not q.shape[1]:
            raise ValueError("q must have k's tokens and dtype, and a head")
        if q_out is not None:
            _check_heads(q_out, "q_out", dim, q.shape[1])
            if q_out.shape != q.shape or q_out.dtype != k_cache.dtype:
                raise ValueError("q_out must have q's shape and the cache's dtype")
    if rotary is not None:
        if rotary.dtype != torch.float32 or rotary.dim() != 2 or not rotary.is_contiguous() or not rotary.shape[0] or \
                rotary.shape[1] < 2 or rotary.shape[1] % 2 or rotary.shape[1] > dim:
            raise ValueError("rotary must be float32 (positions, dims), contiguous, dims even and at most head_dim")
    if positions is not None:
        if positions.dtype != torch.int32 or positions.dim() != 1 or positions.shape[0] != k.shape[0] or \
                not positions.is_contiguous():
            raise ValueError("positions must be int32, one for each token, contiguous")
    _no_gradients(k, v, q, k_cache, v_cache, q_out)
    given = [t for t in (k_cache, v_cache, q_out) if t is not None]
    out, = _run(dev, stream, _launch_append, k, v, q, k_cache, v_cache, page_table, starts, lengths, rotary, positions,
                interleaved, q_out, code)
    torch.autograd.graph.increment_version(given)
    return out


def _launch_attention(dev, q, k_cache, v_cache, page_table, starts, lengths, mask, scale, out, lse, code):
    torch = operators.torch
    cache, batch = _structs(k_cache, v_cache, page_table, starts, lengths, code, q.shape[0])
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    if lse is True:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev)
    qs, os = _strides(q, 2), _strides(out, 2)
    a = _lib.Attention(q=q.data_ptr(), out=out.data_ptr(), q_stride=qs[0], q_head_stride=qs[1], out_stride=os[0],
                       out_head_stride=os[1], q_heads=q.shape[1], scale=scale)
    if lse is not None:
        a.lse = lse.data_ptr()
    if mask is not None:
        a.mask, a.mask_stride, a.mask_cols = mask.data_ptr(), mask.stride(0), mask.shape[1]
    lib = _lib.load()
    nbytes = lib.df11_tree_attention_workspace(cache, batch, a)
    work = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    status = lib.df11_tree_attention(cache, batch, a, work.data_ptr(), nbytes, _stream(dev))
    if status:
        _lib.check(status, "df11_tree_attention")
    return out, lse


def tree_attention(q: "torch.Tensor", k_cache: "torch.Tensor", v_cache: "torch.Tensor",  # noqa: F821
                   page_table: "torch.Tensor", starts: "torch.Tensor", lengths: "torch.Tensor",  # noqa: F821
                   mask: Optional["torch.Tensor"] = None, scale: Optional[float] = None,  # noqa: F821
                   out: Optional["torch.Tensor"] = None, return_lse: bool = False,  # noqa: F821
                   stream=None) -> Union["torch.Tensor", Tuple["torch.Tensor", "torch.Tensor"]]:  # noqa: F821
    """Attention of the new tokens over the cache that already holds their keys
    and values (df11_tree_attention): softmax(scale q k^T) v over what each sees,
    which is its sequence's cached places, and of its new tokens those up to
    itself, or with mask, a bool or uint8 (tokens, columns) tensor, those whose
    column is set (column j: the sequence's j-th new token).

    q: (tokens, heads, head_dim) of the cache's type, heads a multiple of the
    cache's (query head h reads key head h // (heads / kv_heads)), rows 16-byte
    aligned; scale: positive, head_dim^-0.5 by default; out: q's shape and type,
    may be q itself.  Returns out, or with return_lse (out, lse): lse the
    natural logarithm of each query's sum of exponentials, float32 (tokens,
    heads).  A query that sees nothing gets zeros and minus infinity.  Scores
    and sums are float32, and the same call gives the same bits again."""
    if operators.torch is None:
        operators._import_torch()
    torch = operators.torch
    dev, code = _check_cache(k_cache, v_cache, page_table, starts, lengths)
    dim, heads = k_cache.shape[3], k_cache.shape[2]
    _check_heads(q, "q", dim)
    if q.dtype != k_cache.dtype or not q.shape[1] or q.shape[1] % heads:
        raise ValueError("q must have the cache's dtype, and heads a multiple of the cache's")
    if scale is None:
        scale = 1.0 / math.sqrt(dim)
    elif not 0.0 < scale < math.inf:
        raise ValueError("scale must be positive and finite")
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8) or mask.dim() != 2 or mask.shape[0] != q.shape[0] or \
                (mask.shape[1] > 1 and mask.stride(1) != 1):
            raise ValueError("mask must be bool or uint8 (tokens, columns), contiguous along a row")
    if out is not None:
        _check_heads(out, "out", dim)
        if out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must have q's shape and dtype")
    for name, t in (("q", q), ("mask", mask), ("out", out)):
        _same_device(dev, name, t)
    _no_gradients(q, k_cache, v_cache)
    given = None if out is None else _check_outputs(out)
    out, lse = _run(dev, stream, _launch_attention, q, k_cache, v_cache, page_table, starts, lengths, mask, scale, out,
                    True if return_lse else None, code)
    if given:
        torch.autograd.graph.increment_version(given)
    return (out, lse) if return_lse else out
