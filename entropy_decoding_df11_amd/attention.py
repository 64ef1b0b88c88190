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
given.  Serving's operators: they carry no gradients, and refuse tensors that do.
"""

from __future__ import annotations

from typing import Optional, Tuple, Union

from . import _lib, operators
from .operators import _check_outputs, _dtype, _no_tangents, _ptr, _run, _same_device, _stream


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
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{what} must be (tokens, heads, head_dim), with the cache's heads and head_dim")
    if t.stride(2) != 1 and shape[2] > 1 and t.numel():
        raise ValueError(f"{what} must be contiguous along its last dimension")


def _check_cache(k_cache, v_cache, page_table, starts, lengths):
    torch = operators.torch
    dev = k_cache.device
    code = _dtype(k_cache, "k_cache")
    shape = k_cache.shape
    if code == _lib.FP32 or v_cache.dtype != k_cache.dtype or len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be (pages, page, kv_heads, head_dim), bfloat16 or float16, alike")
    pages, page, heads, dim = shape
    if dim % 8 or not 8 <= dim <= _lib.MAX_HEAD_DIM or k_cache.stride(3) != 1 or v_cache.stride(3) != 1:
        raise ValueError("head_dim must be a multiple of 8, 8 to 256, and contiguous")
    if not pages or not page or not heads:
        raise ValueError("the cache must have a page, a place and a head")
    int32 = torch.int32
    if page_table.dtype != int32 or starts.dtype != int32 or lengths.dtype != int32:
        raise ValueError("page_table, starts and lengths must be int32")
    if lengths.dim() != 1 or starts.dim() != 1 or page_table.dim() != 2 or not lengths.is_contiguous() or \
            not starts.is_contiguous() or (page_table.stride(1) != 1 and page_table.shape[1] > 1):
        raise ValueError("starts and lengths must be contiguous vectors, page_table a matrix of contiguous rows")
    seqs = lengths.shape[0]
    if starts.shape[0] != seqs + 1 or page_table.shape[0] != seqs:
        raise ValueError("starts must have one element more than lengths, page_table one row for each")
    if not dev == v_cache.device == page_table.device == starts.device == lengths.device:
        raise ValueError(f"v_cache, page_table, starts and lengths must be on {dev}")
    return dev, code, shape


def _structs(k_cache, v_cache, page_table, starts, lengths, code, tokens):
    pages, page, heads, dim = k_cache.shape
    k0, k1, k2, _ = k_cache.stride()
    v0, v1, v2, _ = v_cache.stride()
    seqs, width = page_table.shape
    return (_lib.KV_CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), k0, k1, k2, v0, v1, v2, pages, page, heads, dim,
                               code, 0),
            _lib.KV_BATCH.pack(starts.data_ptr(), lengths.data_ptr(), page_table.data_ptr(), page_table.stride(0), seqs,
                               width, tokens, 0))


_GRADIENTS = "the cache's operators carry no gradients: call them under torch.no_grad()"


def _launch_append(dev, k, v, q, k_cache, v_cache, page_table, starts, lengths, rotary, positions, interleaved, q_out,
                   code):
    cache, batch = _structs(k_cache, v_cache, page_table, starts, lengths, code, k.shape[0])
    k0, k1, _ = k.stride()
    v0, v1, _ = v.stride()
    q_ptr = out_ptr = q0 = q1 = o0 = o1 = heads = rotary_ptr = rows = dims = 0
    if q is not None:
        if q_out is None:
            q_out = operators.torch.empty(q.shape, dtype=k_cache.dtype, device=dev)
        q_ptr, out_ptr, heads = q.data_ptr(), q_out.data_ptr(), q.shape[1]
        q0, q1, _ = q.stride()
        o0, o1, _ = q_out.stride()
    if rotary is not None:
        rotary_ptr, (rows, dims) = rotary.data_ptr(), rotary.shape
    a = _lib.APPEND.pack(k.data_ptr(), v.data_ptr(), q_ptr, out_ptr, rotary_ptr,
                         0 if positions is None else positions.data_ptr(), k0, k1, v0, v1, q0, q1, o0, o1, rows, dims,
                         1 if interleaved else 0, heads, operators._DTYPES[k.dtype])
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
    dev, code, (_, _, heads, dim) = _check_cache(k_cache, v_cache, page_table, starts, lengths)
    dtype = k.dtype
    _dtype(k, "k")
    _check_heads(k, "k", dim, heads)
    _check_heads(v, "v", dim, heads)
    tokens = k.shape[0]
    if v.shape[0] != tokens or v.dtype != dtype:
        raise ValueError("v must have k's shape and dtype")
    if not dev == k.device == v.device:
        raise ValueError(f"k and v must be on {dev}, the cache's device")
    needs = k.requires_grad or v.requires_grad or k_cache.requires_grad or v_cache.requires_grad
    if q is not None:
        _check_heads(q, "q", dim)
        if q.shape[0] != tokens or q.dtype != dtype or not q.shape[1]:
            raise ValueError("q must have k's tokens and dtype, and a head")
        _same_device(dev, "q", q)
        needs = needs or q.requires_grad
    if q_out is not None:
        if q is None:
            raise ValueError("q_out needs q")
        _check_heads(q_out, "q_out", dim, q.shape[1])
        if q_out.shape[0] != tokens or q_out.dtype != k_cache.dtype:
            raise ValueError("q_out must have q's shape and the cache's dtype")
        _same_device(dev, "q_out", q_out)
        needs = needs or q_out.requires_grad
    if rotary is not None:
        if rotary.dtype != torch.float32 or rotary.dim() != 2 or not rotary.is_contiguous() or not rotary.shape[0] or \
                rotary.shape[1] < 2 or rotary.shape[1] % 2 or rotary.shape[1] > dim:
            raise ValueError("rotary must be float32 (positions, dims), contiguous, dims even and at most head_dim")
        _same_device(dev, "rotary", rotary)
    if positions is not None:
        if positions.dtype != torch.int32 or positions.dim() != 1 or positions.shape[0] != tokens or \
                not positions.is_contiguous():
            raise ValueError("positions must be int32, one for each token, contiguous")
        _same_device(dev, "positions", positions)
    if needs and torch.is_grad_enabled():
        raise ValueError(_GRADIENTS)
    if operators._forward_ad._current_level >= 0:
        _no_tangents(k, v, q, k_cache, v_cache, q_out, rotary)
    out, = _run(dev, stream, _launch_append, k, v, q, k_cache, v_cache, page_table, starts, lengths, rotary, positions,
                interleaved, q_out, code)
    torch.autograd.graph.increment_version((k_cache, v_cache) if q_out is None else (k_cache, v_cache, q_out))
    return out


def _launch_attention(dev, q, k_cache, v_cache, page_table, starts, lengths, mask, scale, out, return_lse, code):
    torch = operators.torch
    cache, batch = _structs(k_cache, v_cache, page_table, starts, lengths, code, q.shape[0])
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev) if return_lse else None
    q0, q1, _ = q.stride()
    o0, o1, _ = out.stride()
    m_ptr = m0 = cols = 0
    if mask is not None:
        m_ptr, m0, cols = mask.data_ptr(), mask.stride(0), mask.shape[1]
        if not cols:
            # (a tensor without elements has no address, which would be no mask: any
            # other does, since none of it is read)
            m_ptr, m0 = starts.data_ptr(), 0
    a = _lib.ATTENTION.pack(q.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), m_ptr, q0, q1, o0, o1, m0,
                            cols, q.shape[1], scale, 0)
    lib = _lib.load()
    nbytes = lib.df11_tree_attention_workspace(cache, batch, a)
    work = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    status = lib.df11_tree_attention(cache, batch, a, _ptr(work), nbytes, _stream(dev))
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
    column is set (column j: the sequence's j-th new token; none past the last).

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
    dev, code, (_, _, heads, dim) = _check_cache(k_cache, v_cache, page_table, starts, lengths)
    _check_heads(q, "q", dim)
    if q.dtype != k_cache.dtype or not q.shape[1] or q.shape[1] % heads:
        raise ValueError("q must have the cache's dtype, and heads a multiple of the cache's")
    _same_device(dev, "q", q)
    if scale is None:
        scale = dim ** -0.5
    elif not 0.0 < scale <= 3.4e38:
        raise ValueError("scale must be positive and finite")
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8) or mask.dim() != 2 or mask.shape[0] != q.shape[0] or \
                (mask.shape[1] > 1 and mask.stride(1) != 1):
            raise ValueError("mask must be bool or uint8 (tokens, columns), contiguous along a row")
        _same_device(dev, "mask", mask)
    given = None
    if out is not None:
        _check_heads(out, "out", dim)
        if out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must have q's shape and dtype")
        _same_device(dev, "out", out)
        given = _check_outputs(out)
    if (q.requires_grad or k_cache.requires_grad or v_cache.requires_grad) and torch.is_grad_enabled():
        raise ValueError(_GRADIENTS)
    if operators._forward_ad._current_level >= 0:
        _no_tangents(q, k_cache, v_cache, out)
    out, lse = _run(dev, stream, _launch_attention, q, k_cache, v_cache, page_table, starts, lengths, mask, scale, out,
                    return_lse, code)
    if given:
        torch.autograd.graph.increment_version(given)
    return (out, lse) if return_lse else out
