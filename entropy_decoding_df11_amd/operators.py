"""Operators around the products of a transformer block, on the GPU.

The framework keeps a block's weights compressed and multiplies by them; this
module has what a forward computes between one product and the next (the C
ABI's operators in include/df11.h), each differentiable: under torch's
autograd they give the gradients of the activations, the biases, the residual
and the norm's weight.  (The compressed weights are frozen: they have none.)

    y = rms_norm(x, weight)                       # norm
    y, s = rms_norm(x, weight, residual=r)        # s = x + r, y = norm of s
    y = matmul_epilogue(w, x, bias, "gelu", r)    # act(x W^T + bias) + r
    h = gated_matmul(gate, up, x)                 # silu(x Wg^T) * (x Wu^T)

As in df11.py every step runs in libdf11.so on torch's current stream, or on
the stream given; this module checks and passes arguments.  The caller orders
a stream that it gives after whatever makes the inputs and before whatever
reads the outputs; the tensors may be freed at once, the weights must stay
until the stream has run.  Calls of one weight may overlap, on any streams and
from any threads, and may be captured into graphs (a backward pass, as with
torch's own operators, from leaves that no eager graph still holds).

A call at one token is a few microseconds on the GPU, so what runs on every
call is kept short here: the stream's handle is asked for without making a
Stream object, and shapes are checked once, in the forward call.
"""

from __future__ import annotations

from typing import Optional, Tuple, Union

from . import _lib

# torch, its types' codes and the autograd functions, filled in by the first
# call (importing this package does not import torch).
torch = None
_DTYPES = {}
_FLOATS = ()
_Norm = _Product = None

_MAX_ROWS = 1 << 30


def _import_torch() -> None:
    global torch, _FLOATS
    import torch as module
    _DTYPES.update({module.bfloat16: _lib.BF16, module.float16: _lib.FP16, module.float32: _lib.FP32})
    _FLOATS = (module.bfloat16, module.float32)
    _make_functions(module)
    torch = module  # last: a call of another thread that sees it needs the rest


def _dtype(t: "torch.Tensor", what: str) -> int:  # noqa: F821
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be bfloat16, float16 or float32, not {t.dtype}")
    return code


def _rows(t: "torch.Tensor", cols: int, what: str) -> Tuple["torch.Tensor", int]:  # noqa: F821
    """t as (rows, cols) with unit stride along a row, and its row stride."""
    if t.is_contiguous():
        return (t if t.dim() == 2 else t.view(-1, cols)), cols
    dim = t.dim()
    if dim != 2:
        try:
            t = t.unsqueeze(0) if dim == 1 else t.view(-1, cols)
        except RuntimeError:
            raise ValueError(f"{what} must have rows at one stride") from None
    if cols > 1 and t.numel() and t.stride(1) != 1:
        raise ValueError(f"{what} must be contiguous along its last dimension")
    return t, (t.stride(0) if t.shape[0] > 1 else cols)


def _same_device(dev, what: str, t) -> None:
    if t is not None and t.device != dev:
        raise ValueError(f"{what} must be on {dev}, not on {t.device}")


def _check_outputs(*outs):
    """The outputs that the caller gave.  They are written behind autograd's
    back: none may be part of a graph itself, and each one's version has to be
    raised afterwards, for the graphs that have kept it."""
    given = [t for t in outs if t is not None]
    if torch.is_grad_enabled() and any(t.requires_grad for t in given):
        raise ValueError("an output that is given must not require a gradient")
    return given


def _run(dev, stream, launch, *args):
    """launch(*args) with dev current and, if given, stream: allocations made
    there belong to the stream of the launch.  The caching allocator is told
    which tensors a given stream uses beside their own, so that one that is
    freed early is not handed out again while the stream has yet to get to it;
    and that the caller's stream will read the outputs."""
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU")
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"stream must be on {dev}, not on {stream.device}")
        caller = torch.cuda.current_stream(dev)
        with torch.cuda.stream(stream):
            outs = launch(dev, *args)
        if stream != caller:
            for group in (args, *(a for a in args if isinstance(a, tuple))):
                for t in group:
                    if isinstance(t, torch.Tensor):
                        t.record_stream(stream)
            for t in outs:
                if isinstance(t, torch.Tensor):
                    t.record_stream(caller)
        return outs
    if dev.index == torch._C._cuda_getDevice():
        return launch(dev, *args)
    with torch.cuda.device(dev):
        return launch(dev, *args)


def _stream(dev) -> int:
    """Handle of torch's current stream on dev."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _rowwise(t):
    """A gradient that autograd hands over, with rows at one stride."""
    if t.numel() == 0:
        return t
    try:
        _rows(t, t.shape[-1], "gradient")
        return t
    except ValueError:
        return t.contiguous()


# ---------------------------------------------------------------------------
# RMS norm.
# ---------------------------------------------------------------------------

def _check_norm(x, weight, residual, out, sum_out):
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x must have at least one column")
    code = wcode = _dtype(x, "x")
    # (the C ABI counts rows and columns in 32 bits)
    if x.shape[-1] > _MAX_ROWS or x.numel() > _MAX_ROWS * x.shape[-1]:
        raise ValueError("x must have at most 2^30 rows and 2^30 columns")
    dev = x.device
    for name, t in (("residual", residual), ("out", out), ("sum_out", sum_out)):
        if t is not None:
            if t.shape != x.shape or t.dtype != x.dtype:
                raise ValueError(f"{name} must have x's shape and dtype")
            _same_device(dev, name, t)
    if sum_out is not None and residual is None:
        raise ValueError("sum_out needs a residual")
    if weight is not None:
        wcode = _dtype(weight, "weight")
        if weight.dim() != 1 or weight.shape[0] != x.shape[-1] or not weight.is_contiguous() or \
                wcode not in (code, _lib.FP32):
            raise ValueError("weight must be contiguous, one element per column, of x's dtype or float32")
        _same_device(dev, "weight", weight)
    return code, wcode


def _launch_norm(dev, x, weight, residual, eps, out, sum_out, keep_rstd, code, wcode):
    cols = x.shape[-1]
    x2, xs = _rows(x, cols, "x")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    y2, ys = _rows(out, cols, "out")
    res = total = None
    rs = ss = 0
    if residual is not None:
        r2, rs = _rows(residual, cols, "residual")
        if sum_out is None:
            sum_out = torch.empty(x.shape, dtype=x.dtype, device=dev)
        s2, ss = _rows(sum_out, cols, "sum_out")
        res, total = r2.data_ptr(), s2.data_ptr()
    rows = x2.shape[0]
    rstd = torch.empty(rows, dtype=torch.float32, device=dev) if keep_rstd else None
    status = _lib.load().df11_rms_norm(x2.data_ptr(), xs, res, rs, _ptr(weight), wcode, rows, cols, code, eps, total,
                                       ss, y2.data_ptr(), ys, _ptr(rstd), _stream(dev))
    if status:
        _lib.check(status, "df11_rms_norm")
    return out, sum_out, rstd


def _launch_norm_grad(dev, s, weight, rstd, dy, dsum, want_weight):
    cols = s.shape[-1]
    code = _DTYPES[s.dtype]
    wcode = code if weight is None else _DTYPES[weight.dtype]
    s2, ss = _rows(s, cols, "s")
    dy2, dys = _rows(dy, cols, "dy")
    d2, ds = (None, 0) if dsum is None else _rows(dsum, cols, "dsum")
    rows = s2.shape[0]
    lib = _lib.load()
    dx = torch.empty(s.shape, dtype=s.dtype, device=dev)
    dw, work, nbytes = None, None, 0
    if want_weight:
        dw = torch.empty_like(weight)
        nbytes = lib.df11_rms_norm_grad_workspace(rows, cols)
        work = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    status = lib.df11_rms_norm_grad(s2.data_ptr(), ss, _ptr(weight), wcode, rstd.data_ptr(), dy2.data_ptr(), dys,
                                    _ptr(d2), ds, rows, cols, code, dx.data_ptr(), cols, _ptr(dw), _ptr(work), nbytes,
                                    _stream(dev))
    if status:
        _lib.check(status, "df11_rms_norm_grad")
    return dx, dw


def rms_norm(x: "torch.Tensor", weight: Optional["torch.Tensor"] = None,  # noqa: F821
             residual: Optional["torch.Tensor"] = None, eps: float = 1e-5,  # noqa: F821
             out: Optional["torch.Tensor"] = None, sum_out: Optional["torch.Tensor"] = None,  # noqa: F821
             stream=None) -> Union["torch.Tensor", Tuple["torch.Tensor", "torch.Tensor"]]:  # noqa: F821
    """The RMS norm of x's last dimension, with the residual's addition
    (df11_rms_norm).  Without a residual: y = x * rsqrt(mean(x^2) + eps) *
    weight.  With one: (y, s), s = x + residual rounded to x's dtype and y the
    norm of s.

    x: bfloat16, float16 or float32, 1 to 2^30 columns and up to 2^30 rows at
    one stride (any stride).  weight: one element per column, of x's dtype or
    float32 (None: ones).  residual, out, sum_out: x's shape and dtype; out and
    sum_out may each be x or residual themselves.  The sums are float32; y and
    s are rounded once.  Where an input requires a gradient the outputs carry
    it (then neither out, sum_out nor stream may be given)."""
    if torch is None:
        _import_torch()
    code, wcode = _check_norm(x, weight, residual, out, sum_out)
    if (x.requires_grad or (weight is not None and weight.requires_grad)
            or (residual is not None and residual.requires_grad)) and torch.is_grad_enabled():
        if out is not None or sum_out is not None or stream is not None:
            raise ValueError("out, sum_out and stream are for calls without gradients")
        return _Norm.apply(x, weight, residual, eps, code, wcode)
    given = None if out is None and sum_out is None else _check_outputs(out, sum_out)
    y, s, _ = _run(x.device, stream, _launch_norm, x, weight, residual, eps, out, sum_out, False, code, wcode)
    if given:
        torch.autograd.graph.increment_version(given)
    return y if residual is None else (y, s)


# ---------------------------------------------------------------------------
# Products with an epilogue.
# ---------------------------------------------------------------------------

def _check_product(ws, x, biases, activation, residual, out, out_dtype):
    """Checks a product's arguments; (device, activation code, out's dtype)."""
    for w in ws:
        if len(w.shape) != 2 or not w.tile_cols:
            raise ValueError("weights must be 2-D and compressed with layout='mfma_tiles'")
    out_f, in_f = ws[0].shape
    dev = ws[0]._bufs["enc"].device
    if len(ws) == 2:
        if ws[1].shape != ws[0].shape or ws[1].decode_table_bits != ws[0].decode_table_bits:
            raise ValueError("gate and up must have the same shape and decode-table width")
        _same_device(dev, "up", ws[1]._bufs["enc"])
    if x.dtype != torch.bfloat16 or x.dim() == 0 or x.shape[-1] != in_f:
        raise ValueError("x must be a bfloat16 (..., in_features) tensor")
    if x.numel() // in_f * max(in_f, out_f) >= 1 << 32:
        raise ValueError("tokens times features must be below 2^32")
    _same_device(dev, "x", x)
    act = _lib.ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be None or one of {sorted(k for k in _lib.ACTIVATIONS if k)}")
    first = None
    for b in biases:
        if b is not None:
            if b.dim() != 1 or b.shape[0] != out_f or b.dtype not in _FLOATS or not b.is_contiguous():
                raise ValueError("a bias must be contiguous bfloat16 or float32, one element per output feature")
            if first is not None and b.dtype != first.dtype:
                raise ValueError("both biases must have one dtype")
            first = b
            _same_device(dev, "bias", b)
    for name, t in (("residual", residual), ("out", out)):
        if t is not None:
            if t.dtype not in _FLOATS or t.shape != x.shape[:-1] + (out_f,):
                raise ValueError(f"{name} must be a bfloat16 or float32 (..., out_features) tensor")
            _same_device(dev, name, t)
    if out is not None:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out_dtype must be out's dtype")
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = torch.bfloat16
    elif out_dtype not in _FLOATS:
        raise ValueError("out_dtype must be bfloat16 or float32")
    return dev, act, out_dtype


def _launch_product(dev, ws, x, biases, act, residual, out, out_dtype, keep):
    """act(x W^T + b) [* (x Wu^T + bu)] + residual; with keep, also the sums
    before the activation, float32."""
    out_f, in_f = ws[0].shape
    x2, xs = _rows(x, in_f, "x")
    x_ptr = x2.data_ptr()
    if x_ptr % 16 or xs % 8:
        raise ValueError("x's rows must be 16-byte aligned")
    tokens = x2.shape[0]
    if out is None:
        out = torch.empty(x.shape[:-1] + (out_f,), dtype=out_dtype, device=dev)
    pre = [torch.empty((tokens, out_f), dtype=torch.float32, device=dev) for _ in ws] if keep else ()
    if tokens == 0 or out_f == 0:
        return out, pre
    y2, ys = _rows(out, out_f, "out")
    e = _lib.Epilogue(out=y2.data_ptr(), out_stride=ys, out_dtype=_DTYPES[out_dtype], activation=act)
    for i, b in enumerate(biases):
        if b is not None:
            e.bias[i], e.bias_dtype = b.data_ptr(), _DTYPES[b.dtype]
    if residual is not None:
        r2, e.residual_stride = _rows(residual, out_f, "residual")
        e.residual, e.residual_dtype = r2.data_ptr(), _DTYPES[residual.dtype]
    for i, p in enumerate(pre):
        e.pre[i] = p.data_ptr()
    lib = _lib.load()
    first, second = ws[0]._stream_struct, ws[1]._stream_struct if len(ws) == 2 else None
    nbytes = lib.df11_epilogue_workspace(first, second, tokens)
    work = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    # (no product uses the weights' work counters: nothing to order it after)
    if second is None:
        status = lib.df11_matmul_epilogue(first, x_ptr, xs, tokens, in_f, out_f, e, work.data_ptr(), nbytes,
                                          _stream(dev))
    else:
        status = lib.df11_gated_matmul(first, second, x_ptr, xs, tokens, in_f, out_f, e, work.data_ptr(), nbytes,
                                       _stream(dev))
    if status:
        _lib.check(status, "df11_matmul_epilogue" if second is None else "df11_gated_matmul")
    return out, pre


def _launch_product_grad(dev, ws, pre, dy, act, x_shape, want_x, biases):
    """(dx or None, the biases' gradients): biases[i] is the type of a bias
    whose gradient is wanted, or None."""
    out_f, in_f = ws[0].shape
    if out_f == 0:
        return (torch.zeros(x_shape, dtype=torch.bfloat16, device=dev) if want_x else None,
                [None if b is None else torch.empty(0, dtype=b, device=dev) for b in biases])
    dy2, dys = _rows(dy, out_f, "dy")
    tokens = dy2.shape[0]
    dx = torch.empty(x_shape, dtype=torch.bfloat16, device=dev) if want_x else None
    db = [None if b is None else torch.empty(out_f, dtype=b, device=dev) for b in biases]
    g = _lib.ProductGrad(dy=dy2.data_ptr(), dy_stride=dys, dy_dtype=_DTYPES[dy.dtype], activation=act)
    for i, p in enumerate(pre):
        g.pre[i] = p.data_ptr()
    if want_x:
        g.dx, g.dx_stride, g.dx_dtype = dx.data_ptr(), in_f, _lib.BF16
    for i, b in enumerate(db):
        if b is not None:
            g.dbias[i], g.bias_dtype = b.data_ptr(), _DTYPES[b.dtype]
    lib = _lib.load()
    first, second = ws[0]._stream_struct, ws[1]._stream_struct if len(ws) == 2 else None
    nbytes = lib.df11_epilogue_grad_workspace(first, second, tokens, g) if tokens else 0
    work = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    status = lib.df11_matmul_epilogue_grad(first, second, tokens, in_f, out_f, g, work.data_ptr(), nbytes,
                                           _stream(dev))
    if status:
        _lib.check(status, "df11_matmul_epilogue_grad")
    return dx, db


def _product(ws, x, biases, activation, residual, out, out_dtype, stream):
    if torch is None:
        _import_torch()
    dev, act, out_dtype = _check_product(ws, x, biases, activation, residual, out, out_dtype)
    if (x.requires_grad or (residual is not None and residual.requires_grad)
            or any(b is not None and b.requires_grad for b in biases)) and torch.is_grad_enabled():
        if out is not None or stream is not None:
            raise ValueError("out and stream are for calls without gradients")
        return _Product.apply(x, residual, biases[0], biases[-1] if len(ws) == 2 else None, ws, act, out_dtype)
    given = None if out is None else _check_outputs(out)
    y = _run(dev, stream, _launch_product, ws, x, biases, act, residual, out, out_dtype, False)[0]
    if given:
        torch.autograd.graph.increment_version(given)
    return y


def matmul_epilogue(w, x: "torch.Tensor", bias: Optional["torch.Tensor"] = None,  # noqa: F821
                    activation: Optional[str] = None, residual: Optional["torch.Tensor"] = None,  # noqa: F821
                    out: Optional["torch.Tensor"] = None, out_dtype=None, stream=None) -> "torch.Tensor":  # noqa: F821
    """act(x W^T + bias) + residual on the matrix cores with W compressed
    (df11_matmul_epilogue), for any number of tokens.

    w: a DF11Tensor compressed with layout="mfma_tiles"; x: bfloat16 (...,
    in_features), rows at one stride and 16-byte aligned, tokens times features
    (in or out) below 2^32; bias: bfloat16 or float32, one element per output
    feature; activation: None, "relu", "silu", "gelu" or "gelu_tanh"; residual:
    bfloat16 or float32 (..., out_features).
    Returns out, bfloat16 unless out or out_dtype says float32; out may be the
    residual itself.  Everything before out is float32, and the same call gives
    the same bits again.  Where x, bias or residual require a gradient the
    output carries it (then neither out nor stream may be given): the sums
    before an activation are kept for it in float32, dz is rounded to bfloat16
    for x's gradient (not for the bias's), and w itself is frozen."""
    return _product((w,), x, (bias,), activation, residual, out, out_dtype, stream)


def gated_matmul(gate, up, x: "torch.Tensor", gate_bias: Optional["torch.Tensor"] = None,  # noqa: F821
                 up_bias: Optional["torch.Tensor"] = None, activation: Optional[str] = "silu",  # noqa: F821
                 residual: Optional["torch.Tensor"] = None, out: Optional["torch.Tensor"] = None,  # noqa: F821
                 out_dtype=None, stream=None) -> "torch.Tensor":  # noqa: F821
    """act(x Wg^T + gate_bias) * (x Wu^T + up_bias) + residual, both
    projections in one launch (df11_gated_matmul): the first half of a gated
    feed-forward block.  gate and up have the same shape; otherwise as
    matmul_epilogue."""
    return _product((gate, up), x, (gate_bias, up_bias), activation, residual, out, out_dtype, stream)


# ---------------------------------------------------------------------------
# Gradients.
# ---------------------------------------------------------------------------

def _make_functions(torch) -> None:
    global _Norm, _Product
    from torch.autograd.function import once_differentiable

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, residual, eps, code, wcode):
            y, s, rstd = _run(x.device, None, _launch_norm, x, weight, residual, eps, None, None, True, code, wcode)
            ctx.save_for_backward(x if residual is None else s, weight, rstd)
            ctx.set_materialize_grads(False)
            return y if residual is None else (y, s)

        @staticmethod
        @once_differentiable
        def backward(ctx, dy, ds=None):
            s, weight, rstd = ctx.saved_tensors
            want_x, want_w, want_r = ctx.needs_input_grad[:3]
            if dy is None:
                dx, dw = ds, None
            else:
                dx, dw = _run(s.device, None, _launch_norm_grad, s, weight, rstd, _rowwise(dy),
                              None if ds is None else _rowwise(ds), want_w)
            return dx if want_x else None, dw, dx if want_r else None, None, None, None

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, residual, bias0, bias1, ws, act, out_dtype):
            biases = (bias0, bias1)[:len(ws)]
            keep = len(ws) == 2 or act != 0
            y, pre = _run(x.device, None, _launch_product, ws, x, biases, act, residual, None, out_dtype, keep)
            ctx.save_for_backward(*pre)
            ctx.ws, ctx.act, ctx.x_shape = ws, act, x.shape
            ctx.types = [None if t is None else t.dtype for t in (residual, bias0, bias1)]
            return y

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            want_x, want_r, want0, want1 = ctx.needs_input_grad[:4]
            residual, bias0, bias1 = ctx.types
            db = None, None
            dx = None
            if want_x or want0 or want1:
                dx, db = _run(dy.device, None, _launch_product_grad, ctx.ws, ctx.saved_tensors, _rowwise(dy), ctx.act,
                              ctx.x_shape, want_x,
                              (bias0 if want0 else None, bias1 if want1 else None)[:len(ctx.ws)])
            return (dx, dy.to(residual) if want_r else None, db[0], db[1] if len(db) == 2 else None, None,
                    None, None)

    _Norm, _Product = Norm, Product
