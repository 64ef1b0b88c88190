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
the stream given; this module checks and passes arguments.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple, Union

from . import _lib


def _dtypes():
    import torch
    return {torch.bfloat16: _lib.BF16, torch.float16: _lib.FP16, torch.float32: _lib.FP32}


_DTYPES = None


def _dtype(t: "torch.Tensor", what: str) -> int:  # noqa: F821
    global _DTYPES
    if _DTYPES is None:
        _DTYPES = _dtypes()
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be bfloat16, float16 or float32, not {t.dtype}")
    return code


def _rows(t: "torch.Tensor", cols: int, what: str) -> Tuple["torch.Tensor", int]:  # noqa: F821
    """t as (rows, cols) with unit stride along a row, and its row stride."""
    if t.dim() == 2:
        v = t
    elif t.dim() == 1:
        v = t.unsqueeze(0)
    else:
        try:
            v = t.view(-1, cols) if t.dim() and t.numel() else t.reshape(0, cols)
        except RuntimeError:
            raise ValueError(f"{what} must have rows at one stride") from None
    if cols > 1 and v.numel() and v.stride(1) != 1:
        raise ValueError(f"{what} must be contiguous along its last dimension")
    stride = v.stride(0) if v.shape[0] > 1 else cols
    if stride < 0:
        raise ValueError(f"{what} must not have negative strides")
    return v, stride


def _same_device(dev, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on {dev}, not on {t.device}")


class _on:
    """The device and stream of a launch: makes dev the current device and
    allocations belong to the stream, and gives its handle."""

    __slots__ = ("dev", "stream", "handle", "_guards")

    def __init__(self, dev, stream):
        import torch
        if dev.type != "cuda":
            raise ValueError("tensors must be on a GPU")
        self.dev, self.stream = dev, stream
        self._guards = ()
        if stream is not None:
            if stream.device != dev:
                raise ValueError(f"stream must be on {dev}, not on {stream.device}")
            self._guards = (torch.cuda.stream(stream),)  # (sets the device as well)
        elif dev.index != torch.cuda.current_device():
            self._guards = (torch.cuda.device(dev),)

    def __enter__(self):
        import torch
        for g in self._guards:
            g.__enter__()
        self.handle = torch.cuda.current_stream(self.dev).cuda_stream if self.stream is None else \
            self.stream.cuda_stream
        return self.handle

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check_norm(x, weight, residual):
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x must have at least one column")
    code = _dtype(x, "x")
    cols = x.shape[-1]
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError("residual must have x's shape and dtype")
    wcode = code
    if weight is not None:
        wcode = _dtype(weight, "weight")
        if weight.shape != (cols,) or not weight.is_contiguous() or wcode not in (code, _lib.FP32):
            raise ValueError("weight must be contiguous, one element per column, of x's dtype or float32")
    _same_device(x.device, weight=weight, residual=residual)
    return code, wcode, cols


def _norm_forward(x, weight, residual, eps, out, sum_out, stream, keep_rstd):
    import torch
    code, wcode, cols = _check_norm(x, weight, residual)
    x2, xs = _rows(x, cols, "x")
    r2, rs = (None, 0) if residual is None else _rows(residual, cols, "residual")
    for name, t in (("out", out), ("sum_out", sum_out)):
        if t is not None and (t.shape != x.shape or t.dtype != x.dtype):
            raise ValueError(f"{name} must have x's shape and dtype")
    _same_device(x.device, out=out, sum_out=sum_out)
    if sum_out is not None and residual is None:
        raise ValueError("sum_out needs a residual")
    with _on(x.device, stream) as st:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        y2, ys = _rows(out, cols, "out")
        s2, ss = None, 0
        if residual is not None:
            if sum_out is None:
                sum_out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            s2, ss = _rows(sum_out, cols, "sum_out")
        rows = x2.shape[0]
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device) if keep_rstd else None
        _lib.check(_lib.load().df11_rms_norm(x2.data_ptr(), xs, _ptr(r2), rs, _ptr(weight), wcode, rows, cols, code,
                                             eps, _ptr(s2), ss, y2.data_ptr(), ys, _ptr(rstd), st), "df11_rms_norm")
    return out, sum_out, rstd


def _norm_backward(s, weight, rstd, dy, dsum, want_weight):
    import torch
    code, wcode, cols = _check_norm(s, weight, None)
    s2, ss = _rows(s, cols, "s")
    dy2, dys = _rows(dy, cols, "dy")
    d2, ds = (None, 0) if dsum is None else _rows(dsum, cols, "dsum")
    rows = s2.shape[0]
    lib = _lib.load()
    with _on(s.device, None) as st:
        dx = torch.empty(s.shape, dtype=s.dtype, device=s.device)
        dw, ws, nbytes = None, None, 0
        if want_weight:
            dw = torch.empty_like(weight)
            nbytes = lib.df11_rms_norm_grad_workspace(rows, cols)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=s.device)
        _lib.check(lib.df11_rms_norm_grad(s2.data_ptr(), ss, _ptr(weight), wcode, rstd.data_ptr(), dy2.data_ptr(),
                                          dys, _ptr(d2), ds, rows, cols, code, dx.data_ptr(), cols, _ptr(dw),
                                          _ptr(ws), nbytes, st), "df11_rms_norm_grad")
    return dx, dw


def _rowwise(t):
    """A gradient that autograd hands over, with rows at one stride."""
    try:
        _rows(t, t.shape[-1], "gradient")
        return t
    except ValueError:
        return t.contiguous()


_FUNCTIONS = {}


def _function(name):
    """torch.autograd.Function classes, made at first use (importing this
    package does not import torch)."""
    if name not in _FUNCTIONS:
        import torch
        from torch.autograd.function import once_differentiable

        class Norm(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, weight, residual, eps):
                y, s, rstd = _norm_forward(x, weight, residual, eps, None, None, None, True)
                ctx.save_for_backward(x if residual is None else s, weight, rstd)
                ctx.has_residual = residual is not None
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
                    dx, dw = _norm_backward(s, weight, rstd, _rowwise(dy), None if ds is None else _rowwise(ds),
                                            want_w)
                return dx if want_x else None, dw, dx if want_r else None, None

        class Product(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, residual, bias0, bias1, ws, activation, out_dtype):
                biases = (bias0, bias1)[:len(ws)]
                keep = len(ws) == 2 or activation not in (None, "none")
                y, pre = _product_forward(ws, x, biases, activation, residual, None, out_dtype, None, keep)
                # (a bias is kept for its type alone)
                ctx.save_for_backward(bias0, bias1, *pre)
                ctx.ws, ctx.activation, ctx.x_shape = ws, activation, x.shape
                ctx.residual_dtype = None if residual is None else residual.dtype
                return y

            @staticmethod
            @once_differentiable
            def backward(ctx, dy):
                bias0, bias1, *pre = ctx.saved_tensors
                want_x, want_r, want0, want1 = ctx.needs_input_grad[:4]
                biases = [b if want else None for b, want in ((bias0, want0), (bias1, want1))][:len(ctx.ws)]
                dx, db = _product_backward(ctx.ws, pre, dy, _lib.ACTIVATIONS[ctx.activation or "none"], ctx.x_shape,
                                           want_x, biases)
                dr = dy.to(ctx.residual_dtype) if want_r else None
                return dx, dr, db[0], db[1] if len(db) == 2 else None, None, None, None

        _FUNCTIONS["norm"] = Norm
        _FUNCTIONS["product"] = Product
    return _FUNCTIONS[name]


def rms_norm(x: "torch.Tensor", weight: Optional["torch.Tensor"] = None,  # noqa: F821
             residual: Optional["torch.Tensor"] = None, eps: float = 1e-5,  # noqa: F821
             out: Optional["torch.Tensor"] = None, sum_out: Optional["torch.Tensor"] = None,  # noqa: F821
             stream=None) -> Union["torch.Tensor", Tuple["torch.Tensor", "torch.Tensor"]]:  # noqa: F821
    """The RMS norm of x's last dimension, with the residual's addition
    (df11_rms_norm).  Without a residual: y = x * rsqrt(mean(x^2) + eps) *
    weight.  With one: (y, s), s = x + residual rounded to x's dtype and y the
    norm of s.

    x: bfloat16, float16 or float32, at least one column, rows at one stride
    (any stride).  weight: one element per column, of x's dtype or float32
    (None: ones).  residual, out, sum_out: x's shape and dtype; out and
    sum_out may each be x or residual themselves.  The sums are float32; y and
    s are rounded once.  Where an input requires a gradient the outputs carry
    it (then neither out, sum_out nor stream may be given)."""
    import torch
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad)
                                    or (residual is not None and residual.requires_grad)):
        if out is not None or sum_out is not None or stream is not None:
            raise ValueError("out, sum_out and stream are for calls without gradients")
        return _function("norm").apply(x, weight, residual, eps)
    y, s, _ = _norm_forward(x, weight, residual, eps, out, sum_out, stream, False)
    return y if residual is None else (y, s)


# ---------------------------------------------------------------------------
# Products with an epilogue.
# ---------------------------------------------------------------------------

def _check_product(ws, x, biases, activation, residual, out, out_dtype):
    """Checks a product's arguments; (x as rows, its stride, activation code,
    out's dtype)."""
    import torch
    for w in ws:
        if len(w.shape) != 2 or not w.tile_cols:
            raise ValueError("weights must be 2-D and compressed with layout='mfma_tiles'")
    out_f, in_f = ws[0].shape
    dev = ws[0]._bufs["enc"].device
    if len(ws) == 2:
        if ws[1].shape != ws[0].shape or ws[1].decode_table_bits != ws[0].decode_table_bits:
            raise ValueError("gate and up must have the same shape and decode-table width")
        if ws[1]._bufs["enc"].device != dev:
            raise ValueError("gate and up must be on one device")
    if x.dtype != torch.bfloat16 or x.dim() == 0 or x.shape[-1] != in_f:
        raise ValueError("x must be a bfloat16 (..., in_features) tensor")
    x2, xs = _rows(x, in_f, "x")
    if x2.numel() and (x2.data_ptr() % 16 or xs % 8):
        raise ValueError("x's rows must be 16-byte aligned")
    act = _lib.ACTIVATIONS.get(activation if activation is not None else "none")
    if act is None:
        raise ValueError(f"activation must be one of {sorted(_lib.ACTIVATIONS)} or None")
    floats = (torch.bfloat16, torch.float32)
    for b in biases:
        if b is not None and (b.shape != (out_f,) or b.dtype not in floats or not b.is_contiguous()):
            raise ValueError("a bias must be contiguous bfloat16 or float32, one element per output feature")
    if len({b.dtype for b in biases if b is not None}) > 1:
        raise ValueError("both biases must have one dtype")
    shape = x.shape[:-1] + (out_f,)
    if residual is not None and (residual.shape != shape or residual.dtype not in floats):
        raise ValueError("residual must be a bfloat16 or float32 (..., out_features) tensor")
    if out is not None and (out.shape != shape or out.dtype not in floats):
        raise ValueError("out must be a bfloat16 or float32 (..., out_features) tensor")
    if out is not None and out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out_dtype must be out's dtype")
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    if out_dtype not in floats:
        raise ValueError("out_dtype must be bfloat16 or float32")
    _same_device(dev, x=x, residual=residual, out=out, bias=biases[0], up_bias=biases[-1])
    return dev, x2, xs, act, out_dtype


def _product_forward(ws, x, biases, activation, residual, out, out_dtype, stream, keep):
    """act(x W^T + b) [* (x Wu^T + bu)] + residual; with keep, also the sums
    before the activation, float32."""
    import torch
    dev, x2, xs, act, out_dtype = _check_product(ws, x, biases, activation, residual, out, out_dtype)
    out_f, in_f = ws[0].shape
    tokens = x2.shape[0]
    lib = _lib.load()
    with _on(dev, stream):
        if out is None:
            out = torch.empty(x.shape[:-1] + (out_f,), dtype=out_dtype, device=dev)
        pre = [torch.empty((tokens, out_f), dtype=torch.float32, device=dev) for _ in ws] if keep else []
        if out.numel() == 0:
            return out, pre
        e = _lib.Epilogue()
        y2, e.out_stride = _rows(out, out_f, "out")
        e.out, e.out_dtype, e.activation = y2.data_ptr(), _dtype(out, "out"), act
        for i, b in enumerate(biases):
            if b is not None:
                e.bias[i], e.bias_dtype = b.data_ptr(), _dtype(b, "bias")
        if residual is not None:
            r2, e.residual_stride = _rows(residual, out_f, "residual")
            e.residual, e.residual_dtype = r2.data_ptr(), _dtype(residual, "residual")
        for i, p in enumerate(pre):
            e.pre[i] = p.data_ptr()
        structs = [ctypes.byref(w._stream_struct) for w in ws]
        nbytes = lib.df11_epilogue_workspace(structs[0], structs[1] if len(ws) == 2 else None, tokens)
        work = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        st = [w._claim(stream) for w in ws][0]
        name = "df11_matmul_epilogue" if len(ws) == 1 else "df11_gated_matmul"
        _lib.check(getattr(lib, name)(*structs, x2.data_ptr(), xs, tokens, in_f, out_f, ctypes.byref(e),
                                      work.data_ptr(), nbytes, st), name)
    return out, pre


def _product_backward(ws, pre, dy, act, x_shape, want_x, biases):
    """(dx or None, the biases' gradients): biases[i] is a tensor like the
    bias whose gradient is wanted, or None."""
    import torch
    out_f, in_f = ws[0].shape
    dev = dy.device
    dy = _rowwise(dy)
    dy2, dys = _rows(dy, out_f, "dy")
    tokens = dy2.shape[0]
    lib = _lib.load()
    with _on(dev, None) as st:
        dx = torch.empty(x_shape, dtype=torch.bfloat16, device=dev) if want_x else None
        db = [None if b is None else torch.empty_like(b) for b in biases]
        g = _lib.ProductGrad()
        g.dy, g.dy_stride, g.dy_dtype, g.activation = dy2.data_ptr(), dys, _dtype(dy, "dy"), act
        for i, p in enumerate(pre):
            g.pre[i] = p.data_ptr()
        if dx is not None:
            g.dx, g.dx_stride, g.dx_dtype = dx.data_ptr(), in_f, _lib.BF16
        for i, b in enumerate(db):
            if b is not None:
                g.dbias[i], g.bias_dtype = b.data_ptr(), _dtype(b, "bias")
        structs = [ctypes.byref(w._stream_struct) for w in ws] + [None] * (2 - len(ws))
        nbytes = lib.df11_epilogue_grad_workspace(*structs, tokens, ctypes.byref(g)) if tokens else 0
        work = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        st = [w._claim(None) for w in ws][0]
        _lib.check(lib.df11_matmul_epilogue_grad(*structs, tokens, in_f, out_f, ctypes.byref(g), work.data_ptr(),
                                                 nbytes, st), "df11_matmul_epilogue_grad")
    return dx, db


def _product(ws, x, biases, activation, residual, out, out_dtype, stream):
    import torch
    inputs = (x, residual, *biases)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs):
        if out is not None or stream is not None:
            raise ValueError("out and stream are for calls without gradients")
        return _function("product").apply(x, residual, biases[0], biases[1] if len(ws) == 2 else None, ws, activation,
                                          out_dtype)
    return _product_forward(ws, x, biases, activation, residual, out, out_dtype, stream, False)[0]


def matmul_epilogue(w, x: "torch.Tensor", bias: Optional["torch.Tensor"] = None,  # noqa: F821
                    activation: Optional[str] = None, residual: Optional["torch.Tensor"] = None,  # noqa: F821
                    out: Optional["torch.Tensor"] = None, out_dtype=None, stream=None) -> "torch.Tensor":  # noqa: F821
    """act(x W^T + bias) + residual on the matrix cores with W compressed
    (df11_matmul_epilogue), for any number of tokens.

    w: a DF11Tensor compressed with layout="mfma_tiles"; x: bfloat16 (...,
    in_features), rows at one stride and 16-byte aligned; bias: bfloat16 or
    float32, one element per output feature; activation: None, "relu", "silu",
    "gelu" or "gelu_tanh"; residual: bfloat16 or float32 (..., out_features).
    Returns out, bfloat16 unless out or out_dtype says float32; out may be the
    residual itself.  Everything before out is float32, and the same call gives
    the same bits again.  Where x, bias or residual require a gradient the
    output carries it (then neither out nor stream may be given): the sums
    before an activation are kept for it in float32, and w itself is frozen."""
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
