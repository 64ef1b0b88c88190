"""Operators around the products of a transformer block, on the GPU.

The framework keeps a block's weights compressed and multiplies by them; this
module has what a forward computes between one product and the next (the C
ABI's operators in include/df11.h), each differentiable: under torch's
autograd they give the gradients of the activations, the biases, the residual
and the norm's weight.  (The compressed weights are frozen: they have none.)

    y = rms_norm(x, weight)                       # norm
    y, s = rms_norm(x, weight, residual=r)        # s = x + r, y = norm of s

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
    if cols > 1 and v.stride(1) != 1:
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

        _FUNCTIONS["norm"] = Norm
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
