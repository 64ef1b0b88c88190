"""The softmax cross entropy through a compressed output head, and its gradient.

    loss = linear_cross_entropy(head, x, targets)     # mean over the tokens

What training below a frozen head, a text's perplexity and the scores of drafted
tokens need: the head's product, the softmax over the vocabulary and the
targets' logarithms in one operator (the C ABI's df11_cross_entropy), which
keeps no logits.  As in operators.py it runs on torch's current stream, or on
the stream given, and its calls may overlap and may be captured into graphs.
"""

from __future__ import annotations

from typing import Optional

from . import _lib, operators
from .operators import _no_tangents, _ptr, _rows, _run, _same_device, _stream

_Loss = None

_REDUCTIONS = ("none", "sum", "mean")


def _check(w, x, targets, vocab, reduction):
    torch = operators.torch
    if len(w.shape) != 2 or not w.tile_cols or not w.shape[0]:
        raise ValueError("the head must be 2-D, not empty, and compressed with layout='mfma_tiles'")
    rows, cols = w.shape
    if x.dtype != torch.bfloat16 or x.dim() == 0 or x.shape[-1] != cols:
        raise ValueError("x must be a bfloat16 (..., in_features) tensor")
    if x.numel() >= 1 << 32:
        raise ValueError("tokens times in_features must be below 2^32")
    if targets.dtype != torch.int64 or targets.shape != x.shape[:-1]:
        raise ValueError("targets must be int64, one for each token")
    if vocab is None:
        vocab = rows
    if not 1 <= vocab <= rows:
        raise ValueError("vocab must be 1 to the head's rows")
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction must be one of {_REDUCTIONS}")
    dev = w._bufs["enc"].device
    _same_device(dev, "x", x)
    _same_device(dev, "targets", targets)
    return dev, vocab


def _launch_loss(dev, w, x, targets, vocab, ignore_index, reduction, with_grad):
    """(each token's loss, their sum or mean, their number, the gradient), the
    last three None where they are not wanted."""
    torch = operators.torch
    rows, cols = w.shape
    x2, xs = _rows(x, cols, "x")
    x_ptr, tokens = x2.data_ptr(), x2.shape[0]
    if x_ptr % 16 or xs % 8:
        raise ValueError("x's rows must be 16-byte aligned")
    targets = targets.contiguous()
    loss = torch.empty(targets.shape, dtype=torch.float32, device=dev)
    total = None if reduction == "none" else torch.empty((), dtype=torch.float32, device=dev)
    count = torch.empty((), dtype=torch.float32, device=dev) if with_grad and reduction == "mean" else None
    grad = torch.empty((tokens, cols), dtype=torch.float32, device=dev) if with_grad else None
    lib = _lib.load()
    nbytes = lib.df11_cross_entropy_workspace(w._stream_struct, tokens, with_grad)
    work = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    l = _lib.Loss(targets.data_ptr(), loss.data_ptr(), _ptr(total), _ptr(count), _ptr(grad),  # noqa: E741
                  ignore_index, vocab, reduction == "mean")
    status = lib.df11_cross_entropy(w._stream_struct, x_ptr, xs, tokens, cols, rows, l, work.data_ptr(), nbytes,
                                    _stream(dev))
    if status:
        _lib.check(status, "df11_cross_entropy")
    return loss, total, count, grad


def _launch_loss_grad(dev, grad, dy, count, x_shape):
    torch = operators.torch
    dx = torch.empty(x_shape, dtype=torch.bfloat16, device=dev)
    dy = dy.reshape(-1)
    tokens, cols = grad.shape
    status = _lib.load().df11_cross_entropy_grad(grad.data_ptr(), dy.data_ptr(), dy.stride(0) if dy.numel() > 1 else 0,
                                                 _ptr(count), tokens, cols, dx.data_ptr(), cols, _lib.BF16, _stream(dev))
    if status:
        _lib.check(status, "df11_cross_entropy_grad")
    return (dx,)


def linear_cross_entropy(w, x: "torch.Tensor", targets: "torch.Tensor", vocab: Optional[int] = None,  # noqa: F821
                         ignore_index: int = -100, reduction: str = "mean", stream=None) -> "torch.Tensor":  # noqa: F821
    """-log softmax(x W^T)[target] with W compressed, logits and softmax in
    float32 and neither stored (df11_cross_entropy).

    w: a DF11Tensor compressed with layout="mfma_tiles", (classes, in_features);
    x: bfloat16 (..., in_features), rows at one stride and 16-byte aligned, fewer
    than 2^32 elements and, with a gradient, 2^24 tokens; targets: int64, one for each token; vocab: the classes
    that count, where w's last rows are padding (None: all rows).  A token whose
    target is ignore_index counts nowhere, one whose target is no class otherwise
    gives NaN.  Returns float32: with reduction "none" the losses, of targets'
    shape, with "sum" and "mean" (over the tokens not ignored; NaN if there are
    none) one number.  Where x requires a gradient the loss carries it (then
    stream may not be given): it is computed with the loss, since both need the
    same exponentials, and kept in float32, rounded once to bfloat16 with the
    loss's own gradient; w itself is frozen.  The same call gives the same bits
    again."""
    if operators.torch is None:
        operators._import_torch()
    torch = operators.torch
    dev, vocab = _check(w, x, targets, vocab, reduction)
    if operators._forward_ad._current_level >= 0:
        _no_tangents(x)
    if x.requires_grad and torch.is_grad_enabled():
        if stream is not None:
            raise ValueError("stream is for calls without gradients")
        if _Loss is None:
            _make_function(torch)
        return _Loss.apply(x, w, targets, vocab, ignore_index, reduction)
    loss, total = _run(dev, stream, _launch_loss, w, x, targets, vocab, ignore_index, reduction, False)[:2]
    return loss if total is None else total


def _make_function(torch) -> None:
    global _Loss
    from torch.autograd.function import once_differentiable

    class Loss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, targets, vocab, ignore_index, reduction):
            loss, total, count, grad = _run(x.device, None, _launch_loss, w, x, targets, vocab, ignore_index, reduction,
                                            True)
            ctx.save_for_backward(grad, count)
            ctx.x_shape = x.shape
            return loss if total is None else total

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            grad, count = ctx.saved_tensors
            dx, = _run(dy.device, None, _launch_loss_grad, grad, dy, count, ctx.x_shape)
            return dx, None, None, None, None, None

    _Loss = Loss
