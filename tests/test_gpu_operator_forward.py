"""A block's forward through the operators around the products, against the
same forward in float64 on the original weights.

Tolerance: every intermediate is rounded to BF16 once (half a step is 2^-8 of
its value at most), about ten times along the longest path, and each rounding
reaches the output through sums of many terms of random sign, where it stays
at most as large relative to the output's largest magnitude.  Ten of them
add to 10 * 2^-8 = 4% of it at most; the test allows 2%, as the fused forward's
test does against the resident weights (which rounds as often)."""

import math
import sys

import numpy as np
import pytest

from entropy_decoding_df11_amd import df11, workloads

pytestmark = pytest.mark.gpu

SHAPES = [("q_proj", (1024, 1024)), ("k_proj", (256, 1024)), ("v_proj", (256, 1024)), ("o_proj", (1024, 1024)),
          ("gate_proj", (2816, 1024)), ("up_proj", (2816, 1024)), ("down_proj", (1024, 2816))]


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    return torch


def _note(msg):
    print(f"[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def block(torch_cuda):
    torch = torch_cuda
    flat, views = workloads.gen_block(seed=11, shapes=SHAPES)
    parts = [(nm, flat[o:o + r * c].reshape(r, c)) for nm, o, (r, c) in views]
    blk = df11.compress_block(parts, codebook="per_weight", layout="mfma_tiles")
    resident = {nm: torch.from_numpy(a.astype(np.int16)).to("cuda").view(torch.bfloat16) for nm, a in parts}
    return blk, resident


def _x(torch, tokens, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(tokens, 1024, device="cuda", generator=g).bfloat16()


def _forward64(torch, x, w, eps=1e-5):
    import torch.nn.functional as F
    x = x.double()
    w = {k: v.double() for k, v in w.items()}

    def rms(h):
        return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps)

    h = rms(x)
    q, k, v = (F.linear(h, w[n]) for n in ("q_proj", "k_proj", "v_proj"))
    x = x + F.linear(q + (k * v).repeat_interleave(q.shape[-1] // k.shape[-1], dim=-1), w["o_proj"])
    h = rms(x)
    return x + F.linear(F.silu(F.linear(h, w["gate_proj"])) * F.linear(h, w["up_proj"]), w["down_proj"])


def _close(got, want, part):
    ok = float((got.double() - want).abs().max()) <= part * float(want.abs().max())
    assert ok


@pytest.mark.parametrize("tokens", [1, 2, 16, 33, 64, 65, 300])
def test_operator_forward(torch_cuda, block, tokens):
    torch = torch_cuda
    from entropy_decoding_df11_amd import runtime
    _note(f"operator forward {tokens}")
    blk, resident = block
    x = _x(torch, tokens, tokens)
    want = _forward64(torch, x, resident)
    got = runtime.operator_block_forward(x, blk)
    assert got.dtype == x.dtype and got.shape == x.shape
    _close(got, want, 0.02)
    _close(runtime.block_forward(x, resident, operators=True), want, 0.02)


@pytest.mark.parametrize("tokens", [1, 40, 130])
def test_operator_forward_gradient(torch_cuda, block, tokens):
    """The gradient of x through the whole block, against float64 autograd."""
    torch = torch_cuda
    from entropy_decoding_df11_amd import runtime
    _note(f"operator gradient {tokens}")
    blk, resident = block
    x, dy = _x(torch, tokens, 3), _x(torch, tokens, 4)
    a = x.clone().requires_grad_()
    got, = torch.autograd.grad(runtime.operator_block_forward(a, blk), a, dy)
    b = x.double().requires_grad_()
    want, = torch.autograd.grad(_forward64(torch, b, resident), b, dy.double())
    _close(got, want, 0.04)  # (forward and backward each round about ten times)


@pytest.mark.parametrize("tokens", [1, 24, 100])
def test_operator_forward_replays(torch_cuda, block, tokens):
    """Three blocks captured into a HIP graph and replayed on new inputs with
    eager forwards between."""
    torch = torch_cuda
    from entropy_decoding_df11_amd import runtime
    _note(f"operator graph {tokens}")
    blk, resident = block
    blocks = [blk, blk.clone(), blk]
    g = runtime.CapturedForward(lambda x: runtime.operator_model_forward(x, blocks), _x(torch, tokens, 1))
    for seed in (5, 6, 7):
        x = _x(torch, tokens, seed)
        got = g(x).clone()
        torch.cuda.synchronize()
        want = x
        for _ in blocks:
            want = _forward64(torch, want, resident)
        _close(got, want, 0.05)
        if tokens > 64:  # (the q, k, v product of fewer tokens adds with atomics)
            same = torch.equal(got, runtime.operator_model_forward(x, blocks))
            assert same


@pytest.mark.parametrize("tokens", [(2, 3), (2, 40), (3, 30), (70, 1), (5, 0), ()])
def test_operator_forward_of_any_leading_dimensions(torch_cuda, block, tokens):
    torch = torch_cuda
    from entropy_decoding_df11_amd import runtime
    _note(f"operator forward {tokens}")
    blk, resident = block
    x = _x(torch, math.prod(tokens), 3).view(*tokens, 1024)
    got = runtime.operator_block_forward(x, blk)
    assert got.shape == x.shape and got.dtype == x.dtype
    if x.numel():
        _close(got.view(-1, 1024), _forward64(torch, x.view(-1, 1024), resident), 0.02)
