"""GPU parity of the compressed products with an epilogue (matmul_epilogue,
gated_matmul) against their formulas in float64 on the original weights.

Tolerances.  u = 2^-24 and h half a step of the output's type.  Every product
of two BF16 is exact in float32; a sum of C of them is added in float32 in
some order, so z is off by at most dz = 1.01 C u sum |x w|, plus u |z| for
the bias (its addition rounds once).  The activations have a slope of at most
1.13 and are computed to 8 u of their value (expf and erfcf to 2 ulp, a
quotient and two products); in a gated product each factor's error meets the
other's size; the residual's addition rounds once and the output once."""

import sys

import numpy as np
import pytest

from entropy_decoding_df11_amd import df11, workloads

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SLOPE = 1.13  # the largest slope of any activation here (GELU's)


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    return torch


def _note(msg):
    print(f"[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


_WEIGHTS = {}


def _weight(rows, cols, kind="normal", seed=0):
    """(compressed weight, its float64 values on the GPU), kept for the module."""
    import torch
    key = (rows, cols, kind, seed)
    if key not in _WEIGHTS:
        rng = np.random.default_rng(seed)
        n = rows * cols
        bits = np.zeros(n, np.uint16) if kind == "zeros" else workloads.gen_stress(seed=seed, n=n) if kind == "stress" \
            else workloads.f32_to_bf16_bits(rng.standard_normal(n) * 0.05)
        w = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16).view(rows, cols).double()
        _WEIGHTS[key] = (df11.compress(bits, shape=(rows, cols), layout="mfma_tiles"), w)
    return _WEIGHTS[key]


def _act64(torch, name, z):
    import torch.nn.functional as F
    return {None: lambda v: v, "none": lambda v: v, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[name](z)


def _half_step(torch, t, v):
    f = torch.finfo(t)
    return torch.clamp(v.abs() * (f.eps / 2), min=f.smallest_normal * f.eps / 2)


def _linear64(x, w64, bias):
    x64 = x.double().reshape(-1, w64.shape[1])
    z = x64 @ w64.t()
    dz = 1.01 * w64.shape[1] * U * (x64.abs() @ w64.abs().t())
    if bias is not None:
        z = z + bias.double()
        dz = dz + U * (z.abs() + dz)
    return z, dz


def _expected(torch, x, ws, biases, act, residual, out_dtype):
    """(value, bound) in float64."""
    z, dz = _linear64(x, ws[0], biases[0])
    y = _act64(torch, act, z)
    dy = SLOPE * dz + 8 * U * (y.abs() + dz)
    if len(ws) == 2:
        z1, dz1 = _linear64(x, ws[1], biases[1])
        dy = dy * (z1.abs() + dz1) + (y.abs() + dy) * dz1
        y = y * z1
        dy = dy + U * y.abs()
    if residual is not None:
        y = y + residual.double().reshape(y.shape)
        dy = dy + U * (y.abs() + dy)
    return y, dy + _half_step(torch, out_dtype, y.abs() + dy)


def _assert_close(y, y64, bound):
    err = (y.double().reshape(y64.shape) - y64).abs()
    ok, worst = bool((err <= bound).all()), float((err / bound).max())
    assert ok, worst


def _x(torch, tokens, cols, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(tokens, cols, device="cuda", generator=g).bfloat16()


def _side(torch, shape, dt, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=g).to(dt)


# one k-step; odd k-steps; panels smaller than a group, so that a range's
# group slots skip panels; panels over many workgroups; long codes; one-bit
# codes (groups of 2048 chunks)
SHAPES = [(64, 32, "normal"), (192, 96, "normal"), (4096, 32, "normal"), (1024, 64, "zeros"), (128, 4096, "normal"),
          (64, 14336, "stress"), (640, 1056, "normal"), (64, 8192, "zeros")]
TOKENS = [1, 2, 8, 9, 16, 17, 33, 64, 65, 130, 300]


def _slope64(torch, name, z):
    z = z.detach().clone().requires_grad_()
    return torch.autograd.grad(_act64(torch, name, z).sum(), z)[0]


@pytest.mark.parametrize("rows,cols,kind", SHAPES)
@pytest.mark.parametrize("tokens", TOKENS)
def test_product(torch_cuda, rows, cols, kind, tokens):
    torch = torch_cuda
    _note(f"product {tokens} x {cols} -> {rows} {kind}")
    w, w64 = _weight(rows, cols, kind)
    u, u64 = _weight(rows, cols, kind, 1)
    x = _x(torch, tokens, cols, seed=tokens)
    for i, (act, bdt, rdt, odt) in enumerate([
            (None, None, None, torch.float32), ("gelu", torch.bfloat16, None, torch.bfloat16),
            ("silu", None, torch.bfloat16, torch.bfloat16), ("gelu_tanh", torch.float32, torch.float32, torch.float32),
            ("relu", torch.bfloat16, torch.float32, torch.bfloat16)]):
        bias = None if bdt is None else _side(torch, (rows,), bdt, 3)
        bias2 = None if bdt is None or i == 3 else _side(torch, (rows,), bdt, 4)
        res = None if rdt is None else _side(torch, (tokens, rows), rdt, 5)
        y = df11.matmul_epilogue(w, x, bias=bias, activation=act, residual=res, out_dtype=odt)
        assert y.dtype == odt and y.shape == (tokens, rows)
        _assert_close(y, *_expected(torch, x, (w64,), (bias,), act, res, odt))
        assert torch.equal(y, df11.matmul_epilogue(w, x, bias=bias, activation=act, residual=res, out_dtype=odt))
        h = df11.gated_matmul(w, u, x, gate_bias=bias, up_bias=bias2, activation=act, residual=res, out_dtype=odt)
        _assert_close(h, *_expected(torch, x, (w64, u64), (bias, bias2), act, res, odt))
        assert torch.equal(h, df11.gated_matmul(w, u, x, gate_bias=bias, up_bias=bias2, activation=act, residual=res,
                                                out_dtype=odt))


@pytest.mark.parametrize("rows,cols", [(4096, 4096), (1024, 8192)])
def test_product_long_streams(torch_cuda, rows, cols):
    """Long streams, and every launch shape: the schedule on and off, a capped
    grid."""
    torch = torch_cuda
    w, w64 = _weight(rows, cols)
    u, u64 = _weight(rows, cols, "normal", 1)
    for tokens in (1, 5, 8, 16, 40, 64, 100):
        _note(f"long product {tokens} x {cols} -> {rows}")
        x = _x(torch, tokens, cols, seed=tokens)
        for t in (w, u):
            t.set_dynamic_schedule(True)
            t.set_max_workgroups(0)
        y = df11.matmul_epilogue(w, x, activation="silu", out_dtype=torch.float32)
        _assert_close(y, *_expected(torch, x, (w64,), (None,), "silu", None, torch.float32))
        h = df11.gated_matmul(w, u, x, out_dtype=torch.float32)
        want = _expected(torch, x, (w64, u64), (None, None), "silu", None, torch.float32)
        _assert_close(h, *want)
        # the same stream as gate and up
        _assert_close(df11.gated_matmul(w, w, x, out_dtype=torch.float32),
                      *_expected(torch, x, (w64, w64), (None, None), "silu", None, torch.float32))
        for dynamic, cap in ((False, 0), (True, 37), (True, 3)):
            for t in (w, u):
                t.set_dynamic_schedule(dynamic)
                t.set_max_workgroups(cap)
            _assert_close(df11.gated_matmul(w, u, x, out_dtype=torch.float32), *want)
            assert torch.equal(df11.gated_matmul(w, u, x), df11.gated_matmul(w, u, x))
    for t in (w, u):
        t.set_dynamic_schedule(True)
        t.set_max_workgroups(0)


@pytest.mark.parametrize("bits", [10, 12])
def test_product_table_widths(torch_cuda, bits):
    torch = torch_cuda
    rng = np.random.default_rng(8)
    raw = workloads.f32_to_bf16_bits(rng.standard_normal(256 * 512) * 0.05)
    w64 = torch.from_numpy(raw.view(np.int16)).cuda().view(torch.bfloat16).view(256, 512).double()
    w = df11.compress(raw, shape=(256, 512), layout="mfma_tiles", decode_table_bits=bits)
    for tokens in (1, 20, 50, 90):
        _note(f"product table {bits} {tokens}")
        x = _x(torch, tokens, 512)
        for table in (True, False):
            w.use_decode_table(table)
            _assert_close(df11.matmul_epilogue(w, x), *_expected(torch, x, (w64,), (None,), None, None, torch.bfloat16))
            _assert_close(df11.gated_matmul(w, w, x),
                          *_expected(torch, x, (w64, w64), (None, None), "silu", None, torch.bfloat16))


@pytest.mark.parametrize("tokens", [1, 7, 40, 150])
def test_product_strides_and_places(torch_cuda, tokens):
    torch = torch_cuda
    _note(f"product strides {tokens}")
    w, w64 = _weight(640, 1056)
    u, u64 = _weight(640, 1056, "normal", 1)
    big = _x(torch, tokens * 3, 1056 + 40, seed=1).view(tokens, 3, 1096)
    x = big[:, 1, 16:1072]  # 16-byte aligned rows, 3288 elements apart
    res = _side(torch, (640,), torch.bfloat16, 2).expand(tokens, 640)  # one row for all
    y = torch.full((tokens, 700), 5.0, device="cuda", dtype=torch.bfloat16)
    got = df11.matmul_epilogue(w, x, activation="gelu", residual=res, out=y[:, 3:643])
    _assert_close(got, *_expected(torch, x, (w64,), (None,), "gelu", res, torch.bfloat16))
    assert bool((y[:, :3] == 5).all()) and bool((y[:, 643:] == 5).all())
    # the residual stream updated in place, on a side stream
    r = res.clone().contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h = df11.gated_matmul(w, u, x, residual=r, out=r, stream=side)
    side.synchronize()
    assert h is r
    _assert_close(r, *_expected(torch, x, (w64, u64), (None, None), "silu", res, torch.bfloat16))
    torch.cuda.current_stream().wait_stream(side)
    # three dimensions, one dimension, no tokens
    x3 = _x(torch, tokens * 2, 1056).view(2, tokens, 1056)
    y3 = df11.matmul_epilogue(w, x3)
    assert y3.shape == (2, tokens, 640)
    _assert_close(y3, *_expected(torch, x3, (w64,), (None,), None, None, torch.bfloat16))
    assert df11.matmul_epilogue(w, x3[0, 0]).shape == (640,)
    assert df11.gated_matmul(w, u, x3[:, :0]).shape == (2, 0, 640)


@pytest.mark.parametrize("tokens", [3, 40, 100])
def test_product_nonfinite_tokens_stay_alone(torch_cuda, tokens):
    torch = torch_cuda
    _note(f"product nonfinite {tokens}")
    w, w64 = _weight(640, 1056)
    u, u64 = _weight(640, 1056, "normal", 1)
    x = _x(torch, tokens, 1056, seed=6)
    x[1, 3] = float("inf")
    x[tokens - 1, 1000] = float("nan")
    keep = [t for t in range(tokens) if t not in (1, tokens - 1)]
    for y, want in ((df11.matmul_epilogue(w, x), _expected(torch, x, (w64,), (None,), None, None, torch.bfloat16)),
                    (df11.gated_matmul(w, u, x),
                     _expected(torch, x, (w64, u64), (None, None), "silu", None, torch.bfloat16))):
        _assert_close(y[keep], want[0][keep], want[1][keep])
        assert not bool(torch.isfinite(y[tokens - 1]).any()) and bool(torch.isnan(y[tokens - 1]).all())
    assert not bool(torch.isfinite(df11.matmul_epilogue(w, x)[1]).any())


@pytest.mark.parametrize("tokens", [1, 24, 64, 200])
def test_product_replays(torch_cuda, tokens):
    """Two captured graphs of the same weights, replayed on new inputs with
    eager calls between them."""
    torch = torch_cuda
    _note(f"product graph {tokens}")
    w, _ = _weight(4096, 4096)
    u, _ = _weight(4096, 4096, "normal", 1)
    x = _x(torch, tokens, 4096)

    def step():
        h = df11.gated_matmul(w, u, x)
        return h, df11.matmul_epilogue(w, h, activation="gelu", residual=x)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = step()
        graphs.append((g, held))
    for seed in (1, 2, 3):
        x.copy_(_x(torch, tokens, 4096, seed=seed))
        for g, held in graphs:
            g.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in held]
            assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_one_step_panels(torch_cuda):
    """A matrix of 32 columns has one k-step per panel: its product and its
    decompression must still tell its panels apart."""
    torch = torch_cuda
    _note("32 columns")
    w, w64 = _weight(4096, 32)
    same = torch.equal(w.decompress().double(), w64)
    assert same
    for tokens in (1, 20, 70):
        x = _x(torch, tokens, 32)
        z, dz = _linear64(x, w64, None)
        _assert_close(w.matmul(x), z, dz)


# Gradients.  dz = dy act'(z) (times the other factor of a gated product) is
# off by the error of z times the slope's own slope (at most 1 here, 1.13 for
# the gated factor act), by 16 u of its value for computing it, and, for dx
# alone, by 2^-9 of its value for its rounding to BF16 (2^-8 / 2 is half a
# step: h = 2^-8 relative to the value at most); dx adds R (2 R gated) products
# in float32 and is rounded once.
@pytest.mark.parametrize("rows,cols,kind", [(64, 32, "normal"), (192, 96, "normal"), (128, 4096, "normal"),
                                            (64, 1024, "stress"), (640, 1056, "normal"), (2048, 320, "normal")])
@pytest.mark.parametrize("tokens", [1, 17, 64, 129, 300])
def test_product_gradients(torch_cuda, rows, cols, kind, tokens):
    torch = torch_cuda
    _note(f"gradient {tokens} x {cols} -> {rows} {kind}")
    w, w64 = _weight(rows, cols, kind)
    u, u64 = _weight(rows, cols, kind, 1)
    x = _x(torch, tokens, cols, seed=tokens)
    for gated in (False, True):
        for act, bdt, odt in (("none", None, torch.bfloat16), ("none", torch.bfloat16, torch.float32),
                              ("gelu", torch.bfloat16, torch.bfloat16), ("silu", torch.float32, torch.float32),
                              ("gelu_tanh", None, torch.bfloat16)):
            ws = (w64, u64) if gated else (w64,)
            biases = [None if bdt is None else _side(torch, (rows,), bdt, 3 + i) for i in range(len(ws))]
            res = _side(torch, (tokens, rows), torch.float32, 5)
            dy = _side(torch, (tokens, rows), odt, 6)
            leaves = [t.clone().requires_grad_() for t in (x, res, *biases) if t is not None]
            bl = leaves[2:] if bdt is not None else [None] * len(ws)
            if gated:
                y = df11.gated_matmul(w, u, leaves[0], gate_bias=bl[0], up_bias=bl[1], activation=act,
                                      residual=leaves[1], out_dtype=odt)
            else:
                y = df11.matmul_epilogue(w, leaves[0], bias=bl[0], activation=act, residual=leaves[1], out_dtype=odt)
            _assert_close(y.detach(), *_expected(torch, x, ws, biases, act, res, odt))
            grads = torch.autograd.grad(y, leaves, dy)
            assert torch.equal(grads[1], dy.float())
            zs = [_linear64(x, m, b) for m, b in zip(ws, biases)]
            z, dz = zs[0]
            d64 = dy.double()
            s64, a64 = _slope64(torch, act, z), _act64(torch, act, z)
            curve = 0.0 if act == "none" else 1.0
            if gated:
                z1, dz1 = zs[1]
                ds = [d64 * z1 * s64, d64 * a64]
                err = [d64.abs() * (dz1 * (s64.abs() + curve * dz) + z1.abs() * curve * dz) + 16 * U * (
                    d64 * z1).abs() * (s64.abs() + z.abs() + 1), d64.abs() * SLOPE * dz + 16 * U * ds[1].abs()]
            else:
                ds = [d64 * s64]
                err = [d64.abs() * curve * dz + 16 * U * d64.abs() * (s64.abs() + z.abs() + 1)]
            dx64 = sum(d @ m for d, m in zip(ds, ws))
            size = sum(d.abs() @ m.abs() for d, m in zip(ds, ws))
            bound = sum((e + 2.0 ** -8 * (d.abs() + e)) @ m.abs() for d, e, m in zip(ds, err, ws))
            bound = bound + 1.01 * len(ws) * rows * U * (size + bound)
            _assert_close(grads[0], dx64, bound + _half_step(torch, torch.bfloat16, dx64.abs() + bound))
            for i, b in enumerate(biases):
                if b is not None:
                    b64 = ds[i].sum(0)
                    eb = err[i].sum(0) + 1.01 * (tokens + 8) * U * (ds[i].abs().sum(0) + err[i].sum(0))
                    assert grads[2 + i].dtype == b.dtype
                    _assert_close(grads[2 + i], b64, eb + _half_step(torch, b.dtype, b64.abs() + eb))


# Whole rounds of large tiles with a rest of small ones, large tiles alone,
# small ones alone, splits along K of either; odd k-steps; outputs that end
# inside a tile.
@pytest.mark.parametrize("tokens,rows,cols", [(2000, 10304, 416), (1030, 6208, 2080), (2300, 4096, 320),
                                              (4100, 192, 4096), (1500, 4096, 4096), (70, 4096, 4096)])
def test_dense_plans(torch_cuda, tokens, rows, cols):
    torch = torch_cuda
    _note(f"dense {tokens} x {cols} -> {rows}")
    w, w64 = _weight(rows, cols)
    u, u64 = _weight(rows, cols, "normal", 1)
    x = _x(torch, tokens, cols, seed=7)
    res = _side(torch, (tokens, rows), torch.bfloat16, 5)
    y = df11.matmul_epilogue(w, x, activation="gelu", residual=res)
    _assert_close(y, *_expected(torch, x, (w64,), (None,), "gelu", res, torch.bfloat16))
    del y
    xg = x.clone().requires_grad_()
    h = df11.gated_matmul(w, u, xg, activation="none", out_dtype=torch.float32)
    want, bound = _expected(torch, x, (w64, u64), (None, None), "none", None, torch.float32)
    _assert_close(h.detach(), want, bound)
    del want, bound
    dy = _side(torch, (tokens, rows), torch.float32, 6)
    dx, = torch.autograd.grad(h, xg, dy)
    del h
    (z0, e0), (z1, e1) = _linear64(x, w64, None), _linear64(x, u64, None)
    d = dy.double()
    dx64 = (d * z1) @ w64 + (d * z0) @ u64
    size = (d * z1).abs() @ w64.abs() + (d * z0).abs() @ u64.abs()
    slack = (d.abs() * e1) @ w64.abs() + (d.abs() * e0) @ u64.abs()
    bound = slack + (2.0 ** -8 + 16 * U + 1.01 * 2 * rows * U) * (size + slack)
    _assert_close(dx, dx64, bound + _half_step(torch, torch.bfloat16, dx64.abs() + bound))


def test_product_gradient_against_differences(torch_cuda):
    """dx along a direction against a central difference of the formula in float64."""
    torch = torch_cuda
    _note("gradient differences")
    w, w64 = _weight(640, 1056)
    u, u64 = _weight(640, 1056, "normal", 1)
    x = _x(torch, 20, 1056, seed=3)
    b = _side(torch, (640,), torch.float32, 4)
    dy = _side(torch, (20, 640), torch.float32, 6)
    for act in ("silu", "gelu", "gelu_tanh", "none"):
        leaves = [x.clone().requires_grad_(), b.clone().requires_grad_()]
        y = df11.gated_matmul(w, u, leaves[0], gate_bias=leaves[1], activation=act, out_dtype=torch.float32)
        grads = torch.autograd.grad(y, leaves, dy)
        v = _side(torch, (20, 1056), torch.float64, 8)
        vb = _side(torch, (640,), torch.float64, 9)

        def value(e):
            x64 = x.double() + e * v
            return (_act64(torch, act, x64 @ w64.t() + b.double() + e * vb) * (x64 @ u64.t()) * dy.double()).sum()

        diff = (value(1e-5) - value(-1e-5)) / 2e-5
        got = (grads[0].double() * v).sum() + (grads[1].double() * vb).sum()
        # dz and dx are rounded to BF16 (2^-8 each, at most): twice that of the sum of sizes, over the
        # root of the 20 * 1056 independent roundings, five times over
        size = (grads[0].double().abs() * v.abs()).sum()
        assert abs(float(diff - got)) <= 5 * 2 * 2.0 ** -8 * float(size) / (20 * 1056) ** 0.5 + 1e-6 * float(size)


def test_product_gradient_parts(torch_cuda):
    """Only what is asked for, expanded and strided gradients, no tokens."""
    torch = torch_cuda
    _note("gradient parts")
    w, w64 = _weight(640, 1056)
    x = _x(torch, 40, 1056, seed=3)
    b = _side(torch, (640,), torch.bfloat16, 4).requires_grad_()
    df11.matmul_epilogue(w, x, bias=b, activation="relu", out_dtype=torch.float32).sum().backward()
    want = (x.double() @ w64.t() + b.detach().double() > 0).double().sum(0)
    assert bool(((b.grad.double() - want).abs() <= want * 2.0 ** -8 + 1).all())
    xg = x.clone().requires_grad_()
    y = df11.matmul_epilogue(w, xg)
    wide = _side(torch, (40, 1280), torch.bfloat16, 6)
    for dy in (wide[:, 320:960], wide[:, 3:643], wide[:1, :640].expand(40, 640), wide[:, ::2]):
        g, = torch.autograd.grad(y, xg, dy, retain_graph=True)
        g2, = torch.autograd.grad(y, xg, dy.contiguous(), retain_graph=True)
        assert torch.equal(g, g2)
    b0 = b.detach().clone().requires_grad_()
    x0 = x[:0].clone().requires_grad_()
    df11.matmul_epilogue(w, x0, bias=b0, activation="silu").sum().backward()
    assert bool((b0.grad == 0).all()) and x0.grad.shape == (0, 1056)


def test_training_step_replays(torch_cuda):
    """Norm, gated product and down product, forward and backward, captured
    and replayed on new inputs with eager steps between."""
    torch = torch_cuda
    _note("training graph")
    w, _ = _weight(4096, 4096)
    u, _ = _weight(4096, 4096, "normal", 1)
    nw = torch.ones(4096, device="cuda", dtype=torch.bfloat16)
    x = _x(torch, 100, 4096)
    dy = _x(torch, 100, 4096, seed=50)

    def step():
        a, n = x.detach().requires_grad_(), nw.detach().requires_grad_()
        h = df11.gated_matmul(w, u, df11.rms_norm(a, weight=n))
        y = df11.matmul_epilogue(u, h, residual=a)
        return (y.detach(),) + torch.autograd.grad(y, (a, n), dy)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (1, 2, 3):
        x.copy_(_x(torch, 100, 4096, seed=seed))
        dy.copy_(_x(torch, 100, 4096, seed=seed + 60))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


@pytest.mark.parametrize("tokens", [4, 32, 33, 200])
def test_products_on_two_streams_at_once(torch_cuda, tokens):
    """The same weights multiplied on two streams without a wait between."""
    torch = torch_cuda
    _note(f"two streams {tokens}")
    w, w64 = _weight(4096, 4096)
    u, u64 = _weight(4096, 4096, "normal", 1)
    xs = [_x(torch, tokens, 4096, seed=s) for s in range(6)]
    want = [df11.gated_matmul(w, u, x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [df11.gated_matmul(w, u, x, stream=streams[i % 2]) for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for st in streams:
        torch.cuda.current_stream().wait_stream(st)


@pytest.mark.parametrize("tokens", [5, 80])
def test_gradients_of_shared_and_broadcast_inputs(torch_cuda, tokens):
    """One bias for both projections, one residual row for every token, x as
    its own residual, the same weights as gate and up; the bias changed in
    place between the passes."""
    torch = torch_cuda
    _note(f"shared gradients {tokens}")
    w, w64 = _weight(4096, 4096)
    x = _x(torch, tokens, 4096, seed=1).requires_grad_()
    b = _side(torch, (4096,), torch.float32, 2).requires_grad_()
    r = _side(torch, (1, 4096), torch.float32, 3).requires_grad_()
    dy = _side(torch, (tokens, 4096), torch.float32, 4)
    y = df11.gated_matmul(w, w, x, gate_bias=b, up_bias=b, residual=r.expand(tokens, 4096), out_dtype=torch.float32)
    with torch.no_grad():
        b += 1  # (the backward pass needs the sums, not the bias)
    dx, db, dr = torch.autograd.grad(y, (x, b, r), dy)
    x64, b64, d64 = x.detach().double().requires_grad_(), (b.detach().double() - 1).requires_grad_(), dy.double()
    z = x64 @ w64.t() + b64
    ex, eb = torch.autograd.grad(torch.nn.functional.silu(z) * z, (x64, b64), d64)
    # (norm-wise: dz rounded to BF16, 2^-8, and dx rounded once more)
    for got, want, part in ((dx, ex, 2.0 ** -7), (db, eb, 1e-4), (dr, d64.sum(0, keepdim=True), 1e-5)):
        off = float((got.double() - want).norm() / want.norm())
        assert got.shape == want.shape and off <= part
    s, = torch.autograd.grad(df11.matmul_epilogue(w, x, residual=x), x, dy.bfloat16())
    p, = torch.autograd.grad(df11.matmul_epilogue(w, x), x, dy.bfloat16())
    off = float((s.double() - p.double() - dy.bfloat16().double()).norm() / s.double().norm())
    assert off <= 2.0 ** -7


def test_replays_on_two_streams_at_once(torch_cuda):
    """Two graphs of the same weights, forward and backward, and eager calls,
    on three streams without a wait between."""
    torch = torch_cuda
    _note("graphs on two streams")
    w, _ = _weight(4096, 4096)
    u, _ = _weight(4096, 4096, "normal", 1)
    dy = _x(torch, 100, 4096, seed=9)

    def step(x):
        a = x.detach().requires_grad_()
        y = df11.matmul_epilogue(u, df11.gated_matmul(w, u, a), residual=a)
        return y.detach(), torch.autograd.grad(y, a, dy)[0]

    xs = [_x(torch, 100, 4096, seed=s) for s in range(3)]
    want = [step(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    graphs = []
    for x in xs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = step(x)
        graphs.append((g, held))
    torch.cuda.synchronize()
    for _ in range(10):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(streams[2]):
            last = step(xs[2])
    torch.cuda.synchronize()
    for got, expected in zip([held for _, held in graphs] + [last], want):
        assert all(torch.equal(a, b) for a, b in zip(got, expected))


@pytest.mark.parametrize("shape", [(5, 1024), (2, 40, 1024), (0, 1024)])
def test_weights_without_outputs(torch_cuda, shape):
    """A weight of no rows gives no outputs, and a gradient of zero."""
    torch = torch_cuda
    _note(f"no outputs {shape}")
    w = df11.compress(np.zeros(0, np.uint16), shape=(0, 1024), layout="mfma_tiles")
    b = torch.zeros(0, device="cuda", requires_grad=True)
    held = torch.full((4, 2, 40, 1024), float("nan"), device="cuda")  # (freed memory is not zero)
    del held
    for op in (lambda x: df11.matmul_epilogue(w, x, bias=b, activation="gelu"),
               lambda x: df11.gated_matmul(w, w, x, gate_bias=b)):
        x = torch.randn(shape, device="cuda").bfloat16().requires_grad_()
        y = op(x)
        assert y.shape == shape[:-1] + (0,)
        dx, db = torch.autograd.grad(y, (x, b), torch.empty_like(y))
        assert dx.shape == x.shape and bool((dx == 0).all()) and db.shape == (0,)


@pytest.mark.parametrize("rows", [4096, 12544])
@pytest.mark.parametrize("tokens", [4, 40, 300])
def test_products_leave_the_work_counters_alone(torch_cuda, tokens, rows):
    """The weights' work counters (those of their dynamic schedule) may be in
    use by another thread's launch while a product or its backward pass runs:
    whatever they hold, the result is the same, and they hold it afterwards."""
    torch = torch_cuda
    _note(f"work counters {tokens} {rows}")
    w, _ = _weight(rows, 4096)
    u, _ = _weight(rows, 4096, "normal", 1)
    x, dy = _x(torch, tokens, 4096, seed=2), _x(torch, tokens, rows, seed=3)

    def step():
        a = x.detach().requires_grad_()
        y = df11.matmul_epilogue(u, a, residual=df11.gated_matmul(w, u, a))
        return y.detach(), torch.autograd.grad(y, a, dy)[0]

    want = step()
    counters = [t._schedule for t in (w, u)]
    assert all(t._stream_struct.schedule == c.data_ptr() and not bool(c.any()) for t, c in zip((w, u), counters))
    for c in counters:
        c.fill_(3)
    got = step()
    left = [bool((c == 3).all()) for c in counters]
    for c in counters:
        c.zero_()
    assert all(left) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_products_from_threads_at_once(torch_cuda):
    """The same weights in two threads with a stream each, forward and
    backward, beside decompressions of them in a third."""
    torch = torch_cuda
    import threading
    _note("threads")
    w, _ = _weight(12544, 4096)
    u, _ = _weight(12544, 4096, "normal", 1)
    xs, dy = [_x(torch, 100, 4096, seed=s) for s in range(2)], _x(torch, 100, 12544, seed=9)

    def step(x):
        a = x.detach().requires_grad_()
        y = df11.matmul_epilogue(u, a, residual=df11.gated_matmul(w, u, a))
        return y.detach(), torch.autograd.grad(y, a, dy)[0]

    want = [step(x) for x in xs]
    flat = w.decompress()
    torch.cuda.synchronize()
    same = [[], [], []]

    def products(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [step(xs[i]) for _ in range(20)]
            torch.cuda.current_stream().synchronize()
            same[i] = [torch.equal(a, b) for g in got for a, b in zip(g, want[i])]

    def decodes():
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [w.decompress() for _ in range(20)]
            torch.cuda.current_stream().synchronize()
            same[2] = [torch.equal(g.view(torch.int16), flat.view(torch.int16)) for g in got]

    threads = [threading.Thread(target=products, args=(i,)) for i in range(2)] + [threading.Thread(target=decodes)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [len(s) for s in same] == [40, 40, 20] and all(all(s) for s in same)


@pytest.mark.parametrize("tokens", [3, 40])
def test_gate_and_up_that_share_a_buffer(torch_cuda, tokens):
    """up = -gate: the same exponents, so the same encoded stream, beside signs
    of its own."""
    torch = torch_cuda
    _note(f"shared buffer {tokens}")
    w, w64 = _weight(640, 1056)
    u = w.clone()
    u._bufs["sm"] ^= 0x80
    u._bufs["enc"] = w._bufs["enc"]
    u._stream_struct.enc = w._bufs["enc"].data_ptr()
    assert torch.equal(u.decompress().double(), -w64)
    x = _x(torch, tokens, 1056, seed=4)
    a = x.clone().requires_grad_()
    h = df11.gated_matmul(w, u, a, activation="none", out_dtype=torch.float32)
    _assert_close(h.detach(), *_expected(torch, x, (w64, -w64), (None, None), "none", None, torch.float32))
    dy = _side(torch, (tokens, 640), torch.float32, 6)
    dx, = torch.autograd.grad(h, a, dy)
    z = x.double() @ w64.t()
    want = -2 * (dy.double() * z) @ w64
    # (norm-wise: dz rounded to BF16, 2^-8, and dx rounded once more)
    assert float((dx.double() - want).norm()) <= 2.0 ** -7 * float(want.norm())


def test_outputs_given_are_known_to_autograd(torch_cuda):
    """A tensor that a graph has kept and an operator then overwrites fails the
    backward pass, as it does under torch's own operators."""
    torch = torch_cuda
    _note("versions")
    w, _ = _weight(640, 1056)
    x = torch.randn(3, 1056, device="cuda").bfloat16()
    r = torch.randn(3, 640, device="cuda").bfloat16()
    for write in (lambda t: df11.rms_norm(t, out=t), lambda t: df11.rms_norm(t, residual=t.clone(), sum_out=t),
                  lambda t: df11.matmul_epilogue(w, x, residual=t, out=t),
                  lambda t: df11.gated_matmul(w, w, x, out=t)):
        kept = r.clone()
        y = torch.ones_like(kept).requires_grad_() * kept
        write(kept)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def test_inputs_freed_before_their_stream_runs(torch_cuda):
    """Inputs of a call on a busy stream, freed at once: their memory is not
    handed out again before the stream has read them, nor an output's while
    the caller's stream may still read it."""
    torch = torch_cuda
    _note("freed inputs")
    w, _ = _weight(4096, 4096)
    u, _ = _weight(4096, 4096, "normal", 1)
    side = torch.cuda.Stream()

    def inputs():
        return _x(torch, 5000, 4096, seed=1), _x(torch, 5000, 4096, seed=2)

    def once(op):
        x, r = inputs()
        want = op(x, r, None)
        del x, r
        torch.cuda.synchronize()
        x, r = inputs()
        at = {x.data_ptr(), r.data_ptr()}
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = op(x, r, side)
        del x, r
        fresh = [torch.full((5000, 4096), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        apart = not at & {t.data_ptr() for t in fresh} or side.query()  # (or the stream is through already)
        torch.cuda.synchronize()
        same = torch.equal(got, want)
        assert apart and same

    once(lambda x, r, s: df11.rms_norm(x, residual=r, stream=s)[0])
    once(lambda x, r, s: df11.matmul_epilogue(w, x, residual=r, stream=s))
    once(lambda x, r, s: df11.gated_matmul(w, u, x, residual=r, stream=s))
    x, _ = inputs()
    side.wait_stream(torch.cuda.current_stream())
    y = df11.rms_norm(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    side.synchronize()
    torch.cuda._sleep(20_000_000)
    kept, at = y.clone(), y.data_ptr()
    del y
    with torch.cuda.stream(side):
        fresh = torch.full((5000, 4096), float("nan"), device="cuda", dtype=torch.bfloat16)
    apart = fresh.data_ptr() != at or torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    same = torch.equal(kept, df11.rms_norm(x))
    assert apart and same


# As test_product_gradients, but for the kink: where z lies within its own
# error dz of 0 the slope may be that of the other side, an error of |dy| (times
# the other factor of a gated product) in that element's dz; elsewhere the slope
# is exact.
@pytest.mark.parametrize("rows,cols,kind", [(64, 32, "normal"), (192, 96, "normal"), (64, 1024, "stress"),
                                            (640, 1056, "normal")])
@pytest.mark.parametrize("tokens", [1, 17, 64, 129, 300])
def test_relu_gradients(torch_cuda, rows, cols, kind, tokens):
    torch = torch_cuda
    _note(f"relu gradient {tokens} x {cols} -> {rows} {kind}")
    w, w64 = _weight(rows, cols, kind)
    u, u64 = _weight(rows, cols, kind, 1)
    x = _x(torch, tokens, cols, seed=tokens)
    for gated in (False, True):
        for bdt, odt in ((None, torch.bfloat16), (torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16)):
            ws = (w64, u64) if gated else (w64,)
            biases = [None if bdt is None else _side(torch, (rows,), bdt, 3 + i) for i in range(len(ws))]
            dy = _side(torch, (tokens, rows), odt, 6)
            leaves = [t.clone().requires_grad_() for t in (x, *biases) if t is not None]
            bl = leaves[1:] if bdt is not None else [None] * len(ws)
            if gated:
                y = df11.gated_matmul(w, u, leaves[0], gate_bias=bl[0], up_bias=bl[1], activation="relu", out_dtype=odt)
            else:
                y = df11.matmul_epilogue(w, leaves[0], bias=bl[0], activation="relu", out_dtype=odt)
            _assert_close(y.detach(), *_expected(torch, x, ws, biases, "relu", None, odt))
            grads = torch.autograd.grad(y, leaves, dy)
            zs = [_linear64(x, m, b) for m, b in zip(ws, biases)]
            z, dz = zs[0]
            d64, on = dy.double(), (z > 0).double()
            kink = (z.abs() <= dz).double()
            if gated:
                z1, dz1 = zs[1]
                ds = [d64 * z1 * on, d64 * z.relu()]
                err = [d64.abs() * (kink * (z1.abs() + dz1) + on * dz1), d64.abs() * (on + kink) * dz]
            else:
                ds = [d64 * on]
                err = [d64.abs() * kink]
            err = [e + 16 * U * d.abs() for e, d in zip(err, ds)]
            dx64 = sum(d @ m for d, m in zip(ds, ws))
            size = sum(d.abs() @ m.abs() for d, m in zip(ds, ws))
            bound = sum((e + 2.0 ** -8 * (d.abs() + e)) @ m.abs() for d, e, m in zip(ds, err, ws))
            bound = bound + 1.01 * len(ws) * rows * U * (size + bound)
            _assert_close(grads[0], dx64, bound + _half_step(torch, torch.bfloat16, dx64.abs() + bound))
            for i, b in enumerate(biases):
                if b is not None:
                    b64 = ds[i].sum(0)
                    eb = err[i].sum(0) + 1.01 * (tokens + 8) * U * (ds[i].abs().sum(0) + err[i].sum(0))
                    assert grads[1 + i].dtype == b.dtype
                    _assert_close(grads[1 + i], b64, eb + _half_step(torch, b.dtype, b64.abs() + eb))
            # (the kink must not swallow the test: hardly any element lies in it)
            assert float(kink.mean()) <= 0.01


def test_long_weights_replay_on_two_streams_at_once(torch_cuda):
    """Gate and up of 51 M weights each, whose decodes take counters from the
    call's workspace: two graphs and eager calls on three streams without a
    wait between, again and again."""
    torch = torch_cuda
    _note("graphs of long weights")
    w, _ = _weight(12544, 4096)
    u, _ = _weight(12544, 4096, "normal", 1)
    dy = _x(torch, 50, 12544, seed=9)

    def step(x):
        a = x.detach().requires_grad_()
        y = df11.gated_matmul(w, u, a)
        return y.detach(), torch.autograd.grad(y, a, dy)[0]

    xs = [_x(torch, 50, 4096, seed=s) for s in range(3)]
    want = [step(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    graphs = []
    for x in xs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = step(x)
        graphs.append((g, held))
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(streams[2]):
            last = step(xs[2])
        torch.cuda.synchronize()
        for got, expected in zip([held for _, held in graphs] + [last], want):
            assert all(torch.equal(a, b) for a, b in zip(got, expected))


def _some_rows(torch, rows, cols):
    """A few rows of a long tensor: its ends, where its elements pass 2^31, its
    BF16 bytes 2^31 and 2^32, and some between."""
    at = {0, 1, rows - 1, rows - 2}
    for limit in (1 << 31, 1 << 30, 1 << 32):
        at |= {t for t in (limit // cols - 1, limit // cols, limit // cols + 1) if t < rows}
    at |= {rows * k // 7 for k in range(1, 7)}
    return torch.tensor(sorted(at), device="cuda")


@pytest.mark.parametrize("gated", [False, True])
def test_outputs_past_32_bits(torch_cuda, gated):
    """Nearly 2^32 outputs, forward and backward: a million tokens of 4096
    features, 8 GB of them, compared where offsets pass 32 bits."""
    torch = torch_cuda
    _note(f"past 32 bits, gated {gated}")
    tokens, rows, cols, act = 1_048_000, 4096, 32, "none" if gated else "silu"
    w, w64 = _weight(rows, cols)
    u, u64 = _weight(rows, cols, "normal", 1)
    ws = (w64, u64) if gated else (w64,)
    x, dy = _x(torch, tokens, cols, seed=1), _x(torch, tokens, rows, seed=2)
    a = x.detach().requires_grad_()
    y = df11.gated_matmul(w, u, a, activation=act) if gated else df11.matmul_epilogue(w, a, activation=act)
    at = _some_rows(torch, tokens, rows)
    few = x[at]
    _assert_close(y.detach()[at], *_expected(torch, few, ws, (None,) * len(ws), act, None, torch.bfloat16))
    dx, = torch.autograd.grad(y, a, dy)
    del y
    # (bounds as in test_product_gradients)
    zs = [_linear64(few, m, None) for m in ws]
    d64, (z, dz) = dy[at].double(), zs[0]
    if gated:
        z1, dz1 = zs[1]
        ds, err = [d64 * z1, d64 * z], [d64.abs() * dz1, d64.abs() * dz]
    else:
        s64 = _slope64(torch, act, z)
        ds, err = [d64 * s64], [d64.abs() * dz + 16 * U * d64.abs() * (s64.abs() + z.abs() + 1)]
    err = [e + 16 * U * d.abs() for e, d in zip(err, ds)]
    want = sum(d @ m for d, m in zip(ds, ws))
    size = sum(d.abs() @ m.abs() for d, m in zip(ds, ws))
    bound = sum((e + 2.0 ** -8 * (d.abs() + e)) @ m.abs() for d, e, m in zip(ds, err, ws))
    bound = bound + 1.01 * len(ws) * rows * U * (size + bound)
    _assert_close(dx[at], want, bound + _half_step(torch, torch.bfloat16, want.abs() + bound))


@pytest.mark.parametrize("tokens", [20, 300])
def test_strides_past_32_bits(torch_cuda, tokens):
    """The longest row strides of x, and outputs and residuals whose last row
    lies past 2^32 elements."""
    torch = torch_cuda
    _note(f"long strides {tokens}")
    w, w64 = _weight(640, 1056)
    u, u64 = _weight(640, 1056, "normal", 1)
    base = _x(torch, tokens, 1056, seed=1)
    x = torch.empty(tokens << 22, device="cuda", dtype=torch.bfloat16).as_strided((tokens, 1056), (1 << 22, 1))
    x.copy_(base)
    stride = (1 << 32) // (tokens - 2)
    r = torch.empty(stride * tokens, device="cuda", dtype=torch.bfloat16).as_strided((tokens, 640), (stride, 1))
    y = torch.empty(stride * tokens, device="cuda", dtype=torch.bfloat16).as_strided((tokens, 640), (stride, 1))
    r.copy_(_side(torch, (tokens, 640), torch.bfloat16, 2))
    df11.matmul_epilogue(w, x, activation="gelu", residual=r, out=y)
    _assert_close(y, *_expected(torch, base, (w64,), (None,), "gelu", r, torch.bfloat16))
    df11.gated_matmul(w, u, x, residual=y, out=r)
    _assert_close(r, *_expected(torch, base, (w64, u64), (None, None), "silu", y, torch.bfloat16))
    a = x.detach().requires_grad_()
    out = df11.matmul_epilogue(w, a)
    y.copy_(_side(torch, (tokens, 640), torch.bfloat16, 3))
    g, = torch.autograd.grad(out, a, y, retain_graph=True)
    g2, = torch.autograd.grad(out, a, y.contiguous())
    assert torch.equal(g, g2)
    # the norm's rows, in place
    n, m = df11.rms_norm(y.contiguous(), residual=r.contiguous())
    df11.rms_norm(y, residual=r, out=y, sum_out=r)
    assert torch.equal(y, n) and torch.equal(r, m)
