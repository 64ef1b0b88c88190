"""GPU parity of the RMS norm with the residual's addition, forward and
backward, against its formula in float64.

Tolerances.  u = 2^-24 is half a step of float32, h half a step of the
output's type.  A sum of `cols` squares is added in chains of at most
D = cols / 1024 + 64 dependent float32 additions (at most 32 elements per
thread and 22 across threads for narrow rows, one per 1024 threads and turn
for wide ones), each product rounded once, so its relative error is at most
(D + 1) u and that of rstd at most half that plus 4 u for the division, the
addition of eps, the root and its reciprocal.  y multiplies three floats (2 u more) and is rounded
once (h).  The sum s is rounded exactly as torch adds two tensors."""

import sys

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    return torch


def _note(msg):
    print(f"[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


def _half_step(torch, t, v):
    """Half a step of type t at the magnitudes v (float64)."""
    f = torch.finfo(t)
    return torch.clamp(v.abs() * (f.eps / 2), min=f.smallest_normal * f.eps / 2)


def _depth(cols):
    return cols / 1024 + 64


def _forward64(torch, x, weight, residual, eps):
    s = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    d = s.double()
    rstd = (d.square().mean(-1, keepdim=True) + eps).rsqrt()
    h = d * rstd
    return s, h, rstd, h if weight is None else h * weight.double()


def _check_y(torch, y, y64, cols):
    bound = _half_step(torch, y.dtype, y64) + y64.abs() * 1.01 * U * ((_depth(cols) + 1) / 2 + 6)
    err = (y.double() - y64).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


def _inputs(torch, rows, cols, kind, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    mk = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return mk(rows, cols).to(kind), (3 * mk(rows, cols)).to(kind), 1 + 0.3 * mk(cols), mk(rows, cols).to(kind), \
        mk(rows, cols).to(kind)


# widths: one column, fewer than a vector, every thread shape at whole
# vectors and at odd ones, beyond what the threads hold; rows that leave
# part of a block empty
SHAPES = [(1, 1), (3, 7), (5, 64), (1, 4096), (130, 512), (9, 1023), (4, 2048), (7, 4104), (3, 5003), (2, 16384),
          (3, 16392), (2, 33001), (1, 70000), (2500, 72)]


@pytest.mark.parametrize("kind", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_forward_and_backward(torch_cuda, rows, cols, kind):
    torch = torch_cuda
    from entropy_decoding_df11_amd import df11
    dt = getattr(torch, kind)
    _note(f"norm {rows}x{cols} {kind}")
    x, r, w, dy, ds = _inputs(torch, rows, cols, dt)
    for residual in (None, r):
        for weight in (None, w.to(dt), w):
            s, h, rstd, y64 = _forward64(torch, x, weight, residual, 1e-5)
            got = df11.rms_norm(x, weight=weight, residual=residual, eps=1e-5)
            y = got if residual is None else got[0]
            _check_y(torch, y, y64, cols)
            if residual is not None:
                assert torch.equal(got[1], s)
            # backward, with and without the sum's own gradient
            leaves = [t.clone().requires_grad_() for t in (x, weight, residual) if t is not None]
            it = iter(leaves)
            args = {"x": next(it), "weight": None if weight is None else next(it),
                    "residual": None if residual is None else next(it)}
            out = df11.rms_norm(**args, eps=1e-5)
            if residual is None:
                assert torch.equal(out, y)
                tops, downs, dsum = (out,), (dy,), torch.zeros_like(dy)
            else:
                assert torch.equal(out[0], y) and torch.equal(out[1], s)
                tops, downs, dsum = out, (dy, ds), ds
            grads = torch.autograd.grad(tops, leaves, downs)
            d = dy.double() if weight is None else dy.double() * weight.double()
            mean = (d * h).mean(-1, keepdim=True)
            core = rstd * (d - h * mean)
            dx64 = core + dsum.double()
            size = rstd * (d.abs() + h.abs() * (d * h).abs().mean(-1, keepdim=True) * 2)
            bound = _half_step(torch, dt, dx64) + 1.01 * U * (size * (_depth(cols) + 16) + dsum.double().abs() + dx64.abs())
            err = (grads[0].double() - dx64).abs()
            assert bool((err <= bound).all()), float((err / bound).max())
            if residual is not None:
                assert torch.equal(grads[-1], grads[0])
            if weight is not None:
                dw64 = (dy.double() * h).sum(0)
                wb = _half_step(torch, weight.dtype, dw64) + 1.01 * U * (dy.double() * h).abs().sum(0) * (
                    rows + _depth(cols) / 2 + 8)
                err = (grads[1].double() - dw64).abs()
                assert grads[1].dtype == weight.dtype and bool((err <= wb).all()), float((err / wb).max())


def test_norm_gradient_against_differences(torch_cuda):
    """The gradient along a direction against a central difference of the
    formula in float64."""
    torch = torch_cuda
    from entropy_decoding_df11_amd import df11
    _note("norm differences")
    x, r, w, dy, ds = _inputs(torch, 6, 96, torch.float32, seed=4)
    leaves = [t.clone().requires_grad_() for t in (x, w, r)]
    y, s = df11.rms_norm(leaves[0], weight=leaves[1], residual=leaves[2], eps=1e-3)
    grads = torch.autograd.grad((y, s), leaves, (dy, ds))
    g = torch.Generator(device="cuda")
    g.manual_seed(9)

    def value(dx, dw, dr):
        t = x.double() + dx + r.double() + dr
        n = t * (t.square().mean(-1, keepdim=True) + 1e-3).rsqrt() * (w.double() + dw)
        return (n * dy.double()).sum() + (t * ds.double()).sum()

    for _ in range(3):
        v = [torch.randn(t.shape, device="cuda", generator=g, dtype=torch.float64) for t in leaves]
        e = 1e-5
        diff = (value(*[e * t for t in v]) - value(*[-e * t for t in v])) / (2 * e)
        got = sum((a.double() * b).sum() for a, b in zip(grads, v))
        # e^2 / 6 of the third derivative and float32's rounding of ~1700 terms of size ~1
        assert abs(float(diff - got)) <= 1e-3 * max(1.0, abs(float(diff)))


def test_norm_strides_aliases_and_streams(torch_cuda):
    torch = torch_cuda
    from entropy_decoding_df11_amd import df11
    _note("norm strides")
    for dt in (torch.bfloat16, torch.float32):
        wide = torch.randn(40, 3, 1000, device="cuda").to(dt)
        x = wide[:, 1, :777]  # odd base, rows 3000 elements apart
        res = torch.randn(777, device="cuda").to(dt).expand(40, 777)  # one row for all
        w = torch.randn(778, device="cuda").to(dt)[1:]  # not 16-byte aligned
        y, s = df11.rms_norm(x, weight=w, residual=res)
        s64, _, _, y64 = _forward64(torch, x, w, res, 1e-5)
        assert torch.equal(s, s64)
        _check_y(torch, y, y64, 777)
        # outputs with their own strides leave what lies between their rows alone
        out = torch.full((40, 1000), 7.0, device="cuda", dtype=dt)
        sums = torch.full((40, 800), 9.0, device="cuda", dtype=dt)
        got = df11.rms_norm(x, weight=w, residual=res, out=out[:, 3:780], sum_out=sums[:, :777])
        assert torch.equal(got[0], y) and torch.equal(got[1], s)
        assert bool((out[:, :3] == 7).all()) and bool((out[:, 780:] == 7).all()) and bool((sums[:, 777:] == 9).all())
        # in place: the sum on the residual stream, the norm on x
        xi, ri = x.contiguous(), res.contiguous()
        got = df11.rms_norm(xi, weight=w, residual=ri, out=xi, sum_out=ri)
        assert torch.equal(xi, y) and torch.equal(ri, s)
        # a side stream, three dimensions, an empty batch, one dimension
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y3 = df11.rms_norm(wide, stream=side)
        side.synchronize()
        assert y3.shape == wide.shape
        _check_y(torch, y3, _forward64(torch, wide, None, None, 1e-5)[3], 1000)
        assert df11.rms_norm(wide[:0]).shape == (0, 3, 1000)
        assert torch.equal(df11.rms_norm(wide[0, 0]), y3[0, 0])
        # no rows: the weight's gradient is zero
        w0 = torch.ones(1000, device="cuda", dtype=dt, requires_grad=True)
        df11.rms_norm(wide[:0].clone(), weight=w0).sum().backward()
        assert bool((w0.grad == 0).all())


def test_norm_extremes_stay_in_their_rows(torch_cuda):
    torch = torch_cuda
    from entropy_decoding_df11_amd import df11
    _note("norm extremes")
    x = torch.randn(6, 4096, device="cuda")
    x[1, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4] = 0
    for dt in (torch.bfloat16, torch.float16, torch.float32):
        y = df11.rms_norm(x.to(dt))
        assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[1, 5])) and bool((y[4] == 0).all())
        _check_y(torch, y[[0, 2, 5]], _forward64(torch, x.to(dt)[[0, 2, 5]], None, None, 1e-5)[3], 4096)


def test_norm_repeats_and_replays(torch_cuda):
    """The same call gives the same bits, and a captured call replays them on
    new inputs."""
    torch = torch_cuda
    from entropy_decoding_df11_amd import df11
    _note("norm graph")
    x, r, w, dy, ds = _inputs(torch, 300, 4096, torch.bfloat16, seed=2)
    w = w.bfloat16()

    def step():
        a, b, c = (t.detach().requires_grad_() for t in (x, w, r))
        y, s = df11.rms_norm(a, weight=b, residual=c)
        return (y, s) + torch.autograd.grad((y, s), (a, b, c), (dy, ds))

    first = step()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    del first
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (5, 6, 7):
        nx, nr, nw, ny, ns = _inputs(torch, 300, 4096, torch.bfloat16, seed=seed)
        for t, n in ((x, nx), (r, nr), (w, nw.bfloat16()), (dy, ny), (ds, ns)):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


@pytest.mark.parametrize("kind", ["bfloat16", "float32"])
def test_norm_unaligned_rows_leave_their_surroundings(torch_cuda, kind):
    """Widths around every number of threads a row takes, whole vectors and
    one element off, at bases and strides aligned to one element only: the
    values, and the elements between the rows, which stay as they were."""
    torch = torch_cuda
    from entropy_decoding_df11_amd import df11
    dt = getattr(torch, kind)
    vec = 16 // dt.itemsize
    for threads in (1, 16, 32, 64, 128, 256, 512, 1024, 2048, 4096):
        for cols in (threads * vec - 1, threads * vec, threads * vec + 1):
            _note(f"norm unaligned {kind} {cols}")
            base = torch.randn(3, cols + 5, device="cuda").to(dt)
            x, r = base[:, 1:cols + 1], base.roll(7, 1)[:, 3:cols + 3]
            w = (1 + 0.3 * torch.randn(cols + 1, device="cuda")).to(dt)[1:]
            y64 = _forward64(torch, x, w, r, 1e-5)[3]
            s64 = (x.float() + r.float()).to(dt)
            out, sums = (torch.full((3, cols + 3), v, device="cuda", dtype=dt) for v in (7.0, 9.0))
            y, s = df11.rms_norm(x, weight=w, residual=r, out=out[:, 1:cols + 1], sum_out=sums[:, 2:cols + 2])
            _check_y(torch, y, y64, cols)
            assert torch.equal(s, s64)
            assert bool((out[:, :1] == 7).all()) and bool((out[:, cols + 1:] == 7).all())
            assert bool((sums[:, :2] == 9).all()) and bool((sums[:, cols + 2:] == 9).all())
            # the same in place, in rows that touch
            xi, ri = x.contiguous(), r.contiguous()
            df11.rms_norm(xi, weight=w, residual=ri, out=ri, sum_out=xi)
            assert torch.equal(ri, y) and torch.equal(xi, s)


@pytest.mark.parametrize("rows,cols", [(1, 100), (37, 128), (700, 200), (3000, 520), (700, 1030), (1100, 4096),
                                       (600, 8200), (300, 33000)])
def test_norm_weight_gradient_over_many_rows(torch_cuda, rows, cols):
    """The weight's gradient where row groups of one block, blocks and rows
    beyond them each add up."""
    torch = torch_cuda
    from entropy_decoding_df11_amd import df11
    _note(f"norm weight gradient {rows}x{cols}")
    for dt in (torch.bfloat16, torch.float32):
        x, _, w, dy, _ = _inputs(torch, rows, cols, dt, seed=rows)
        leaves = x.clone().requires_grad_(), w.clone().requires_grad_()
        dw = torch.autograd.grad(df11.rms_norm(leaves[0], weight=leaves[1]), leaves, dy)[1]
        h = _forward64(torch, x, w, None, 1e-5)[1]
        t = dy.double() * h
        # each product rounded and added at most once per row, rstd's own error
        bound = _half_step(torch, torch.float32, t.sum(0)) + 1.01 * U * t.abs().sum(0) * (rows + _depth(cols) / 2 + 8)
        assert bool(((dw.double() - t.sum(0)).abs() <= bound).all())


@pytest.mark.parametrize("cols", [(1 << 26) + 70, 1 << 28])
def test_norm_weight_gradient_of_the_widest_rows(torch_cuda, cols):
    """More columns than one launch has threads for.  x is 1 or -1: a wave's
    sum of squares is a whole number up to 2^24 and exact, the 16 waves' sum is
    rounded at most 16 times, so rstd is within 2^-20 of 1, and dweight = dy x
    rstd rounds to dy x, which is a BF16 number itself."""
    torch = torch_cuda
    from entropy_decoding_df11_amd import df11
    _note(f"norm gradient of {cols} columns")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = (torch.randint(0, 2, (1, cols), device="cuda", generator=g, dtype=torch.int8) * 2 - 1).bfloat16()
    dy = torch.randn(1, cols, device="cuda", generator=g, dtype=torch.bfloat16)
    w = torch.ones(cols, device="cuda", dtype=torch.bfloat16).requires_grad_()
    dw, = torch.autograd.grad(df11.rms_norm(x, weight=w, eps=0.0), w, dy)
    same = torch.equal(dw, (dy * x)[0])
    assert same
    dw0, = torch.autograd.grad(df11.rms_norm(x[:0], weight=w), w, dy[:0])
    zero = not bool(dw0.any())
    assert zero


def test_norm_of_more_than_32_bits_of_bytes(torch_cuda):
    """600000 rows of 4096, 4.9 GB, forward and backward: the rows whose
    elements pass 2^31 and whose bytes pass 2^31 and 2^32, and others, against
    the same rows by themselves (a row's result depends on the row alone)."""
    torch = torch_cuda
    from entropy_decoding_df11_amd import df11
    _note("norm past 32 bits")
    rows, cols = 600_000, 4096
    x, r, dy, ds = (torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16).normal_() for _ in range(4))
    at = sorted({0, 1, rows - 1} | {limit // cols + k for limit in (1 << 30, 1 << 31) for k in (-1, 0, 1)}
                | {rows * k // 7 for k in range(1, 7)})
    at = torch.tensor(at, device="cuda")

    def both(x, r, dy, ds):
        a = x.detach().requires_grad_()
        y, s = df11.rms_norm(a, residual=r)
        return y.detach(), s.detach(), torch.autograd.grad((y, s), a, (dy, ds))[0]

    want = both(x[at], r[at], dy[at], ds[at])
    assert all(torch.equal(a[at], b) for a, b in zip(both(x, r, dy, ds), want))
