"""Argument checks of the operators around the products, through the C ABI
and the binding.  Every refusal comes before any launch, so these run without
a GPU; the addresses are never read."""

import os

import pytest

from entropy_decoding_df11_amd import _lib

INVALID, SMALL, TOO_LARGE = -1, -5, -7


def _lib_or_skip():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libdf11.so is not built")
    return _lib.load()


# (far apart, 16-byte aligned)
A, B, C, D, E, F, G = (0x10000000 * (i + 1) for i in range(7))


def _norm(**k):
    a = dict(x=A, xs=64, r=None, rs=0, w=None, wt=0, rows=4, cols=64, t=0, eps=1e-5, sum=None, ss=0, y=B, ys=64,
             rstd=None)
    a.update(k)
    return _lib_or_skip().df11_rms_norm(a["x"], a["xs"], a["r"], a["rs"], a["w"], a["wt"], a["rows"], a["cols"], a["t"],
                                        a["eps"], a["sum"], a["ss"], a["y"], a["ys"], a["rstd"], None)


@pytest.mark.parametrize("bad", [
    dict(t=3), dict(cols=0), dict(rows=(1 << 30) + 1), dict(cols=(1 << 30) + 1), dict(eps=-1.0),
    dict(eps=float("nan")), dict(x=None), dict(y=None), dict(x=A + 1), dict(y=B + 1), dict(t=2, x=A + 2),
    dict(w=C, wt=1), dict(w=C, wt=7), dict(w=C, wt=2, t=1, x=A + 1), dict(w=C + 2, wt=2), dict(rstd=C + 2),
    dict(sum=C, ss=64),                                    # a sum without a residual
    dict(ys=63), dict(r=C, sum=D, ss=63),                  # output rows that overlap
    dict(y=A + 2), dict(y=A, ys=80), dict(r=C, rs=64, y=C + 128), dict(r=C, rs=64, sum=B, ss=64),
    dict(w=B, wt=0), dict(rstd=B), dict(rstd=A), dict(r=C, rs=64, rstd=C), dict(w=C, rstd=C),
])
def test_norm_refuses(bad):
    assert _norm(**bad) == INVALID


def test_norm_takes_no_rows():
    assert _norm(rows=0) == 0
    assert _norm(rows=0, x=None, y=None) == 0


def _grad(**k):
    a = dict(s=A, ss=64, w=None, wt=0, rstd=B, dy=C, dys=64, ds=None, dss=0, rows=4, cols=64, t=0, dx=D, dxs=64,
             dw=None, ws=None, wb=0)
    a.update(k)
    return _lib_or_skip().df11_rms_norm_grad(a["s"], a["ss"], a["w"], a["wt"], a["rstd"], a["dy"], a["dys"], a["ds"],
                                             a["dss"], a["rows"], a["cols"], a["t"], a["dx"], a["dxs"], a["dw"],
                                             a["ws"], a["wb"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(t=9), INVALID), (dict(cols=0), INVALID), (dict(rstd=None), INVALID), (dict(dy=None), INVALID),
    (dict(dx=None), INVALID), (dict(s=None), INVALID), (dict(dxs=60), INVALID), (dict(dw=E), INVALID),
    (dict(w=E, dw=F, ws=None), INVALID), (dict(w=E, dw=F, ws=G + 4, wb=1 << 20), INVALID),
    (dict(w=E, dw=F, ws=G, wb=16), SMALL), (dict(dx=A + 2), INVALID), (dict(dx=B), INVALID),
    (dict(w=E, dw=E, ws=G, wb=1 << 20), INVALID), (dict(w=E, dw=A, ws=G, wb=1 << 20), INVALID),
    (dict(w=E, dw=F, ws=D, wb=1 << 20), INVALID), (dict(w=E, dw=F, ws=C, wb=1 << 20), INVALID),
])
def test_norm_grad_refuses(bad, status):
    assert _grad(**bad) == status


def test_norm_binding_refuses():
    import torch
    from entropy_decoding_df11_amd import df11
    x = torch.zeros(4, 8)
    for bad in (dict(x=x), dict(x=torch.zeros(4, 0)), dict(x=x.double()), dict(x=torch.zeros(())),
                dict(x=x, residual=torch.zeros(4, 7)), dict(x=x, residual=x.half()),
                dict(x=x, weight=torch.zeros(7)), dict(x=x, weight=torch.zeros(8).half()),
                dict(x=x.half(), weight=torch.zeros(8).bfloat16()), dict(x=x.t()), dict(x=x, sum_out=x),
                dict(x=x, out=torch.zeros(4, 8).half()), dict(x=x.clone().requires_grad_(), out=x)):
        with pytest.raises(ValueError):
            df11.rms_norm(**bad)


def _stream(rows=128, cols=64, bits=11, at=0x200000000, tile=True):
    """A device stream whose header is sound and whose addresses are never read."""
    import numpy as np
    from entropy_decoding_df11_amd import df11, workloads
    w = workloads.f32_to_bf16_bits(np.random.default_rng(0).standard_normal(rows * cols) * 0.02)
    host = df11.encode(w)
    s = _lib.DeviceStream()
    s.h = host.header
    for i, name in enumerate(("enc", "sm", "gaps", "out_pos", "luts", "code_lengths", "decode_table")):
        setattr(s, name, at + i * 0x1000000)
    s.decode_table_bits = bits
    s.tile_cols = cols if tile else 0
    return s


def _product(gated=False, **k):
    import ctypes
    lib = _lib_or_skip()
    a = dict(w=_stream(), u=_stream(at=0x300000000), x=A, xs=64, t=4, inf=64, outf=128, ws=G, wb=0, bias=(None, None),
             bt=0, res=None, rs=128, rt=0, out=B, os=128, ot=0, pre=(None, None), act=0, e=True)
    a.update(k)
    e = _lib.Epilogue()
    for i in range(2):
        e.bias[i], e.pre[i] = a["bias"][i], a["pre"][i]
    e.residual, e.residual_stride, e.residual_dtype = a["res"], a["rs"], a["rt"]
    e.out, e.out_stride, e.out_dtype = a["out"], a["os"], a["ot"]
    e.bias_dtype, e.activation = a["bt"], a["act"]
    ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
    tail = (a["x"], a["xs"], a["t"], a["inf"], a["outf"], ctypes.byref(e) if a["e"] else None, a["ws"], a["wb"], None)
    if gated:
        return lib.df11_gated_matmul(ref(a["w"]), ref(a["u"]), *tail)
    return lib.df11_matmul_epilogue(ref(a["w"]), *tail)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bad", [
    dict(w=None), dict(inf=32), dict(outf=64), dict(inf=60), dict(outf=100), dict(e=False), dict(act=5),
    dict(ot=1), dict(ot=3), dict(res=C, rt=1), dict(bias=(C, None), bt=1), dict(bias=(C, None), bt=9),
    dict(x=None), dict(x=A + 8), dict(xs=68), dict(xs=(1 << 22) + 8), dict(out=None), dict(out=B + 1),
    dict(ot=2, out=B + 2), dict(os=127), dict(os=(1 << 31) + 1), dict(res=C + 1), dict(rt=2, res=C + 2),
    dict(rs=(1 << 31) + 1, res=C), dict(bias=(C + 1, None)), dict(pre=(C + 2, D)), dict(pre=(C + 4, D)), dict(out=A), dict(out=A + 128),
    dict(res=B + 2), dict(res=B, rs=256), dict(res=B, rt=2), dict(bias=(B, None)), dict(pre=(B, D)), dict(pre=(A, D)),
    dict(out=0x200000000), dict(out=0x201000000), dict(ws=G + 128),
])
def test_product_refuses(gated, bad):
    assert _product(gated, **bad) == INVALID


def test_product_refuses_streams():
    assert _product(w=_stream(tile=False)) == INVALID       # not in tile order
    assert _product(bias=(None, C)) == INVALID              # a second bias without a second matrix
    assert _product(pre=(C, D)) == INVALID
    assert _product(True, pre=(C, None)) == INVALID         # both or neither
    assert _product(True, u=None) == INVALID
    assert _product(True, u=_stream(rows=64, at=0x300000000)) == INVALID
    assert _product(True, u=_stream(bits=10, at=0x300000000)) == INVALID
    broken = _stream()
    broken.h.n_groups += 1
    assert _product(w=broken) == -6
    assert _product(t=1 << 26) == TOO_LARGE


def test_product_takes_nothing():
    assert _product(t=0, x=None, out=None, ws=None) == 0
    assert _product(True, t=0) == 0
    import ctypes
    lib = _lib_or_skip()
    s, plain = _stream(), _stream(tile=False)
    assert lib.df11_epilogue_workspace(None, None, 4) == 0
    assert lib.df11_epilogue_workspace(ctypes.byref(s), None, 0) == 0
    assert lib.df11_epilogue_workspace(ctypes.byref(plain), None, 4) == 0


class _FakeWeight:
    shape, tile_cols, decode_table_bits = (128, 64), 64, 11

    def __init__(self, **k):
        import torch
        self._bufs = {"enc": torch.zeros(4)}
        self.__dict__.update(k)


def test_product_binding_refuses():
    import torch
    from entropy_decoding_df11_amd import df11
    w, x = _FakeWeight(), torch.zeros(4, 64, dtype=torch.bfloat16)
    bf = torch.bfloat16
    for bad in (dict(x=x.float()), dict(x=x[:, :32]), dict(x=torch.zeros(64, 4, dtype=bf).t()),
                dict(x=torch.zeros(4, 68, dtype=bf)[:, 4:]), dict(x=torch.zeros(4, 68, dtype=bf)[:, :64]),
                dict(x=x, bias=torch.zeros(64)), dict(x=x, bias=torch.zeros(128).half()),
                dict(x=x, bias=torch.zeros(256)[::2]), dict(x=x, activation="tanh"),
                dict(x=x, residual=torch.zeros(4, 64)), dict(x=x, residual=torch.zeros(4, 128).half()),
                dict(x=x, out=torch.zeros(3, 128)), dict(x=x, out=torch.zeros(4, 128).half()),
                dict(x=x, out=torch.zeros(4, 128), out_dtype=bf), dict(x=x, out_dtype=torch.float16), dict(x=x)):
        with pytest.raises(ValueError):
            df11.matmul_epilogue(w, **bad)
    for fake in (_FakeWeight(tile_cols=0), _FakeWeight(shape=(128,))):
        with pytest.raises(ValueError):
            df11.matmul_epilogue(fake, x)
    for u in (_FakeWeight(shape=(64, 64)), _FakeWeight(decode_table_bits=12)):
        with pytest.raises(ValueError):
            df11.gated_matmul(w, u, x)
    with pytest.raises(ValueError):
        df11.gated_matmul(w, w, x, gate_bias=torch.zeros(128), up_bias=torch.zeros(128, dtype=bf))


def _product_grad(gated=False, **k):
    import ctypes
    lib = _lib_or_skip()
    a = dict(w=_stream(), u=_stream(at=0x300000000) if gated else None, t=4, inf=64, outf=128, ws=G, wb=0, dy=A, dys=128,
             dyt=0, pre=(C, D if gated else None), dx=B, dxs=64, dxt=0, db=(None, None), bt=0, act=2, g=True)
    a.update(k)
    g = _lib.ProductGrad()
    g.dy, g.dy_stride, g.dy_dtype, g.activation = a["dy"], a["dys"], a["dyt"], a["act"]
    g.dx, g.dx_stride, g.dx_dtype, g.bias_dtype = a["dx"], a["dxs"], a["dxt"], a["bt"]
    for i in range(2):
        g.pre[i], g.dbias[i] = a["pre"][i], a["db"][i]
    ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
    return lib.df11_matmul_epilogue_grad(ref(a["w"]), ref(a["u"]), a["t"], a["inf"], a["outf"],
                                         ctypes.byref(g) if a["g"] else None, a["ws"], a["wb"], None)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bad", [
    dict(w=None), dict(inf=32), dict(g=False), dict(act=7), dict(dyt=1), dict(dxt=1), dict(db=(E, None), bt=1),
    dict(dy=None), dict(dy=A + 1), dict(dyt=2, dy=A + 2), dict(dys=(1 << 31) + 1), dict(pre=(None, None)),
    dict(pre=(C + 4, D)), dict(dx=B + 1), dict(dxs=63), dict(dxs=(1 << 31) + 1), dict(db=(E + 1, None)),
    dict(dx=A), dict(dx=C + 16), dict(dx=0x202000000), dict(db=(A, None)), dict(db=(B, None)), dict(ws=G + 8),
])
def test_product_grad_refuses(gated, bad):
    if not gated and bad.get("pre") == (C + 4, D):
        bad = dict(pre=(C + 4, None))
    assert _product_grad(gated, **bad) == INVALID


def test_product_grad_refuses_second_parts():
    assert _product_grad(db=(None, E)) == INVALID
    assert _product_grad(pre=(C, D)) == INVALID
    assert _product_grad(True, u=_stream(rows=64, at=0x300000000)) == INVALID
    assert _product_grad(True, db=(E, E)) == INVALID
    assert _product_grad(t=1 << 26) == TOO_LARGE
    assert _product_grad(dx=None) == 0  # nothing asked for, nothing launched
    assert _product_grad(t=0, dy=None, dx=None, pre=(None, None)) == 0


def test_bindings_refuse_sizes_beyond_32_bits():
    """Counts that the C ABI takes in 32 bits are refused, not taken modulo 2^32
    (expanded tensors: their one row is all the memory there is)."""
    import torch
    from entropy_decoding_df11_amd import df11
    for shape in (((1 << 32) + 4, 1), ((1 << 32), 1), (1, (1 << 32) + 4), ((1 << 30) + 1, 1), (1, (1 << 30) + 1)):
        x = torch.zeros(1, 1, dtype=torch.bfloat16).expand(shape)
        with pytest.raises(ValueError, match="2\\^30"):
            df11.rms_norm(x)
    for tokens in ((1 << 32) + 4, 1 << 26):
        x = torch.zeros(1, 64, dtype=torch.bfloat16).expand(tokens, 64)
        with pytest.raises(ValueError, match="2\\^32"):
            df11.matmul_epilogue(_FakeWeight(), x)
        with pytest.raises(ValueError, match="2\\^32"):
            df11.gated_matmul(_FakeWeight(), _FakeWeight(), x)


def test_first_call_publishes_torch_last(monkeypatch):
    """A call that finds the module's torch set relies on everything else the
    first call fills in, which another thread may still be doing."""
    from entropy_decoding_df11_amd import operators
    seen = []
    make = operators._make_functions

    def watched(*a):
        make(*a)
        seen.append(operators.torch)

    monkeypatch.setattr(operators, "torch", None)
    monkeypatch.setattr(operators, "_make_functions", watched)
    monkeypatch.setattr(operators, "_Norm", None)
    monkeypatch.setattr(operators, "_Product", None)
    operators._import_torch()
    import torch
    assert seen == [None] and operators.torch is torch and operators._Norm and operators._Product


def test_bindings_refuse_outputs_that_require_a_gradient():
    import torch
    from entropy_decoding_df11_amd import df11
    x, y = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=torch.bfloat16)
    for call in (lambda: df11.rms_norm(x, out=x.clone().requires_grad_()),
                 lambda: df11.rms_norm(x, residual=x, sum_out=x.clone().requires_grad_() * 1),
                 lambda: df11.matmul_epilogue(_FakeWeight(), x, out=y.clone().requires_grad_()),
                 lambda: df11.gated_matmul(_FakeWeight(), _FakeWeight(), x, out=y.clone().requires_grad_() * 1)):
        with pytest.raises(ValueError, match="must not require a gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="on a GPU"):
            call()


# (a last row ends 2^65 bytes on: the extent of a tensor in 64 bits, 128 here, hides what it overlaps)
@pytest.mark.parametrize("bad", [
    dict(rows=(1 << 24) + 1, xs=1 << 40, y=A + 0x1000, ys=64),
    dict(rows=(1 << 24) + 1, ys=1 << 40, y=A - 0x1000, x=A),
    dict(rows=(1 << 24) + 1, r=C, rs=1 << 40, y=C + 0x1000),
])
def test_norm_refuses_strides_past_the_address_space(bad):
    assert _norm(**bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(rows=(1 << 24) + 1, ss=1 << 40, dx=A + 0x1000), dict(rows=(1 << 24) + 1, dys=1 << 40, dx=C + 0x1000),
    dict(rows=(1 << 24) + 1, dxs=1 << 40, dx=C - 0x1000), dict(rows=(1 << 24) + 1, ds=E, dss=1 << 40, dx=E + 0x1000),
])
def test_norm_grad_refuses_strides_past_the_address_space(bad):
    assert _grad(**bad) == INVALID
