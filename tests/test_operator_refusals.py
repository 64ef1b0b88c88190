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
