"""Refusals and sizes of the dense layer on the host: every call here must
fail (or do nothing) before a kernel is launched, so no GPU is needed and the
pointers are never read."""

import ctypes

import pytest
import torch

import segmented_polynomials_amd as sp

P = 4096


def need(dtype, act, n, d_in, d_out, backward):
    v = ctypes.c_size_t()
    return sp.lib.dense_workspace(dtype, act, n, d_in, d_out, backward, ctypes.byref(v)), v.value


COMMON = [(dict(dtype=sp.F64), sp.E_UNSUPPORTED), (dict(dtype=9), sp.E_INVALID), (dict(act=5), sp.E_INVALID),
          (dict(act=-1), sp.E_INVALID), (dict(n=-1), sp.E_INVALID), (dict(d_in=0), sp.E_INVALID),
          (dict(d_out=0), sp.E_INVALID), (dict(d_in=1 << 22), sp.E_UNSUPPORTED), (dict(n=1 << 31), sp.E_UNSUPPORTED),
          (dict(n=1 << 30), sp.E_UNSUPPORTED), (dict(d_in=1 << 20, d_out=1 << 20, os=1 << 20), sp.E_UNSUPPORTED),
          (dict(xs=-1), sp.E_INVALID), (dict(xs=1 << 22), sp.E_INVALID), (dict(x=None), sp.E_INVALID),
          (dict(w=None), sp.E_INVALID), (dict(x=P + 1), sp.E_INVALID), (dict(w=P + 1), sp.E_INVALID),
          (dict(bias=P + 1), sp.E_INVALID), (dict(ws=None), sp.E_INVALID), (dict(ws=P + 64), sp.E_INVALID),
          (dict(short=1), sp.E_INVALID)]


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(out=None), sp.E_INVALID), (dict(out=P + 1), sp.E_INVALID), (dict(res=P + 1), sp.E_INVALID),
    (dict(os=7), sp.E_INVALID), (dict(rs=-1), sp.E_INVALID),
    (dict(n=0, x=None, w=None, out=None, ws=None), sp.OK)])
def test_dense_fwd(change, code):
    a = dict(dtype=sp.BF16, act=0, x=P, xs=512, w=P, bias=P, res=P, rs=8, n=40, d_in=512, d_out=8, out=P, os=8, ws=P, short=0)
    a.update(change)
    rc, size = need(sp.BF16, 0, 40, 512, 8, 0)
    assert rc == sp.OK and size > 0
    assert sp.lib.dense_fwd(a["dtype"], a["act"], a["x"], a["xs"], a["w"], a["bias"], a["res"], a["rs"], a["n"],
                            a["d_in"], a["d_out"], a["out"], a["os"], a["ws"], size - a["short"], None) == code


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(gout=None), sp.E_INVALID), (dict(gout=P + 1), sp.E_INVALID), (dict(gs=-1), sp.E_INVALID),
    (dict(gs=1 << 22), sp.E_INVALID), (dict(gx=None, gw=None, gb=None), sp.E_INVALID), (dict(gx=P + 1), sp.E_INVALID),
    (dict(gw=P + 1), sp.E_INVALID), (dict(gb=P + 1), sp.E_INVALID)])
def test_dense_bwd(change, code):
    a = dict(dtype=sp.BF16, act=0, x=P, xs=8, w=P, bias=P, gout=P, gs=8, n=40, d_in=8, d_out=8, gx=P, gw=P, gb=P, ws=P,
             short=0)
    a.update(change)
    rc, size = need(sp.BF16, 0, 40, 8, 8, 1)
    assert rc == sp.OK and size > 0
    assert sp.lib.dense_bwd(a["dtype"], a["act"], a["x"], a["xs"], a["w"], a["bias"], a["gout"], a["gs"], a["n"],
                            a["d_in"], a["d_out"], a["gx"], a["gw"], a["gb"], a["ws"], size - a["short"], None) == code


def test_workspace():
    assert need(sp.F32, 0, 0, 8, 8, 1) == (sp.OK, 0)
    assert need(sp.F64, 0, 4, 8, 8, 0)[0] == sp.E_UNSUPPORTED
    assert need(sp.F32, 7, 4, 8, 8, 0)[0] == sp.E_INVALID
    assert need(sp.F32, 0, 4, -8, 8, 0)[0] == sp.E_INVALID
    assert sp.lib.dense_workspace(sp.F32, 0, 1, 1, 1, 0, None) == sp.E_INVALID
    assert sp.dense_workspace(sp.BF16, "none", 100, 64, 64, backward=True) % 256 == 0


def test_binding_checks_host_tensors():
    t, w = torch.zeros(4, 8), torch.zeros(8, 8)
    with pytest.raises(ValueError):
        sp.dense_fwd(t, w)
    with pytest.raises(ValueError):
        sp.dense_fwd(t, w, act="tanh")
    with pytest.raises(ValueError):
        sp.dense_fwd(t.double(), w.double())
    with pytest.raises(ValueError):
        sp.dense_fwd(t[0], w)
    with pytest.raises(ValueError):
        sp.dense_bwd(t, w, t)
