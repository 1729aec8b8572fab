"""Refusals and sizes of dropout and of the routing to experts on the host:
every call here must fail (or do nothing) before a kernel is launched, so no
GPU is needed and the pointers are never read."""

import ctypes

import pytest
import torch

import segmented_polynomials_amd as sp

P = 4096
NAN = float("nan")


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("change,code", [
    (dict(dtype=7), sp.E_INVALID), (dict(dtype=sp.F64), sp.E_UNSUPPORTED), (dict(mode=2), sp.E_INVALID),
    (dict(p=-0.1), sp.E_INVALID), (dict(p=1.1), sp.E_INVALID), (dict(p=NAN), sp.E_INVALID), (dict(n=-1), sp.E_INVALID),
    (dict(dim=-1), sp.E_INVALID), (dict(n=1 << 31), sp.E_UNSUPPORTED), (dict(dim=1 << 22, os=1 << 22), sp.E_UNSUPPORTED),
    (dict(xs=-8), sp.E_INVALID), (dict(os=7), sp.E_INVALID), (dict(x=None), sp.E_INVALID), (dict(out=None), sp.E_INVALID),
    (dict(x=P + 1), sp.E_INVALID), (dict(out=P + 1), sp.E_INVALID), (dict(state=P + 4), sp.E_INVALID),
    (dict(n=0, x=None, out=None), sp.OK), (dict(dim=0), sp.OK)])
def test_dropout(change, code, bwd):
    a = dict(dtype=sp.BF16, mode=0, x=P, xs=8, res=P, rs=8, p=0.5, state=P, n=3, dim=8, out=P, os=8)
    a.update(change)
    if bwd:
        rc = sp.lib.dropout_bwd(a["dtype"], a["mode"], a["x"], a["xs"], a["p"], 1, 2, a["state"], a["n"], a["dim"],
                                a["out"], a["os"], None)
    else:
        rc = sp.lib.dropout_fwd(a["dtype"], a["mode"], a["x"], a["xs"], a["res"], a["rs"], a["p"], 1, 2, a["state"],
                                a["n"], a["dim"], a["out"], a["os"], None)
    assert rc == code


def test_dropout_residual():
    def call(res, rs):
        return sp.lib.dropout_fwd(sp.F16, 0, P, 8, res, rs, 0.5, 1, 2, None, 3, 8, P, 8, None)
    assert call(P + 1, 8) == sp.E_INVALID and call(P, -8) == sp.E_INVALID


def sort_bytes(entries, num):
    v = ctypes.c_size_t()
    return sp.lib.expert_sort_workspace(entries, num, ctypes.byref(v)), v.value


@pytest.mark.parametrize("change,code", [
    (dict(idx=2), sp.E_INVALID), (dict(entries=-1), sp.E_INVALID), (dict(num=0), sp.E_INVALID),
    (dict(num=2049), sp.E_UNSUPPORTED), (dict(entries=1 << 31), sp.E_UNSUPPORTED), (dict(e=None), sp.E_INVALID),
    (dict(order=None), sp.E_INVALID), (dict(place=None), sp.E_INVALID), (dict(offsets=None), sp.E_INVALID),
    (dict(ids=None), sp.E_INVALID), (dict(e=P + 4), sp.E_INVALID), (dict(order=P + 2), sp.E_INVALID),
    (dict(offsets=P + 1), sp.E_INVALID), (dict(ws=None), sp.E_INVALID), (dict(ws=P + 64), sp.E_INVALID),
    (dict(short=1), sp.E_INVALID)])
def test_expert_sort(change, code):
    a = dict(e=P, idx=sp.I64, entries=100000, num=7, order=P, place=P, offsets=P, ids=P, ws=P, short=0)
    a.update(change)
    need = sort_bytes(100000, 7)[1]
    assert need > 0
    assert sp.lib.expert_sort(a["e"], a["idx"], a["entries"], a["num"], a["order"], a["place"], a["offsets"], a["ids"],
                              a["ws"], need - a["short"], None) == code


def test_expert_sort_workspace():
    assert sort_bytes(100, 8) == (sp.OK, 0) and sort_bytes(0, 1) == (sp.OK, 0)
    assert sort_bytes(100, 2049)[0] == sp.E_UNSUPPORTED and sort_bytes(-1, 8)[0] == sp.E_INVALID
    assert sp.lib.expert_sort_workspace(1, 1, None) == sp.E_INVALID


ROWS = [(dict(dtype=sp.F64), sp.E_UNSUPPORTED), (dict(dtype=9), sp.E_INVALID), (dict(n=-1), sp.E_INVALID),
        (dict(k=0), sp.E_INVALID), (dict(dim=-1), sp.E_INVALID), (dict(num=0), sp.E_INVALID),
        (dict(num=4000), sp.E_UNSUPPORTED), (dict(n=1 << 20, k=1 << 11), sp.E_UNSUPPORTED),
        (dict(n=1 << 40), sp.E_UNSUPPORTED), (dict(k=1 << 62, n=4), sp.E_UNSUPPORTED),
        (dict(dim=1 << 22, os=1 << 22), sp.E_UNSUPPORTED), (dict(xs=-1), sp.E_INVALID), (dict(x=None), sp.E_INVALID),
        (dict(place=None), sp.E_INVALID), (dict(offsets=None), sp.E_INVALID), (dict(out=None), sp.E_INVALID),
        (dict(x=P + 1), sp.E_INVALID), (dict(place=P + 2), sp.E_INVALID), (dict(offsets=P + 2), sp.E_INVALID),
        (dict(out=P + 1), sp.E_INVALID), (dict(n=0), sp.OK)]


@pytest.mark.parametrize("change,code", ROWS)
def test_expert_rows(change, code):
    a = dict(dtype=sp.BF16, x=P, xs=8, place=P, offsets=P, num=4, n=3, k=2, dim=8, out=P, os=8, w=P)
    a.update(change)
    sizes = (a["n"], a["k"], a["dim"])
    at = (a["place"], a["offsets"], a["num"])
    assert sp.lib.expert_dispatch_fwd(a["dtype"], a["x"], a["xs"], *at, *sizes, a["out"], None) == code
    assert sp.lib.expert_dispatch_bwd(a["dtype"], a["x"], a["xs"], *at, *sizes, a["out"], a["os"], None) == code
    assert sp.lib.expert_combine_fwd(a["dtype"], a["x"], a["xs"], *at, a["w"], None, 0, *sizes, a["out"], a["os"],
                                     None) == code
    assert sp.lib.expert_combine_bwd(a["dtype"], P, 8, a["x"], a["xs"], *at, a["w"], *sizes, a["out"], P, None) == code


def test_expert_rows_of_their_own():
    f, b, d = sp.lib.expert_combine_fwd, sp.lib.expert_combine_bwd, sp.lib.expert_dispatch_bwd
    assert f(sp.F32, P, 8, P, P, 4, None, None, 0, 3, 2, 8, P, 8, None) == sp.E_INVALID
    assert f(sp.F32, P, 8, P, P, 4, P + 2, None, 0, 3, 2, 8, P, 8, None) == sp.E_INVALID
    assert f(sp.F32, P, 8, P, P, 4, P, P, -1, 3, 2, 8, P, 8, None) == sp.E_INVALID
    assert f(sp.F32, P, 8, P, P, 4, P, P + 1, 8, 3, 2, 8, P, 8, None) == sp.E_INVALID
    assert f(sp.F32, P, 8, P, P, 4, P, None, 0, 3, 2, 8, P, 7, None) == sp.E_INVALID
    assert d(sp.F32, P, 8, P, P, 4, 3, 2, 8, P, 7, None) == sp.E_INVALID
    assert b(sp.F32, None, 8, P, 8, P, P, 4, P, 3, 2, 8, P, P, None) == sp.E_INVALID
    assert b(sp.F32, P, 8, P, 8, P, P, 4, None, 3, 2, 8, P, P, None) == sp.E_INVALID
    assert b(sp.F32, P, 8, P, 8, P, P, 4, P, 3, 2, 8, P, None, None) == sp.E_INVALID
    assert b(sp.F32, P, 8, P, 8, P, P, 4, P, 3, 2, 8, P, P + 2, None) == sp.E_INVALID
    assert b(sp.F32, P, -1, P, 8, P, P, 4, P, 3, 2, 8, P, P, None) == sp.E_INVALID


def test_binding_checks_host_tensors():
    t, e = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    off, w = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        sp.dropout_fwd(t, 0.5, 1)
    with pytest.raises(ValueError):
        sp.dropout_fwd(t.double(), 0.5, 1)
    with pytest.raises(ValueError):
        sp.dropout_fwd(t, 0.5, 1, mode="column")
    with pytest.raises(ValueError):
        sp.dropout_bwd(t, 0.5, 1)
    with pytest.raises(ValueError):
        sp.expert_sort(e, 2)
    with pytest.raises(TypeError):
        sp.expert_sort(t, 2)
    with pytest.raises(ValueError):
        sp.expert_dispatch_fwd(t, e, off)
    with pytest.raises(ValueError):
        sp.expert_dispatch_fwd(t, e.long(), off)
    with pytest.raises(ValueError):
        sp.expert_dispatch_bwd(t, e, off)
    with pytest.raises(ValueError):
        sp.expert_combine_fwd(t, e, off, w)
    with pytest.raises(ValueError):
        sp.expert_combine_bwd(t, t, e, off, w)


def test_calls_run_on_the_device_of_their_tensors(monkeypatch):
    current, seen = [0], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(sp, "_raw_stream", lambda index: 100 + index)

    def call(*args):
        seen.append((current[0], args))
        return sp.OK if args[0] == "good" else sp.E_INVALID

    sp._call(0, call, "good")
    sp._call(1, call, "good", 7)
    with pytest.raises(sp.SegpolyError):
        sp._call(1, call, "bad")
    assert seen == [(0, ("good", 100)), (1, ("good", 7, 101)), (1, ("bad", 101))] and current[0] == 0
