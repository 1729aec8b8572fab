"""Refusals and sizes of the invariant-channel operators on the host: every
call here must fail (or do nothing) before a kernel is launched, so no GPU is
needed and the pointers are never read."""

import ctypes

import pytest
import torch

import segmented_polynomials_amd as sp

P = 4096          # a non-null address, 256-byte aligned
WS = ctypes.c_size_t


def size(fn, *args):
    v = WS()
    rc = fn(*args, ctypes.byref(v))
    return rc, v.value


@pytest.mark.parametrize("change,code", [
    (dict(dtype=7), sp.E_INVALID), (dict(dtype=sp.F64), sp.E_UNSUPPORTED), (dict(idx=2), sp.E_INVALID),
    (dict(rows=-1), sp.E_INVALID), (dict(n=-1), sp.E_INVALID), (dict(dim=-1), sp.E_INVALID),
    (dict(dim=1 << 22, stride=1 << 22), sp.E_UNSUPPORTED), (dict(rows=1 << 31), sp.E_UNSUPPORTED),
    (dict(n=1 << 31), sp.E_UNSUPPORTED), (dict(table=None), sp.E_INVALID), (dict(tokens=None), sp.E_INVALID),
    (dict(out=None), sp.E_INVALID), (dict(stride=7), sp.E_INVALID), (dict(out=P + 1), sp.E_INVALID),
    (dict(n=0, table=None, tokens=None, out=None), sp.OK), (dict(dim=0, stride=0), sp.OK)])
def test_embedding_fwd(change, code):
    a = dict(dtype=sp.BF16, table=P, rows=5, dim=8, tokens=P, idx=sp.I32, n=3, out=P, stride=8)
    a.update(change)
    assert sp.lib.embedding_fwd(a["dtype"], a["table"], a["rows"], a["dim"], a["tokens"], a["idx"], a["n"], 1.0,
                                a["out"], a["stride"], None) == code


@pytest.mark.parametrize("change,code", [
    (dict(dtype=sp.F64), sp.E_UNSUPPORTED), (dict(stride=-1), sp.E_INVALID), (dict(grad=None), sp.E_INVALID),
    (dict(tokens=None), sp.E_INVALID), (dict(out=None), sp.E_INVALID), (dict(ws=None), sp.E_INVALID),
    (dict(ws=P + 64), sp.E_INVALID), (dict(short=1), sp.E_INVALID), (dict(rows=0), sp.OK), (dict(dim=0), sp.OK)])
def test_embedding_bwd(change, code):
    a = dict(dtype=sp.F32, grad=P, stride=8, tokens=P, n=3, rows=5, dim=8, out=P, ws=P, short=0)
    a.update(change)
    rc, need = size(sp.lib.embedding_bwd_workspace, a["n"], a["rows"], a["dim"])
    assert rc == sp.OK
    assert sp.lib.embedding_bwd(a["dtype"], a["grad"], a["stride"], a["tokens"], sp.I64, a["n"], a["rows"], a["dim"], 1.0,
                                a["out"], a["ws"], need - a["short"], None) == code


def test_embedding_workspace():
    assert size(sp.lib.embedding_bwd_workspace, 10, 0, 4) == (sp.OK, 0)
    assert size(sp.lib.embedding_bwd_workspace, -1, 4, 4)[0] == sp.E_INVALID
    assert sp.lib.embedding_bwd_workspace(1, 1, 1, None) == sp.E_INVALID
    # sorted keys and positions twice, the row ranges, one float32 row per 32 tokens
    n, rows, dim = 100000, 40000, 70
    need = sp.embedding_bwd_workspace(n, rows, dim)
    assert need >= 16 * n + 4 * (rows + 1) + 4 * (n // 32) * dim
    assert need % 256 == 0


@pytest.mark.parametrize("change,code", [
    (dict(dtype=sp.F64), sp.E_UNSUPPORTED), (dict(kind=2), sp.E_INVALID), (dict(mode=3), sp.E_INVALID),
    (dict(act=2), sp.E_INVALID), (dict(eps=-1e-6), sp.E_INVALID), (dict(eps=float("nan")), sp.E_INVALID),
    (dict(n=-1), sp.E_INVALID), (dict(dim=-1), sp.E_INVALID), (dict(dim=16385), sp.E_UNSUPPORTED),
    (dict(xs=-8), sp.E_INVALID), (dict(x=None), sp.E_INVALID), (dict(f=None), sp.E_INVALID),
    (dict(gate=None), sp.E_INVALID), (dict(post=None), sp.E_INVALID), (dict(y=None), sp.E_INVALID),
    (dict(h=None), sp.E_INVALID), (dict(pre=None), sp.E_INVALID), (dict(n=0), sp.OK), (dict(dim=0), sp.OK)])
def test_block_norm_fwd(change, code):
    a = dict(dtype=sp.F16, kind=1, mode=2, act=1, x=P, xs=8, f=P, gate=P, post=P, pre=P, eps=1e-6, n=3, dim=8, y=P, h=P)
    a.update(change)
    assert sp.lib.block_norm_fwd(a["dtype"], a["kind"], a["mode"], a["act"], a["x"], a["xs"], a["f"], 8, a["gate"], 8,
                                 a["post"], P, a["pre"], a["eps"], a["n"], a["dim"], a["y"], a["h"], None) == code


@pytest.mark.parametrize("change,code", [
    (dict(dtype=9), sp.E_INVALID), (dict(y=None), sp.E_INVALID), (dict(gy=None), sp.E_INVALID),
    (dict(gh=None), sp.E_INVALID), (dict(ggate=None), sp.E_INVALID), (dict(gpost=None), sp.E_INVALID),
    (dict(gscale=None), sp.E_INVALID), (dict(gpre=None), sp.E_INVALID), (dict(short=1), sp.E_INVALID),
    (dict(ws=None), sp.E_INVALID), (dict(ws=P + 8), sp.E_INVALID), (dict(dim=0), sp.OK)])
def test_block_norm_bwd(change, code):
    a = dict(dtype=sp.F32, y=P, gy=P, gh=P, ggate=P, gpost=P, gscale=P, gpre=P, ws=P, short=0, n=3, dim=8)
    a.update(change)
    rc, need = size(sp.lib.block_norm_bwd_workspace, a["n"], a["dim"])
    assert rc == sp.OK
    assert sp.lib.block_norm_bwd(a["dtype"], 0, 2, 0, a["y"], 8, a["gy"], 8, a["gh"], 8, P, 8, P, 8, P, P, P, 1e-6,
                                 a["n"], a["dim"], P, P, a["ggate"], a["gpost"], a["gscale"], a["gpre"], a["ws"],
                                 need - a["short"], None) == code


@pytest.mark.parametrize("change,code", [
    (dict(dtype=sp.F64), sp.E_UNSUPPORTED), (dict(act=4), sp.E_INVALID), (dict(act=-1), sp.E_INVALID),
    (dict(n=-1), sp.E_INVALID), (dict(hidden=0), sp.E_INVALID), (dict(d_in=0), sp.E_INVALID),
    (dict(xs=-1), sp.E_INVALID), (dict(xs=1 << 22), sp.E_INVALID), (dict(os=7), sp.E_INVALID),
    (dict(x=None), sp.E_INVALID), (dict(wd=None), sp.E_INVALID), (dict(out=None), sp.E_INVALID),
    (dict(ws=None), sp.E_INVALID), (dict(short=1), sp.E_INVALID), (dict(n=0), sp.OK)])
def test_gated_ffn_fwd(change, code):
    a = dict(dtype=sp.BF16, act=0, x=P, xs=8, wd=P, n=3, d_in=8, hidden=16, out=P, os=8, ws=P, short=0)
    a.update(change)
    rc, need = size(sp.lib.gated_ffn_workspace, sp.BF16, 3, 8, 16, 8, 0)
    assert rc == sp.OK
    assert sp.lib.gated_ffn_fwd(a["dtype"], a["act"], a["x"], a["xs"], P, P, a["wd"], a["n"], a["d_in"], a["hidden"], 8,
                                a["out"], a["os"], a["ws"], need - a["short"], None) == code


@pytest.mark.parametrize("change,code", [
    (dict(gs=-1), sp.E_INVALID), (dict(gout=None), sp.E_INVALID), (dict(gwu=None), sp.E_INVALID),
    (dict(gx=None, gwg=None, gwu=None, gwd=None), sp.E_INVALID), (dict(ws=None), sp.E_INVALID),
    (dict(short=1), sp.E_INVALID), (dict(dtype=sp.F64), sp.E_UNSUPPORTED)])
def test_gated_ffn_bwd(change, code):
    a = dict(dtype=sp.F32, gout=P, gs=8, gx=P, gwg=P, gwu=P, gwd=P, ws=P, short=0)
    a.update(change)
    rc, need = size(sp.lib.gated_ffn_workspace, sp.F32, 3, 8, 16, 8, 1)
    assert rc == sp.OK
    assert sp.lib.gated_ffn_bwd(a["dtype"], 0, P, 8, P, P, P, a["gout"], a["gs"], 3, 8, 16, 8, a["gx"], a["gwg"],
                                a["gwu"], a["gwd"], a["ws"], need - a["short"], None) == code


def test_workspace_queries_refuse_what_the_calls_refuse():
    assert size(sp.lib.block_norm_bwd_workspace, 4, 16385)[0] == sp.E_UNSUPPORTED
    assert size(sp.lib.gated_ffn_workspace, sp.F64, 4, 8, 8, 8, 0)[0] == sp.E_UNSUPPORTED
    assert size(sp.lib.gated_ffn_workspace, sp.F32, 4, 8, -8, 8, 0)[0] == sp.E_INVALID
    assert size(sp.lib.gated_ffn_workspace, sp.F32, 0, 8, 8, 8, 0) == (sp.OK, 0)


def test_binding_checks_host_tensors():
    """Tensors that are not on a GPU, or of another type or shape, are
    refused by the binding."""
    t = torch.zeros(4, 8)
    w = torch.ones(8)
    with pytest.raises(ValueError):
        sp.embedding_fwd(t, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        sp.embedding_bwd(t.double(), torch.zeros(4, dtype=torch.int32), 3)
    with pytest.raises(TypeError):
        sp.embedding_bwd(t, torch.zeros(4), 3)
    with pytest.raises(ValueError):
        sp.block_norm_fwd(t, t, w)
    with pytest.raises(ValueError):
        sp.block_norm_fwd(t, t, w, kind="batch")
    with pytest.raises(ValueError):
        sp.gated_ffn_fwd(t, t, t, t)
    with pytest.raises(ValueError):
        sp.gated_ffn_fwd(t, t, t, t, act="tanh")


def test_embedding_workspace_of_small_tables():
    """Tables summed in LDS: the sums of the segments, bounded for wide rows."""
    assert sp.embedding_bwd_workspace(50000, 10, 128) == 4 * 512 * 10 * 128
    assert sp.embedding_bwd_workspace(1, 10, 128) == 4 * 10 * 128
    assert sp.embedding_bwd_workspace(1 << 30, 16, 1 << 21) == 4 * 16 << 21
    assert sp.embedding_bwd_workspace(1 << 30, 16, 8192) == 4 * 64 * 16 * 8192
