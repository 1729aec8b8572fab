"""GPU parity of dropout: the mask bit for bit against the generator in NumPy,
the values against float64.

A value is x times a scale that is itself a rounded float32, plus the residual:
three roundings of at most half a step of float32, then the one of the store."""

import numpy as np
import pytest
import torch

from tests._gpu import announce, need_gpu
from tests._philox import kept, philox

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {k: torch.finfo(v).eps / 2 for k, v in T.items()}
TINY = {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -24}
E24 = 2.0 ** -24


def test_generator_known_answers():
    """The published known-answer vectors of Philox 4x32-10."""
    one = 0xFFFFFFFF
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((one,) * 4, (one, one), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert tuple(int(v) for v in philox(counter, key)) == want


def normal(n, d, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(n, d, generator=g, device="cuda").to(T[dtype])


def check(got, x, keep, p, res, dtype):
    scale = 1 / (1 - p) if p < 1 else 0.0
    keep = torch.from_numpy(np.array(keep)).cuda()
    v = torch.where(keep, x.double() * scale, 0.0)
    ref = v if res is None else v + res.double()
    bound = 2 * E24 * v.abs() + (0 if res is None else E24 * (ref.abs() + 1e-30))
    lim = bound + HALF[dtype] * (ref.abs() + bound) + TINY[dtype]
    assert ((got.double() - ref).abs() <= lim).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,d,p,mode,residual", [
    (1, 1, 0.5, "element", False), (3, 5, 0.3, "element", True), (1, 4099, 0.1, "element", True),
    (700, 128, 0.2, "element", False), (257, 1030, 0.5, "element", True), (33, 64, 0.0, "element", True),
    (33, 64, 1.0, "element", True), (5000, 3, 0.25, "element", False), (999, 77, 0.4, "row", True),
    (4100, 16, 0.9, "row", False), (20, 40, 1e-9, "element", False), (64, 64, 1 - 2.0 ** -32, "element", False)])
def test_dropout(n, d, p, mode, residual, dtype):
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dropout n={n} d={d} p={p} {mode} residual={residual} {dtype}")
    seed, offset = 0x1234567890ABCDEF, 2 ** 40 + 7
    x, res = normal(n, d, dtype, 1), normal(n, d, dtype, 2) if residual else None
    keep = kept(n, d, p, seed, offset, mode == "row")
    out = sp.dropout_fwd(x, p, seed, offset=offset, residual=res, mode=mode)
    check(out, x, keep, p, res, dtype)
    g = normal(n, d, dtype, 3)
    dx = sp.dropout_bwd(g, p, seed, offset=offset, mode=mode)
    check(dx, g, keep, p, None, dtype)
    # columns of wider tensors at odd places give the same bits, the others stay
    wide = torch.full((n, d + 3), 5.0, dtype=T[dtype], device="cuda")
    wx, wr = wide.clone(), wide.clone()
    wx[:, 1:1 + d] = x
    if residual:
        wr[:, 2:2 + d] = res
    sp.dropout_fwd(wx[:, 1:1 + d], p, seed, offset=offset, residual=wr[:, 2:2 + d] if residual else None, mode=mode,
                   out=wide[:, 1:1 + d])
    assert torch.equal(wide[:, 1:1 + d], out) and bool((wide[:, 0] == 5).all()) and bool((wide[:, 1 + d:] == 5).all())
    # in place, over x and over the residual
    assert torch.equal(sp.dropout_fwd(x.clone(), p, seed, offset=offset, residual=res, mode=mode), out)
    y = x.clone()
    assert torch.equal(sp.dropout_fwd(y, p, seed, offset=offset, residual=res, mode=mode, out=y), out)
    if residual:
        r = res.clone()
        assert torch.equal(sp.dropout_fwd(x, p, seed, offset=offset, residual=r, mode=mode, out=r), out)
    # seed and offset from the device, partly
    state = torch.tensor([seed, offset - 3], device="cuda")
    assert torch.equal(sp.dropout_fwd(x, p, state, offset=3, residual=res, mode=mode), out)
    # one row for all
    one = sp.dropout_fwd(x[:1].expand(n, d), p, seed, offset=offset, mode=mode)
    check(one, x[:1].expand(n, d), keep, p, None, dtype)


@pytest.mark.gpu
def test_mask_does_not_depend_on_the_width():
    need_gpu()
    import segmented_polynomials_amd as sp
    announce("dropout: mask of the first columns of a wider call")
    x = torch.ones(50, 301, device="cuda")
    a = sp.dropout_fwd(x, 0.5, 9)
    assert torch.equal(sp.dropout_fwd(x[:20, :130], 0.5, 9), a[:20, :130])
    assert not torch.equal(sp.dropout_fwd(x, 0.5, 9, offset=1), a) and not torch.equal(sp.dropout_fwd(x, 0.5, 10), a)
    assert torch.equal(sp.dropout_fwd(x, 0.5, -1), sp.dropout_fwd(x, 0.5, 2 ** 64 - 1))


@pytest.mark.gpu
def test_dropped_values_count_for_nothing():
    need_gpu()
    import segmented_polynomials_amd as sp
    announce("dropout: NaN and infinities in dropped places")
    n, d, p = 64, 200, 0.5
    keep = torch.from_numpy(np.array(kept(n, d, p, 3, 0))).cuda()
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = torch.where(keep, torch.ones(n, d, device="cuda"), bad)
        assert torch.equal(sp.dropout_fwd(x, p, 3), keep * 2.0)
    keep = torch.from_numpy(np.array(kept(n, d, p, 3, 0, True))).cuda()
    x = torch.where(keep, torch.ones(n, d, device="cuda"), float("nan"))
    assert torch.equal(sp.dropout_fwd(x, p, 3, mode="row"), keep * 2.0)
    assert not sp.dropout_fwd(torch.full((n, d), float("nan"), device="cuda"), 1.0, 3).any()


@pytest.mark.gpu
def test_captured_graph_takes_the_state_of_each_replay():
    need_gpu()
    import segmented_polynomials_amd as sp
    announce("dropout: captured into a graph")
    n, d, p = 300, 130, 0.3
    x, res = normal(n, d, "f32", 1), normal(n, d, "f32", 2)
    state = torch.tensor([17, 0], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sp.dropout_fwd(x, p, state, residual=res)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sp.dropout_fwd(x, p, state, residual=res)
        dx = sp.dropout_bwd(x, p, state)
        state[1] += 1
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, sp.dropout_fwd(x, p, 17, offset=step, residual=res))
        assert torch.equal(dx, sp.dropout_bwd(x, p, 17, offset=step))
        assert state.tolist() == [17, step + 1]


@pytest.mark.gpu
def test_share_that_is_kept():
    """Of m draws the kept share is off by at most six standard deviations."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce("dropout: kept share")
    for p in (0.1, 0.5, 0.8):
        out = sp.dropout_fwd(torch.ones(2000, 1000, device="cuda"), p, 5)
        share = (out != 0).double().mean().item()
        assert abs(share - (1 - p)) <= 6 * (p * (1 - p) / 2e6) ** 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["element", "row"])
def test_rows_past_32_bits_of_elements(mode):
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dropout: rows far apart, and more than 2^31 elements, {mode}")
    n, d, stride = 1100, 130, 1 << 21
    x = normal(n, d, "bf16", 5)
    want = sp.dropout_fwd(x, 0.3, 8, offset=2, mode=mode)
    held = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda")
    far = torch.as_strided(held, (n, d), (stride, 1))
    far.copy_(x)
    assert torch.equal(sp.dropout_fwd(far, 0.3, 8, offset=2, mode=mode, out=far), want)
    # the first columns of a wide call: a row's mask does not depend on the width
    rows, wide = (1 << 17) + 5, 1 << 14
    held = held[:rows * wide].view(rows, wide)
    assert held.numel() > 2 ** 31
    held.fill_(1.0)
    a = sp.dropout_fwd(held[:, :40], 0.3, 8, mode=mode)
    assert torch.equal(sp.dropout_fwd(held, 0.3, 8, mode=mode, out=held)[:, :40], a)
