"""GPU parity of the routing of rows to experts: the order against a stable
sort on the host, the rows against float64.

A sum of K terms in float32 is off by at most K 2^-24 of the sum of its
absolute terms (a product counts as one more), a store by half a step."""

import pytest
import torch

from tests._gpu import announce, need_gpu

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {k: torch.finfo(v).eps / 2 for k, v in T.items()}
TINY = {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -24}
E24 = 2.0 ** -24


def check(got, ref, bound, dtype, what):
    off = (got.double() - ref).abs()
    lim = bound + HALF[dtype] * (ref.abs() + bound) + TINY[dtype]
    worst = (off / lim).max().item() if off.numel() else 0.0
    print(f"[parity] {what}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, f"{what}: {worst:.3f} times the bound"


def chosen(n, k, num, seed, idx=torch.int32, missing=0.05):
    g = torch.Generator()
    g.manual_seed(seed)
    e = (torch.rand(n, k, generator=g, dtype=torch.float64) ** 2 * num).long().clamp_(max=num - 1)
    u = torch.rand(n, k, generator=g)
    e = torch.where(u < missing / 2, torch.full_like(e, -1), e)
    e = torch.where(u > 1 - missing / 2, torch.full_like(e, num), e)
    return e.to(idx)


def sorted_on_host(e, num):
    flat = e.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < num), flat, num)
    ids, order = torch.sort(flat, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel())
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(torch.bincount(flat, minlength=num + 1)[:num], 0)])
    return order, place.reshape(e.shape), offsets, torch.where(ids < num, ids, -1)


SORTS = [(0, 2, 5), (1, 1, 1), (5, 2, 8), (64, 1, 3), (65, 1, 2048), (1024, 1, 64), (1025, 1, 64), (1000, 8, 128),
         (4096, 1, 1), (4097, 1, 7), (16384, 8, 128), (30000, 2, 2048), (70001, 4, 10), (300000, 2, 513),
         (300000, 4, 2047), (40000, 3, 400), (262144, 1, 50), (262145, 1, 50), (300000, 8, 20)]


@pytest.mark.parametrize("idx", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,k,num", SORTS)
def test_sort(n, k, num, idx):
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"expert sort n={n} k={k} experts={num} {idx}")
    e = chosen(n, k, num, n + k + num, idx)
    got = sp.expert_sort(e.cuda(), num)
    for a, b, what in zip(got, sorted_on_host(e, num), ("order", "place", "offsets", "ids")):
        assert a.dtype == torch.int32 and a.shape == b.shape
        assert torch.equal(a.cpu().long(), b), what


def test_sort_of_equal_and_missing_experts():
    need_gpu()
    import segmented_polynomials_amd as sp
    for n, value, num in ((5000, 3, 7), (5000, -1, 7), (100, 7, 7), (100000, 0, 1), (300, -2 ** 31, 9), (300, 2 ** 31 - 1, 9)):
        announce(f"expert sort: {n} times {value} of {num}")
        e = torch.full((n, 1), value, dtype=torch.int32)
        for idx in (torch.int32, torch.int64):
            got = sp.expert_sort(e.to(idx).cuda(), num)
            for a, b in zip(got, sorted_on_host(e, num)):
                assert torch.equal(a.cpu().long(), b)
    announce("expert sort: numbers past 32 bits are no expert")
    e = torch.tensor([[2 ** 32 + 1, 1, -2 ** 40]])
    order, place, offsets, ids = sp.expert_sort(e.cuda(), 4)
    assert order.tolist() == [1, 0, 2] and offsets.tolist() == [0, 0, 1, 1, 1] and ids.tolist() == [1, -1, -1]


ROWS = [(1, 1, 1, 1), (5, 2, 8, 1000), (33, 3, 4, 7), (700, 2, 16, 128), (257, 9, 5, 70), (100, 1, 3, 1030),
        (40, 17, 64, 264), (6, 2, 3, 8200), (3000, 4, 10, 33), (64, 8, 8, 2048),
        (20000, 2, 8, 300), (2000, 3, 4, 1500), (3000, 2, 4, 1500)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,k,num,d", ROWS)
def test_rows(n, k, num, d, dtype):
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"expert rows n={n} k={k} experts={num} d={d} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(n + d)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(T[dtype])
    e = chosen(n, k, num, n * k, missing=0.2).cuda()
    order, place, offsets, ids = sp.expert_sort(e, num)
    total, row = int(offsets[-1]), order.long() // k
    used = (place < total)
    at = place.long()

    x = rnd(n, d)
    xs = sp.expert_dispatch_fwd(x, place, offsets)
    want = x[row] * (ids >= 0)[:, None]
    assert torch.equal(xs, want)
    gxs = rnd(n * k, d)
    dx = sp.expert_dispatch_bwd(gxs, place, offsets)
    terms = gxs.double()[at] * used[:, :, None]
    check(dx, terms.sum(1), k * E24 * terms.abs().sum(1), dtype, "grad_x")

    ys, w, res, gout = rnd(n * k, d), rnd(n, k).float(), rnd(n, d), rnd(n, d)
    ys[total:] = float("nan")  # slots without an expert count for nothing
    clean = torch.where((ids >= 0)[:, None], ys, 0)
    terms = clean.double()[at] * (w.double() * used)[:, :, None]
    out = sp.expert_combine_fwd(ys, place, offsets, w)
    check(out, terms.sum(1), (k + 1) * E24 * terms.abs().sum(1), dtype, "out")
    out = sp.expert_combine_fwd(ys, place, offsets, w, residual=res)
    ref = terms.sum(1) + res.double()
    check(out, ref, (k + 2) * E24 * (terms.abs().sum(1) + res.double().abs()), dtype, "out with residual")
    gys, gw = sp.expert_combine_bwd(gout, ys, place, offsets, w)
    ref = torch.zeros(n * k, d, dtype=torch.float64, device="cuda")
    ref[at.reshape(-1)] = ((w.double() * used)[:, :, None] * gout.double()[:, None]).reshape(n * k, d)
    check(gys, ref, E24 * ref.abs(), dtype, "grad_ys")
    prod = clean.double()[at] * gout.double()[:, None]
    check(gw, prod.sum(2) * used, (d + 1) * E24 * prod.abs().sum(2), "f32", "grad_weights")
    assert bool((gw[~used] == 0).all()) and bool((gys[total:] == 0).all())

    # rows of wider tensors at odd places: the same bits, neighbours untouched
    def wide(t):
        v = torch.full((t.shape[0], d + 3), 5.0, dtype=t.dtype, device="cuda")
        v[:, 1:1 + d] = t
        return v[:, 1:1 + d]

    assert torch.equal(sp.expert_dispatch_fwd(wide(x), place, offsets), xs)
    o = wide(torch.zeros_like(x))
    sp.expert_dispatch_bwd(wide(gxs), place, offsets, grad_x=o)
    assert torch.equal(o, dx) and bool((o._base[:, 0] == 5).all()) and bool((o._base[:, 1 + d:] == 5).all())
    o = wide(res)
    sp.expert_combine_fwd(wide(ys), place, offsets, w, residual=o, out=o)
    assert torch.equal(o, out) and bool((o._base[:, 0] == 5).all()) and bool((o._base[:, 1 + d:] == 5).all())
    again = sp.expert_combine_bwd(wide(gout), wide(ys), place, offsets, w)
    assert torch.equal(again[0], gys) and torch.equal(again[1], gw)
    one = sp.expert_dispatch_fwd(x[:1].expand(n, d), place, offsets)
    assert torch.equal(one, x[:1].expand(n * k, d) * (ids >= 0)[:, None])


def test_rows_without_any_expert_and_no_rows():
    need_gpu()
    import segmented_polynomials_amd as sp
    announce("expert rows: none has an expert")
    n, k, d = 70, 3, 40
    place, offsets = sp.expert_sort(torch.full((n, k), -1, device="cuda"), 4)[1:3]
    x, ys = torch.randn(n, d, device="cuda"), torch.full((n * k, d), float("nan"), device="cuda")
    w = torch.full((n, k), float("nan"), device="cuda")
    assert not sp.expert_dispatch_fwd(x, place, offsets).any()
    assert not sp.expert_dispatch_bwd(ys, place, offsets).any()
    assert torch.equal(sp.expert_combine_fwd(ys, place, offsets, w, residual=x), x)
    gys, gw = sp.expert_combine_bwd(x, ys, place, offsets, w)
    assert not gys.any() and not gw.any()
    announce("expert rows: no rows")
    e = torch.zeros(0, 2, dtype=torch.int64, device="cuda")
    order, place, offsets, ids = sp.expert_sort(e, 3)
    assert offsets.tolist() == [0, 0, 0, 0] and order.numel() == ids.numel() == 0
    assert sp.expert_dispatch_fwd(x[:0], place, offsets).shape == (0, d)
    assert sp.expert_combine_fwd(ys[:0], place, offsets, w[:0, :2]).shape == (0, d)
    announce("expert rows: no columns")
    place, offsets = sp.expert_sort(torch.zeros(5, 2, dtype=torch.int32, device="cuda"), 1)[1:3]
    assert not sp.expert_combine_bwd(x[:5, :0], ys[:10, :0], place, offsets, torch.ones(5, 2, device="cuda"))[1].any()


def test_places_out_of_range_are_passed_over():
    need_gpu()
    import segmented_polynomials_amd as sp
    announce("expert rows: places out of range")
    n, k, d = 4, 2, 24
    place = torch.tensor([[0, -1], [2, 8], [2 ** 31 - 1, 5], [-2 ** 31, 7]], dtype=torch.int32, device="cuda")
    x, ys, w = torch.randn(n, d, device="cuda"), torch.randn(n * k, d, device="cuda"), torch.rand(n, k, device="cuda")
    for end in (8, 100, -5):  # the last of the offsets out of range too
        offsets = torch.tensor([0, end], dtype=torch.int32, device="cuda")
        ref = torch.stack([ys[0] * w[0, 0], ys[2] * w[1, 0], ys[5] * w[2, 1], ys[7] * w[3, 1]])
        assert torch.equal(sp.expert_combine_fwd(ys, place, offsets, w), ref)
        assert torch.equal(sp.expert_dispatch_fwd(x, place, offsets)[[0, 2, 5, 7]], x)
        gys, gw = sp.expert_combine_bwd(x, ys, place, offsets, w)
        assert torch.equal(gys[[0, 2, 5, 7]], x * torch.stack([w[0, 0], w[1, 0], w[2, 1], w[3, 1]])[:, None])
        assert gw[0, 1] == 0 and gw[1, 1] == 0 and gw[2, 0] == 0 and gw[3, 0] == 0


def test_slots_past_32_bits_of_bytes():
    """Rows by slot of more than 2^32 elements."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce("expert rows: more than 2^32 elements by slot")
    n, k, d = 2 ** 16 + 5, 2, 2 ** 15 + 8
    x = torch.arange(n, device="cuda").remainder(251).to(torch.bfloat16)[:, None].repeat(1, d)
    e = torch.arange(n * k, device="cuda", dtype=torch.int32).reshape(n, k).flip(0) % 3
    order, place, offsets, ids = sp.expert_sort(e.contiguous(), 3)
    xs = sp.expert_dispatch_fwd(x, place, offsets)
    rows = (order.long() // k) % 251
    assert torch.equal(xs[:, 0], rows.bfloat16()) and torch.equal(xs[:, d - 1], rows.bfloat16())
    w = torch.full((n, k), 0.5, device="cuda")
    out = sp.expert_combine_fwd(xs, place, offsets, w)
    assert torch.equal(out[:, 0], x[:, 0]) and torch.equal(out[:, -1], x[:, 0])


def test_captured_graph():
    need_gpu()
    import segmented_polynomials_amd as sp
    announce("experts: captured into a graph")
    n, k, num, d = 9000, 2, 6, 72
    e = torch.zeros(n, k, dtype=torch.int32, device="cuda")
    x, w = torch.randn(n, d, device="cuda"), torch.rand(n, k, device="cuda")

    def run():
        order, place, offsets, ids = sp.expert_sort(e, num)
        xs = sp.expert_dispatch_fwd(x, place, offsets)
        out = sp.expert_combine_fwd(xs, place, offsets, w, residual=x)
        gys, gw = sp.expert_combine_bwd(out, xs, place, offsets, w)
        return order, offsets, ids, out, gys, gw, sp.expert_dispatch_bwd(gys, place, offsets)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for seed in range(3):
        e.copy_(chosen(n, k, num, seed))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, run()):
            assert torch.equal(a, b)
