"""GPU parity of the dense layer and its gradient against the definition in
float64.

Tolerances are bounds carried through the definition beside the value: a
float32 sum of K terms is off by at most about K 2^-24 of the sum of its
absolute terms, the gradient before the activation is held with half a step of
its type (float32: 24 bits in three parts; float16: in blocks, whose small
values are off by at most 2^-16 of the block's largest), a store by half a
step."""

import math

import pytest
import torch

from tests._gpu import announce, need_gpu

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {k: torch.finfo(v).eps / 2 for k, v in T.items()}
TINY = {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -24}
E24 = 2.0 ** -24
ACTS = ["none", "silu", "gelu", "relu", "sigmoid"]


def check(got, ref, bound, dtype, what):
    assert got.dtype == T[dtype] and got.shape == ref.shape
    assert torch.isfinite(got).all(), what
    off = (got.double() - ref).abs()
    lim = bound + HALF[dtype] * (ref.abs() + bound) + TINY[dtype]
    worst = (off / lim).max().item() if off.numel() else 0.0
    print(f"[parity] {what}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, f"{what}: {worst:.3f} times the bound"


def act64(z, act):
    """Value, slope and a bound of the slope's change."""
    if act == "none":
        return z, torch.ones_like(z), 0.0
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s)), 0.5
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi), 0.8
    if act == "relu":
        return z.clamp_min(0), (z > 0).double(), 0.0
    s = torch.sigmoid(z)
    return s, s * (1 - s), 0.1


def reference(x, w, b, res, g, act, dtype):
    """(out, bound) and the gradients with theirs."""
    x, w, g = x.double(), w.double(), g.double()
    s = lambda k: (k + 64) * E24
    n, di, do = x.shape[0], x.shape[1], w.shape[0]
    z, ez = x @ w.T, s(di) * (x.abs() @ w.abs().T)
    if b is not None:
        z = z + b.double()
        ez = ez + E24 * z.abs()
    a, da, d2 = act64(z, act)
    fast = 0.0 if act in ("none", "relu") else 2.0 ** -18  # exp and erf in float32, |z| < 64 here
    ea = 1.13 * ez + fast * a.abs() + fast * E24
    eda = d2 * ez + fast
    if act == "relu":
        ea, eda = ez, (z.abs() <= ez).double()  # the step may fall on the other side
    out, eout = (a, ea) if res is None else (a + res.double(), ea + E24 * (a.abs() + res.double().abs()))
    d = g * da
    ed = g.abs() * eda + E24 * d.abs()
    eb = ed.sum(0) + s(n) * d.abs().sum(0)
    if act != "none":
        held = HALF[dtype] if dtype != "f32" else 2 * E24
        ed = ed + held * (d.abs() + ed) + TINY[dtype]
        if dtype == "f16":
            ed = ed + 2.0 ** -16 * d.abs().max()
    dx, edx = d @ w, ed @ w.abs() + s(do) * (d.abs() @ w.abs())
    dw, edw = d.T @ x, ed.T @ x.abs() + s(n) * (d.abs().T @ x.abs())
    return (out, eout), ((dx, edx), (dw, edw), (d.sum(0), eb))


def case(n, di, do, dtype, seed, bias=True):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device="cuda") * std).to(T[dtype])
    return r(n, di), r(do, di, std=di ** -0.5), r(do, std=0.3) if bias else None, r(n, do), r(n, do)


def run(n, di, do, dtype, act, seed, bias=True, residual=True):
    import segmented_polynomials_amd as sp
    announce(f"dense n={n} d_in={di} d_out={do} {dtype} {act} bias={bias} residual={residual}")
    x, w, b, res, g = case(n, di, do, dtype, seed, bias)
    (out, eout), grads = reference(x, w, b, res if residual else None, g, act, dtype)
    check(sp.dense_fwd(x, w, bias=b, act=act, residual=res if residual else None), out, eout, dtype, "out")
    got = sp.dense_bwd(x, w, g, bias=b, act=act)
    for name, a, (r, e) in zip(("grad_x", "grad_w", "grad_bias"), got, grads):
        if a is None:
            assert name == "grad_bias" and b is None
            continue
        check(a, r, e, dtype, name)
    assert all(p is q or torch.equal(p, q) for p, q in zip(got, sp.dense_bwd(x, w, g, bias=b, act=act)))
    return x, w, b, res, g, got


SHAPES = [(1, 1, 1), (1, 8, 8), (3, 64, 128), (16, 72, 40), (17, 61, 35), (5, 1001, 333), (65, 128, 96), (130, 322, 257),
          (300, 200, 520), (33, 2048, 96), (1000, 8, 64), (1000, 64, 64), (777, 128, 100), (700, 7, 3), (64, 256, 1),
          (24, 1000, 70), (32, 130, 1030), (20, 1024, 33), (12, 100, 90), (12, 520, 90),
          (1500, 40, 24), (1025, 64, 63), (129, 5, 64)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,do", SHAPES)
def test_dense(n, di, do, dtype, act):
    need_gpu()
    run(n, di, do, dtype, act, n + di + do, bias=(n + di) % 3 != 0, residual=n % 2 == 1)


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,do", [(4096, 72, 2048), (2048, 4096, 136), (4100, 1030, 1032), (300, 8000, 20),
                                     (40, 3000, 5000), (70, 9000, 64), (20000, 33, 17), (50000, 64, 64), (9, 64, 4000),
                                     (30000, 128, 512), (257, 64, 8000), (8000, 512, 512)])
def test_dense_large(n, di, do, dtype, act):
    """Every tile, sums shared out over workgroups, many rows of few columns."""
    need_gpu()
    run(n, di, do, dtype, act, 11)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,do", [(90, 64, 48), (7, 136, 33), (4000, 40, 72)])
def test_strides_and_parts(n, di, do, dtype, act):
    need_gpu()
    import segmented_polynomials_amd as sp
    x, w, b, res, g = case(n, di, do, dtype, 2)
    announce(f"dense on columns of wider tensors {n} {di} {do} {dtype} {act}")
    out = sp.dense_fwd(x, w, bias=b, act=act, residual=res)
    full = sp.dense_bwd(x, w, g, bias=b, act=act)

    def wide(t, shift, fill=float("nan")):
        v = torch.full((t.shape[0], t.shape[1] + 40), fill, dtype=t.dtype, device="cuda")
        v[:, shift:shift + t.shape[1]] = t
        return v[:, shift:shift + t.shape[1]]

    for shift in (8, 3):  # the second leaves rows off 16 bytes
        to = wide(res, shift, 5.0)
        sp.dense_fwd(wide(x, shift), w, bias=b, act=act, residual=to, out=to)
        assert torch.equal(to, out)
        assert bool((to._base[:, :shift] == 5).all()) and bool((to._base[:, shift + do:] == 5).all())
        got = sp.dense_bwd(wide(x, shift), w, wide(g, shift), bias=b, act=act)
        assert all(torch.equal(p, q) for p, q in zip(got, full))
    announce("dense: one row read by all")
    one = sp.dense_fwd(x[:1].expand(n, di), w, bias=b, act=act, residual=res[:1].expand(n, do))
    same = sp.dense_fwd(x[:1].repeat(n, 1), w, bias=b, act=act, residual=res[:1].repeat(n, 1))
    assert torch.equal(one, same)
    got = sp.dense_bwd(x[:1].expand(n, di), w, g[:1].expand(n, do), bias=b, act=act)
    same = sp.dense_bwd(x[:1].repeat(n, 1), w, g[:1].repeat(n, 1), bias=b, act=act)
    assert all(torch.equal(p, q) for p, q in zip(got, same))
    announce("dense: parts of the backward, no rows")
    only = sp.dense_bwd(x, w, g, bias=b, act=act, need_dw=False)
    assert torch.equal(only[0], full[0]) and only[1] is None and only[2] is None
    only = sp.dense_bwd(x, w, g, bias=b, act=act, need_dx=False)
    assert only[0] is None and torch.equal(only[1], full[1]) and torch.equal(only[2], full[2])
    assert sp.dense_bwd(x, w, g, bias=b, act=act, need_dx=False, need_dw=False) == (None, None, None)
    none = sp.dense_bwd(x[:0], w, g[:0], bias=b, act=act)
    assert none[0].shape == (0, di) and not none[1].any() and not none[2].any()
    assert sp.dense_fwd(x[:0], w, bias=b, act=act).shape == (0, do)
    # a row of a tensor whose stride is far past what the kernels take
    long = torch.as_strided(x, (1, di), (1 << 40, 1))
    assert torch.equal(sp.dense_fwd(long, w, bias=b, act=act), sp.dense_fwd(x[:1], w, bias=b, act=act))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,do", [(3, 72, 40), (5, 72, 40), (40, 72, 40), (700, 72, 40), (40000, 72, 40),
                                     (700, 64, 40), (40000, 50, 33), (900, 300, 200)])
def test_infinities_and_nan(n, di, do, dtype):
    """They come through as the formula has them, and stay in their row,
    column or sum."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dense: infinities and NaN n={n} {di} {do} {dtype}")
    x, w, b, res, g = case(n, di, do, dtype, 3)
    clean, cgx = sp.dense_fwd(x, w, bias=b), sp.dense_bwd(x, w, g, bias=b)
    for bad in (float("inf"), float("nan")):
        y = x.clone()
        y[2, 5] = bad
        out = sp.dense_fwd(y, w, bias=b)
        want = y.double()[2] @ w.double().T + b.double()
        assert torch.equal(torch.isnan(out[2]), torch.isnan(want)) and torch.equal(torch.isinf(out[2]), torch.isinf(want))
        assert torch.equal(out[2][torch.isinf(want)].sign(), want[torch.isinf(want)].to(out.dtype).sign())
        keep = torch.arange(n, device="cuda") != 2
        assert torch.equal(out[keep], clean[keep])
        dx, dw, db = sp.dense_bwd(y, w, g, bias=b)
        assert torch.equal(dx, cgx[0]) and torch.equal(db, cgx[2])
        cols = torch.arange(di, device="cuda") != 5
        assert torch.equal(dw[:, cols], cgx[1][:, cols]) and not torch.isfinite(dw[:, 5]).any()
        h = g.clone()
        h[1, 3] = bad
        dx, dw, db = sp.dense_bwd(x, w, h, bias=b, act="relu")
        ref = sp.dense_bwd(x, w, g, bias=b, act="relu")
        keep = torch.arange(n, device="cuda") != 1
        assert torch.equal(dx[keep], ref[0][keep])
        rows = torch.arange(do, device="cuda") != 3
        if dtype != "f16":  # a block's power of two may change with its largest value
            assert torch.equal(dw[rows], ref[1][rows])
        assert torch.equal(db[rows], ref[2][rows])
        assert not torch.isfinite(db[3]) and not torch.isfinite(dw[3]).any()  # an infinity times a slope of zero is NaN


@pytest.mark.parametrize("scale", [2.0 ** -22, 2.0 ** -14, 2.0 ** 8])
@pytest.mark.parametrize("act", ["gelu", "sigmoid"])
@pytest.mark.parametrize("n,di,do", [(40, 72, 136), (3000, 130, 300), (3, 72, 136), (20000, 60, 64), (70, 9000, 64)])
def test_float16_range(n, di, do, act, scale):
    """Gradients at the ends of float16's range: the gradient before the
    activation, which may be past them, keeps its 11 bits."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dense: float16 gradients of about {scale} {act} n={n}")
    x, w, b, res, g = case(n, di, do, "f16", 5)
    g = (g.float().clamp(-4, 4) * scale).half()
    x = (x.float() * (1 if scale < 1 else 2.0 ** -6)).half()
    w = (w.float() * (1 if scale < 1 else 2.0 ** -3)).half()
    b = b * 4 - 2  # slopes below one
    # the bound of a held value's error: half a step of 11 bits, small ones 2^-16 of the block's largest
    _, grads = reference(x, w, b, None, g, act, "f16")
    d = g.double() * act64(x.double() @ w.double().T + b.double(), act)[1]
    got = sp.dense_bwd(x, w, g, bias=b, act=act)
    for name, a, (r, e), k in zip(("grad_x", "grad_w", "grad_bias"), got, grads, (do, n, n)):
        rms = ((a.double() - r).square().mean().sqrt()).item()
        # a rounding of d (2^-11 / sqrt 3 of each), one of the store, and a subnormal store's 2^-25
        size = r.square().mean().sqrt().item()
        assert rms <= 2 * 2.0 ** -11 * size + 2.0 ** -25, (name, rms, size)


def test_float32_accuracy():
    """Root mean square errors are those of float32 sums: an addition is off
    by 0.41 2^-24 of its result, a sum of K random terms by 0.29 sqrt(K) 2^-24
    of its own size; half sqrt(K) 2^-24 is allowed for each sum in the chain and
    6 2^-24 for activation, products and roundings."""
    need_gpu()
    import segmented_polynomials_amd as sp
    for n, di, do in ((3, 333, 1001), (5, 333, 1001), (33, 2048, 96), (300, 512, 512), (60000, 64, 64), (700, 96, 1500),
                      (4000, 300, 300)):
        announce(f"dense: float32 accuracy {n} {di} {do}")
        x, w, b, res, g = case(n, di, do, "f32", 7)
        (out, _), grads = reference(x, w, b, None, g, "silu", "f32")
        got = (sp.dense_fwd(x, w, bias=b, act="silu"), *sp.dense_bwd(x, w, g, bias=b, act="silu"))
        for name, a, r, sums in zip(("out", "grad_x", "grad_w", "grad_bias"), got, (out, *(v for v, _ in grads)),
                                    ((di,), (di, do), (di, n), (di, n))):
            rms = ((a.double() - r).square().mean().sqrt() / r.square().mean().sqrt()).item() / E24
            lim = 6 + 0.5 * sum(math.sqrt(k) for k in sums)
            print(f"[parity] {name}: {rms:.2f} of 2^-24, allowed {lim:.2f}", flush=True)
            assert rms <= lim, name


def test_float32_range():
    """Values past the largest bf16 and far below one keep float32's accuracy."""
    need_gpu()
    import segmented_polynomials_amd as sp
    for n in (20, 3000):
        announce(f"dense: float32 range n={n}")
        x, w, b, res, g = case(n, 64, 64, "f32", 9)
        big = torch.finfo(torch.float32).max
        x[0, 0] = big
        w[:, 0] = 1e-39
        x[1] *= 1e-12
        (out, eout), _ = reference(x, w, b, None, g, "none", "f32")
        # planes below the smallest normal bf16 lose their last bits: 2^-133 of |x| each
        check(sp.dense_fwd(x, w, bias=b), out, eout + big * 2.0 ** -133 * 64, "f32", "out")


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
def test_gradients_against_differences(act):
    """The gradient against central differences of the forward, float32, in a
    random direction, the loss in float64; truncation is of the third
    derivative."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dense: gradients against differences {act}")
    n, di, do = 40, 48, 24
    x, w, b, res, g = case(n, di, do, "f32", 12)
    p = dict(x=x, w=w, bias=b)

    def loss(q):
        out = sp.dense_fwd(q["x"], q["w"], bias=q["bias"], act=act, residual=res)
        return (out.double() * g.double()).sum().item()

    grads = dict(zip(("x", "w", "bias"), sp.dense_bwd(x, w, g, bias=b, act=act)))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for name in p:
        v = torch.randn(p[name].shape, generator=gen, device="cuda")
        v /= v.norm()
        slope = (grads[name].double() * v.double()).sum().item()
        d1, d2 = ((loss({**p, name: p[name] + e * v}) - loss({**p, name: p[name] - e * v})) / (2 * e)
                  for e in (2.0 ** -6, 2.0 ** -7))
        noise = E24 * math.sqrt(n * do) * 8 * 2.0 ** 7
        assert abs(slope - (4 * d2 - d1) / 3) <= noise + abs(d1 - d2) + 1e-4 * abs(slope), name


@pytest.mark.parametrize("n,di,do,dtype", [(700, 64, 130, "bf16"), (9, 200, 40, "f16"), (20000, 64, 64, "f32")])
def test_graph_replays_and_side_stream(n, di, do, dtype):
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dense: captured into a graph {n} {di} {do} {dtype}")
    x, w, b, res, g = case(n, di, do, dtype, 4)

    def step():
        h = sp.dense_fwd(x, w, bias=b, act="silu", residual=res)
        return [h, *sp.dense_bwd(x, w, g, bias=b, act="silu"), *sp.dense_bwd(x, w, h, bias=b)]

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(other, step()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for r in range(3):
        y, *_, h = case(n, di, do, dtype, 50 + r)
        x.copy_(y)
        g.copy_(h)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(captured, step()))


@pytest.mark.parametrize("n,di,do,dtype,stride", [(1100, 64, 40, "f32", 1 << 21), (1100, 64, 72, "f32", 1 << 21),
                                                  (1100, 520, 72, "f32", 1 << 21), (1100, 72, 520, "bf16", 1 << 21),
                                                  (1100, 520, 72, "f16", 1 << 21), (12300, 64, 64, "bf16", 180000)])
def test_rows_past_32_bits_of_elements(n, di, do, dtype, stride):
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dense: rows {stride} elements apart {n} {di} {do} {dtype}")
    x, w, b, res, g = case(n, di, do, dtype, 4)
    out = sp.dense_fwd(x, w, bias=b, act="silu", residual=res)
    full = sp.dense_bwd(x, w, g, bias=b, act="silu")
    held = torch.empty(n * stride, dtype=T[dtype], device="cuda")
    assert held.numel() > 2 ** 31

    def apart(t, at):
        v = torch.as_strided(held, t.shape, (stride, 1), at)
        v.copy_(t)
        return v

    far, to = apart(x, 0), apart(res, 1024)
    sp.dense_fwd(far, w, bias=b, act="silu", residual=to, out=to)
    assert torch.equal(to, out)
    got = sp.dense_bwd(far, w, apart(g, 2048), bias=b, act="silu")
    assert all(torch.equal(p, q) for p, q in zip(got, full))
