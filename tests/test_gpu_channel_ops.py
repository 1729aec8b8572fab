"""GPU parity of the invariant-channel operators (embedding, block norm, gated
feed-forward, each with its backward) through the C ABI, against their
definitions in float64 evaluated by plain tensor operations.

Tolerances are bounds carried through the definition beside the value: every
sum of K terms evaluated in float32 is off by at most about K 2^-24 of the sum
of its absolute terms, every store by half a step of its type (HALF)."""

import math

import pytest
import torch

from tests._gpu import announce, need_gpu

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {k: torch.finfo(v).eps / 2 for k, v in T.items()}
# below the smallest normal number a step no longer shrinks with the value
TINY = {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -24}
E24 = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, std=1.0, dtype="f32"):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(T[dtype])


def check(got, ref, bound, dtype, what):
    assert torch.isfinite(got).all(), what
    off = (got.double() - ref).abs()
    lim = bound + HALF[dtype] * (ref.abs() + bound) + TINY[dtype]
    worst = (off / lim).max().item() if off.numel() else 0.0
    print(f"[parity] {what}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, f"{what}: {worst:.3f} times the bound"


# ------------------------------------------------------------------ embedding

EMB = [(0, 5, 8), (1, 1, 1), (5, 3, 33), (257, 10, 128), (4096, 7, 70), (4097, 300, 64), (9000, 2500, 257),
       (20000, 1500, 40), (12289, 70000, 24), (600, 4000, 2056)]


def tokens_of(g, n, rows, idx):
    """Ids with a heavy head, some out of range on both sides."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    t = (u ** 3 * rows).long().clamp_(0, rows - 1)
    bad = torch.rand(n, generator=g, device="cuda")
    t = torch.where(bad < 0.02, torch.full_like(t, -1), t)
    t = torch.where((bad > 0.98), torch.full_like(t, rows), t)
    return t.to(idx)


@pytest.mark.parametrize("idx", [torch.int32, torch.int64])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,rows,dim", EMB)
def test_embedding(n, rows, dim, dtype, idx):
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"embedding n={n} rows={rows} dim={dim} {dtype} {idx}")
    g = gen(n + rows + dim)
    scale = 1.7
    s32 = torch.tensor(scale, dtype=torch.float32).double().item()
    tok = tokens_of(g, n, rows, idx)
    table, grad = rnd(g, rows, dim, dtype=dtype), rnd(g, n, dim, dtype=dtype)
    ok = (tok >= 0) & (tok < rows)
    at = tok.long().clamp(0, rows - 1)
    out = sp.embedding_fwd(table, tok, scale=scale)
    ref = table.double()[at] * s32 * ok[:, None]
    check(out, ref, E24 * ref.abs(), dtype, "out")
    # columns of a wider tensor, the others untouched
    wide = torch.full((n, dim + 5), 3.0, dtype=T[dtype], device="cuda")
    sp.embedding_fwd(table, tok, scale=scale, out=wide[:, 2:2 + dim])
    assert torch.equal(wide[:, 2:2 + dim], out) and bool((wide[:, :2] == 3).all()) and bool((wide[:, 2 + dim:] == 3).all())
    d = sp.embedding_bwd(grad, tok, rows, scale=scale)
    src = grad.double() * s32 * ok[:, None]
    ref = torch.zeros(rows, dim, dtype=torch.float64, device="cuda").index_add_(0, at, src)
    mag = torch.zeros(rows, dim, dtype=torch.float64, device="cuda").index_add_(0, at, src.abs())
    count = torch.zeros(rows, dtype=torch.float64, device="cuda").index_add_(0, at, ok.double())
    check(d, ref, (count[:, None] + 2) * E24 * mag, dtype, "grad_table")
    wideg = torch.zeros(n, dim + 3, dtype=T[dtype], device="cuda")
    wideg[:, 1:1 + dim] = grad
    assert torch.equal(sp.embedding_bwd(wideg[:, 1:1 + dim], tok, rows, scale=scale), d)  # strides, and the same bits


def test_embedding_one_row_and_no_valid_token():
    need_gpu()
    import segmented_polynomials_amd as sp
    n, rows, dim = 10000, 40, 64
    g = gen(5)
    grad = rnd(g, n, dim)
    tok = torch.full((n,), 17, dtype=torch.int32, device="cuda")
    announce("embedding: every token the same")
    d = sp.embedding_bwd(grad, tok, rows)
    ref = torch.zeros(rows, dim, dtype=torch.float64, device="cuda")
    ref[17] = grad.double().sum(0)
    mag = torch.zeros_like(ref)
    mag[17] = grad.double().abs().sum(0)
    check(d, ref, (n + 2) * E24 * mag, "f32", "one row")
    announce("embedding: no token in range")
    assert not sp.embedding_bwd(grad, torch.full_like(tok, rows), rows).any()
    assert not sp.embedding_fwd(rnd(g, rows, dim), torch.full_like(tok, -3)).any()


# ------------------------------------------------------------------ block norm

def norm64(v, kind, eps):
    m = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    c = v - m
    r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    # absolute companion: the centred value's operands
    a = (v.abs() + (v.abs().mean(1, keepdim=True) if kind == "layer" else 0)) * r
    return c * r, r, a


def nvjp64(q, nv, r, kind):
    d = q - nv * (q * nv).mean(1, keepdim=True)
    return (d - q.mean(1, keepdim=True) if kind == "layer" else d) * r


def nvjp_abs(q, na, r, kind):
    d = q + na * (q * na).mean(1, keepdim=True)
    return (d + q.mean(1, keepdim=True) if kind == "layer" else d) * r


# A row's statistics take at most 16 + 10 additions in a chain and a value of
# the backward passes three of them, a dozen products and a sigmoid (a few
# 2^-22): 2^-16 of the absolute companion is above all of them together.
NORM_F32 = 2.0 ** -16


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,dim,kind,gate,act,scale,nxt", [
    (1, 1, "rms", "element", "none", True, True),
    (1, 8, "layer", "row", "sigmoid", True, True),
    (3, 33, "rms", "row", "none", False, True),
    (70, 128, "layer", "element", "sigmoid", True, True),
    (37, 200, "layer", "none", "none", True, False),
    (65, 511, "rms", "element", "sigmoid", True, True),
    (5, 1000, "rms", "none", "none", True, True),
    (300, 1030, "layer", "row", "sigmoid", False, False),
    (9, 2047, "layer", "element", "none", True, True),
    (1200, 2048, "rms", "element", "sigmoid", True, True),
    (6, 4099, "rms", "row", "sigmoid", True, True),
    (4, 8192, "layer", "element", "sigmoid", True, True),
    (3, 16383, "layer", "element", "sigmoid", True, True),
    (2500, 130, "rms", "row", "sigmoid", True, True),
])
def test_block_norm(n, dim, kind, gate, act, scale, nxt, dtype):
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"block norm n={n} dim={dim} {kind} gate={gate}/{act} scale={scale} next={nxt} {dtype}")
    g = gen(n * 7 + dim)
    eps = 1e-5
    x, f, gy, gh = rnd(g, n, dim, dtype=dtype), rnd(g, n, dim, std=0.6, dtype=dtype), rnd(g, n, dim, dtype=dtype), \
        rnd(g, n, dim, dtype=dtype)
    f[n // 2] = 0  # a row of zeros: norm 0, gradient through 1 / sqrt(eps)
    gt = None if gate == "none" else rnd(g, n, 1 if gate == "row" else dim, dtype=dtype)
    wp = 1 + rnd(g, dim, std=0.1)
    rs = 0.5 + rnd(g, dim, std=0.1) if scale else None
    wn = 1 + rnd(g, dim, std=0.1) if nxt else None
    kw = dict(f=f, gate=gt, w_post=wp, res_scale=rs, w_pre=wn, kind=kind, gate_act=act, eps=eps)
    e32 = torch.tensor(eps, dtype=torch.float32).double().item()

    nf, rf, nfa = norm64(f.double(), kind, e32)
    s = torch.ones(1, dim, dtype=torch.float64, device="cuda") if rs is None else rs.double()
    if gt is None:
        G, dact = torch.ones(n, 1, dtype=torch.float64, device="cuda"), None
    else:
        G = gt.double()
        dact = torch.ones_like(G)
        if act == "sigmoid":
            G = torch.sigmoid(G)
            dact = G * (1 - G)
    v, va = nf * wp.double(), nfa * wp.double().abs()
    y64 = x.double() + s * G * v
    ya = x.double().abs() + (s * G).abs() * va
    y, h = sp.block_norm_fwd(x, **kw)
    check(y, y64, NORM_F32 * ya, dtype, "y")
    if nxt:
        ny, ry, _ = norm64(y64, kind, e32)
        na = (ya + (ya.mean(1, keepdim=True) if kind == "layer" else 0)) * ry
        # the second norm sees y's own error, and its statistic the whole row's
        na = na + ny.abs() * (ny.abs() * na).mean(1, keepdim=True)
        check(h, ny * wn.double(), 2 * NORM_F32 * na * wn.double().abs(), dtype, "h")
    else:
        assert h is None

    # backward, from the stored y
    Y = y.double()
    dy, dya = gy.double(), gy.double().abs()
    if nxt:
        ny, ry, nya = norm64(Y, kind, e32)
        q = gh.double() * wn.double()
        dy = dy + nvjp64(q, ny, ry, kind)
        dya = dya + nvjp_abs(q.abs(), nya, ry, kind)
        dpre, dprea = (gh.double() * ny).sum(0), (gh.double().abs() * nya).sum(0)
    else:
        dpre = None
    got = sp.block_norm_bwd(y, gy, gh if nxt else None, **kw)
    p, pa = dy * s * G * wp.double(), dya * (s * G).abs() * wp.double().abs()
    ref = [(dy, dya), (nvjp64(p, nf, rf, kind), nvjp_abs(pa, nfa, rf, kind)), None,
           ((dy * s * G * nf).sum(0), (dya * (s * G).abs() * nfa).sum(0)),
           None if rs is None else ((dy * G * v).sum(0), (dya * G.abs() * va).sum(0)),
           None if wn is None else (dpre, dprea)]
    if gt is not None:
        dg, dga = dy * s * v * dact, dya * s.abs() * va * dact.abs()
        # s (1 - s) of a saturated sigmoid keeps the absolute error of s
        dga = dga + dya * s.abs() * va * (2.0 ** -6 if act == "sigmoid" else 0)
        ref[2] = (dg.sum(1, keepdim=True), dga.sum(1, keepdim=True)) if gate == "row" and dim > 1 else (dg, dga)
    names = ("grad_x", "grad_f", "grad_gate", "grad_w_post", "grad_res_scale", "grad_w_pre")
    for i, (name, r) in enumerate(zip(names, ref)):
        if r is None:
            assert got[i] is None
        else:
            check(got[i], r[0], NORM_F32 * r[1], dtype if i < 3 else "f32", name)
    again = sp.block_norm_bwd(y, gy, gh if nxt else None, **kw)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


def test_block_norm_strides_and_empty():
    need_gpu()
    import segmented_polynomials_amd as sp
    g = gen(3)
    n, d = 45, 96
    wide = rnd(g, n, 4 * d, dtype="bf16")
    x, f = wide[:, :d], wide[:, d + 1:2 * d + 1]
    row = rnd(g, 1, d, dtype="bf16").expand(n, d)  # one gate row read by every row
    wp = 1 + rnd(g, d, std=0.1)
    announce("block norm on columns of a wider tensor")
    y, h = sp.block_norm_fwd(x, f, wp, gate=row, w_pre=wp)
    y2, h2 = sp.block_norm_fwd(x.contiguous(), f.contiguous(), wp, gate=row.contiguous(), w_pre=wp)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    a = sp.block_norm_bwd(x, f, wide[:, :d], f, wp, gate=row, w_pre=wp)
    b = sp.block_norm_bwd(*(t.contiguous() for t in (x, f, x, f)), wp, gate=row.contiguous(), w_pre=wp)
    assert all(p is None and q is None or torch.equal(p, q) for p, q in zip(a, b))
    announce("block norm without rows")
    e = torch.empty(0, d, device="cuda")
    y, h = sp.block_norm_fwd(e, e, wp, w_pre=wp)
    assert y.shape == (0, d) and h.shape == (0, d)
    grads = sp.block_norm_bwd(e, e, e, e, wp, w_pre=wp, res_scale=wp)
    assert not grads[3].any() and not grads[4].any() and not grads[5].any()


# ------------------------------------------------------------------ gated feed-forward

def act64(g, act):
    """Value, derivative, and a bound of the second derivative."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s)), 0.5
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi), 0.8
    if act == "relu":
        return g.clamp_min(0), (g > 0).double(), 0.0
    s = torch.sigmoid(g)
    return s, s * (1 - s), 0.1


def ffn_reference(x, wg, wu, wd, gy, act, dtype):
    """Values and error bounds of the forward and the backward."""
    half = HALF[dtype] if dtype != "f32" else 2 * E24  # what is held between the products
    x, wg, wu, wd, gy = (t.double() for t in (x, wg, wu, wd, gy))
    s = lambda k: (k + 64) * E24   # a float32 sum of k terms
    di, F, do, n = x.shape[1], wg.shape[0], wd.shape[0], x.shape[0]
    g, u = x @ wg.T, x @ wu.T
    eg, eu = s(di) * (x.abs() @ wg.abs().T), s(di) * (x.abs() @ wu.abs().T)
    a, da, d2 = act64(g, act)
    fast = 2.0 ** -18  # exp and erf in float32: a few units of 2^-23 and 2^-24 |g|, |g| < 64 here
    ea = 1.13 * eg + fast * a.abs() + fast * E24
    eda = d2 * eg + fast
    if act == "relu":
        ea, eda = eg, (g.abs() <= eg).double()  # the step may fall on the other side
    h = a * u
    eh = ea * u.abs() + a.abs() * eu + ea * eu
    eh = eh + half * (h.abs() + eh) + TINY[dtype]
    out = h @ wd.T
    eout = eh @ wd.abs().T + s(F) * (h.abs() @ wd.abs().T)
    dh = gy @ wd
    edh = s(do) * (gy.abs() @ wd.abs())
    edh = edh + half * (dh.abs() + edh) + TINY[dtype]
    dg, du = dh * u * da, dh * a
    edg = edh * (u * da).abs() + dh.abs() * (eu * da.abs() + (u.abs() + eu) * eda) + edh * (eu + eda)
    edu = edh * a.abs() + dh.abs() * ea + edh * ea
    edg = edg + half * (dg.abs() + edg) + TINY[dtype]
    edu = edu + half * (du.abs() + edu) + TINY[dtype]
    dx = dg @ wg + du @ wu
    edx = edg @ wg.abs() + edu @ wu.abs() + s(2 * F) * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
    dwg, dwu, dwd = dg.T @ x, du.T @ x, gy.T @ h
    ewg = edg.T @ x.abs() + s(n) * (dg.abs().T @ x.abs())
    ewu = edu.T @ x.abs() + s(n) * (du.abs().T @ x.abs())
    ewd = gy.abs().T @ eh + s(n) * (gy.abs().T @ h.abs())
    return (out, eout), ((dx, edx), (dwg, ewg), (dwu, ewu), (dwd, ewd))


def ffn_case(n, di, F, do, dtype, seed):
    g = gen(seed)
    return (rnd(g, n, di, dtype=dtype), rnd(g, F, di, std=di ** -0.5, dtype=dtype),
            rnd(g, F, di, std=di ** -0.5, dtype=dtype), rnd(g, do, F, std=F ** -0.5, dtype=dtype),
            rnd(g, n, do, dtype=dtype))


FFN = [(1, 8, 8, 8), (1, 1, 1, 1), (3, 64, 128, 64), (16, 72, 136, 40), (17, 61, 67, 35), (65, 128, 256, 96),
       (130, 322, 853, 257), (300, 200, 520, 328), (1, 1024, 640, 512), (5, 333, 1001, 77), (33, 2048, 96, 2048),
       (700, 64, 64, 64)]


@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,F,do", FFN)
def test_gated_ffn(n, di, F, do, dtype, act):
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated ffn n={n} d_in={di} hidden={F} d_out={do} {dtype} {act}")
    x, wg, wu, wd, gy = ffn_case(n, di, F, do, dtype, n + di + F + do)
    (out, eout), grads = ffn_reference(x, wg, wu, wd, gy, act, dtype)
    check(sp.gated_ffn_fwd(x, wg, wu, wd, act=act), out, eout, dtype, "out")
    got = sp.gated_ffn_bwd(x, wg, wu, wd, gy, act=act)
    for name, a, (r, e) in zip(("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down"), got, grads):
        check(a, r, e, dtype, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,F,do", [(4096, 72, 2048, 64), (2048, 4096, 136, 4096), (4100, 1030, 1032, 1100)])
def test_gated_ffn_large_tiles(n, di, F, do, dtype):
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated ffn, large tiles n={n} d_in={di} hidden={F} d_out={do} {dtype}")
    x, wg, wu, wd, gy = ffn_case(n, di, F, do, dtype, 11)
    (out, eout), grads = ffn_reference(x, wg, wu, wd, gy, "silu", dtype)
    check(sp.gated_ffn_fwd(x, wg, wu, wd), out, eout, dtype, "out")
    got = sp.gated_ffn_bwd(x, wg, wu, wd, gy)
    for name, a, (r, e) in zip(("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down"), got, grads):
        check(a, r, e, dtype, name)
    assert all(torch.equal(p, q) for p, q in zip(got, sp.gated_ffn_bwd(x, wg, wu, wd, gy)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gated_ffn_strides_parts_and_empty(dtype):
    need_gpu()
    import segmented_polynomials_amd as sp
    n, di, F, do = 90, 64, 136, 48
    x, wg, wu, wd, gy = ffn_case(n, di, F, do, dtype, 2)
    announce(f"gated ffn on columns of wider tensors {dtype}")
    out = sp.gated_ffn_fwd(x, wg, wu, wd)
    full = sp.gated_ffn_bwd(x, wg, wu, wd, gy)
    for shift in (8, 3):  # the second leaves rows off 16 bytes
        wide = torch.full((n, di + 40), float("nan"), dtype=T[dtype], device="cuda")
        wide[:, shift:shift + di] = x
        wideg = torch.full((n, do + 40), float("nan"), dtype=T[dtype], device="cuda")
        wideg[:, shift:shift + do] = gy
        to = torch.full((n, do + 9), 5.0, dtype=T[dtype], device="cuda")
        sp.gated_ffn_fwd(wide[:, shift:shift + di], wg, wu, wd, out=to[:, 4:4 + do])
        assert torch.equal(to[:, 4:4 + do], out) and bool((to[:, :4] == 5).all()) and bool((to[:, 4 + do:] == 5).all())
        got = sp.gated_ffn_bwd(wide[:, shift:shift + di], wg, wu, wd, wideg[:, shift:shift + do])
        assert all(torch.equal(a, b) for a, b in zip(got, full))
    announce("gated ffn: parts of the backward, no rows")
    only = sp.gated_ffn_bwd(x, wg, wu, wd, gy, need_dw=False)
    assert torch.equal(only[0], full[0]) and only[1] is None
    only = sp.gated_ffn_bwd(x, wg, wu, wd, gy, need_dx=False)
    assert only[0] is None and torch.equal(only[3], full[3])
    none = sp.gated_ffn_bwd(x[:0], wg, wu, wd, gy[:0])
    assert none[0].shape == (0, di) and not any(t.any() for t in none[1:])
    assert sp.gated_ffn_fwd(x[:0], wg, wu, wd).shape == (0, do)


def test_gated_ffn_float32_range():
    """Values past the largest bf16 and far below one keep float32's accuracy."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce("gated ffn float32 range")
    x, wg, wu, wd, gy = ffn_case(20, 64, 64, 64, "f32", 9)
    big = torch.finfo(torch.float32).max
    x[0, 0] = big
    wg[:, 0] = 1e-39
    wu[:, 0] = 0
    x[1] *= 1e-12
    (out, eout), _ = ffn_reference(x, wg, wu, wd, gy, "relu", "f32")
    # planes below the smallest normal bf16 lose their last bits: 2^-133 of |x| each
    eout = eout + big * 2.0 ** -133 * 64
    check(sp.gated_ffn_fwd(x, wg, wu, wd, act="relu"), out, eout, "f32", "out")


def test_gradients_against_differences():
    """The backward of the three operators together against central
    differences of the forward: a tiny network, float32, step 2^-6 in a random
    direction, the loss in float64.  Truncation is of the third derivative."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce("gradients against differences")
    g = gen(12)
    n, rows, d, F = 24, 5, 32, 48
    tok = torch.randint(0, rows, (n,), generator=g, device="cuda", dtype=torch.int32)
    p = dict(table=rnd(g, rows, d), wg=rnd(g, F, d, std=d ** -0.5), wu=rnd(g, F, d, std=d ** -0.5),
             wd=rnd(g, d, F, std=F ** -0.5), post=1 + rnd(g, d, std=0.1), pre=1 + rnd(g, d, std=0.1),
             scale=0.5 + rnd(g, d, std=0.1), gate=rnd(g, n, 1))
    cy, ch = rnd(g, n, d), rnd(g, n, d)
    kw = lambda q: dict(gate=q["gate"], w_post=q["post"], res_scale=q["scale"], w_pre=q["pre"], kind="layer",
                        gate_act="sigmoid")

    def loss(q):
        x = sp.embedding_fwd(q["table"], tok, scale=2.0)
        f = sp.gated_ffn_fwd(x, q["wg"], q["wu"], q["wd"])
        y, h = sp.block_norm_fwd(x, f, **kw(q))
        return ((y.double() * cy.double()).sum() + (h.double() * ch.double()).sum()).item()

    x = sp.embedding_fwd(p["table"], tok, scale=2.0)
    f = sp.gated_ffn_fwd(x, p["wg"], p["wu"], p["wd"])
    y, _ = sp.block_norm_fwd(x, f, **kw(p))
    dx, df, dgate, dpost, dscale, dpre = sp.block_norm_bwd(y, cy, ch, f, **kw(p))
    dx2, dwg, dwu, dwd = sp.gated_ffn_bwd(x, p["wg"], p["wu"], p["wd"], df)
    grads = dict(table=sp.embedding_bwd(dx + dx2, tok, rows, scale=2.0), wg=dwg, wu=dwu, wd=dwd, post=dpost, pre=dpre,
                 scale=dscale, gate=dgate)
    for name in p:
        v = torch.randn(p[name].shape, generator=g, device="cuda")
        v /= v.norm()
        slope = (grads[name].double() * v.double()).sum().item()
        d1, d2 = ((loss({**p, name: p[name] + e * v}) - loss({**p, name: p[name] - e * v})) / (2 * e)
                  for e in (2.0 ** -6, 2.0 ** -7))
        extrapolated = (4 * d2 - d1) / 3
        # half a step of n d float32 outputs near one, added at random: 2^-24 sqrt(2 n d) 2 over the step
        noise = E24 * math.sqrt(2 * n * d) * 8 * 2.0 ** 7
        bound = noise + abs(d1 - d2) + 1e-4 * abs(slope)
        print(f"[parity] d {name}: {slope:.6f} differences {extrapolated:.6f} bound {bound:.2e}", flush=True)
        assert abs(slope - extrapolated) <= bound


def test_graph_replays_and_side_stream():
    """Every operator captured into one graph; three replays with new inputs
    and eager work between them give the eager results' bits, and so does a
    call on another stream."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce("channel operators captured into a graph")
    g = gen(1)
    n, rows, d, F = 300, 5000, 64, 160
    tok = torch.randint(-1, rows, (n,), generator=g, device="cuda", dtype=torch.int64)
    table, wg, wu, wd = rnd(g, rows, d, dtype="bf16"), *(rnd(g, *s, std=0.1, dtype="bf16") for s in
                                                        ((F, d), (F, d), (d, F)))
    w = 1 + rnd(g, d, std=0.1)
    gy = rnd(g, n, d, dtype="bf16")

    def step():
        x = sp.embedding_fwd(table, tok, scale=3.0)
        f = sp.gated_ffn_fwd(x, wg, wu, wd)
        y, h = sp.block_norm_fwd(x, f, w, res_scale=w, w_pre=w)
        grads = sp.block_norm_bwd(y, gy, h, f, w, res_scale=w, w_pre=w)
        ffn = sp.gated_ffn_bwd(x, wg, wu, wd, grads[1])
        return [y, h, *(t for t in grads if t is not None), *ffn, sp.embedding_bwd(grads[0], tok, rows, scale=3.0)]

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, step()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for r in range(3):
        tok.copy_(torch.randint(-1, rows, (n,), generator=gen(r), device="cuda", dtype=torch.int64))
        gy.copy_(rnd(gen(r + 50), n, d, dtype="bf16"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, step()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,rows,dim", [(3000, 16, 2056), (50001, 10, 128), (700, 2, 9), (16384, 17, 33),
                                        (16385, 65536, 40), (40000, 5000, 24), (15000, 30000, 1032), (5, 4, 4097)])
def test_embedding_gradient_variants(n, rows, dim, dtype):
    """Tables summed in LDS (at most 16 rows; several column tiles), the list
    sorted by one workgroup and by several, ranges with and without whole chunks."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"embedding gradient n={n} rows={rows} dim={dim} {dtype}")
    g = gen(n + 3 * rows + dim)
    tok, grad = tokens_of(g, n, rows, torch.int64), rnd(g, n, dim, dtype=dtype)
    ok = (tok >= 0) & (tok < rows)
    at, src = tok.clamp(0, rows - 1), grad.double() * ok[:, None]
    ref = torch.zeros(rows, dim, dtype=torch.float64, device="cuda").index_add_(0, at, src)
    mag = torch.zeros(rows, dim, dtype=torch.float64, device="cuda").index_add_(0, at, src.abs())
    count = torch.zeros(rows, dtype=torch.float64, device="cuda").index_add_(0, at, ok.double())
    d = sp.embedding_bwd(grad, tok, rows)
    check(d, ref, (count[:, None] + 2) * E24 * mag, dtype, "grad_table")
    assert torch.equal(sp.embedding_bwd(grad, tok, rows), d)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,F,do", [(1, 2048, 5632, 2048), (16, 70, 33, 130), (31, 129, 1000, 15), (64, 515, 77, 64),
                                       (40, 5, 3, 2)])
def test_gated_ffn_few_rows(n, di, F, do, dtype):
    """The form of at most 64 rows, with rows off 16 bytes, one row read by
    all, and untouched neighbours of the output."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated ffn, few rows n={n} d_in={di} hidden={F} d_out={do} {dtype}")
    x, wg, wu, wd, gy = ffn_case(n, di, F, do, dtype, n + di)
    (out, eout), _ = ffn_reference(x, wg, wu, wd, gy, "gelu", dtype)
    got = sp.gated_ffn_fwd(x, wg, wu, wd, act="gelu")
    check(got, out, eout, dtype, "out")
    wide = torch.full((n, di + 7), float("nan"), dtype=T[dtype], device="cuda")
    wide[:, 3:3 + di] = x
    to = torch.full((n, do + 9), 5.0, dtype=T[dtype], device="cuda")
    sp.gated_ffn_fwd(wide[:, 3:3 + di], wg, wu, wd, act="gelu", out=to[:, 4:4 + do])
    assert torch.equal(to[:, 4:4 + do], got) and bool((to[:, :4] == 5).all()) and bool((to[:, 4 + do:] == 5).all())
    one = sp.gated_ffn_fwd(x[:1].expand(n, di), wg, wu, wd, act="gelu")
    assert torch.equal(one, got[:1].expand(n, do))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,F,do", [(70, 200, 3001, 65), (66, 1030, 2052, 30), (5000, 65, 70, 33), (9, 64, 4000, 700),
                                       (300, 20, 8000, 640)])
def test_gated_ffn_long_sums(n, di, F, do, dtype):
    """Products of few tiles whose long sums are shared out and added."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated ffn, long sums n={n} d_in={di} hidden={F} d_out={do} {dtype}")
    x, wg, wu, wd, gy = ffn_case(n, di, F, do, dtype, n + F)
    (out, eout), grads = ffn_reference(x, wg, wu, wd, gy, "silu", dtype)
    check(sp.gated_ffn_fwd(x, wg, wu, wd), out, eout, dtype, "out")
    got = sp.gated_ffn_bwd(x, wg, wu, wd, gy)
    for name, a, (r, e) in zip(("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down"), got, grads):
        check(a, r, e, dtype, name)
    assert all(torch.equal(p, q) for p, q in zip(got, sp.gated_ffn_bwd(x, wg, wu, wd, gy)))
