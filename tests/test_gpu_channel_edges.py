"""GPU tests of the invariant-channel operators at the ends of their ranges:
eps of zero, empty calls, single rows of any stride, values outside the element
type's range between products, infinities and NaN, the limits of the embedding
gradient's ordering, and the accuracy that the forms promise.  Tolerances as in
``test_gpu_channel_ops``, whose references are used where they fit."""

import pytest
import torch

from tests import _ffn_accuracy as acc
from tests._gpu import announce, need_gpu
from tests.test_gpu_channel_ops import (E24, NORM_F32, T, act64, check, ffn_case, ffn_reference, gen, norm64,
                                        nvjp64, nvjp_abs, rnd, tokens_of)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ block norm

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "row", "element"])
@pytest.mark.parametrize("n,dim,nxt", [(1, 64, True), (3, 33, True), (37, 64, False), (37, 200, True), (5, 511, True),
                                       (37, 1000, True), (1, 1000, False)])
def test_block_norm_without_eps(n, dim, nxt, gate, kind, dtype):
    """eps = 0, numbers of rows that are no multiple of a workgroup's: what
    stands past the last row takes no part in the parameters' gradients."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"block norm, eps 0, n={n} dim={dim} {kind} gate={gate} next={nxt} {dtype}")
    g = gen(n + dim)
    x, f, gy, gh = (rnd(g, n, dim, dtype=dtype) for _ in range(4))
    gt = None if gate == "none" else rnd(g, n, 1 if gate == "row" else dim, dtype=dtype)
    wp, rs = 1 + rnd(g, dim, std=0.1), 0.5 + rnd(g, dim, std=0.1)
    wn = 1 + rnd(g, dim, std=0.1) if nxt else None
    kw = dict(f=f, gate=gt, w_post=wp, res_scale=rs, w_pre=wn, kind=kind, eps=0.0)
    nf, rf, nfa = norm64(f.double(), kind, 0.0)
    s = rs.double()
    G = torch.ones(n, 1, dtype=torch.float64, device="cuda") if gt is None else gt.double()
    v, va = nf * wp.double(), nfa * wp.double().abs()
    y, _ = sp.block_norm_fwd(x, **kw)
    check(y, x.double() + s * G * v, NORM_F32 * (x.double().abs() + (s * G).abs() * va), dtype, "y")
    Y, dy, dya = y.double(), gy.double(), gy.double().abs()
    if nxt:
        ny, ry, nya = norm64(Y, kind, 0.0)
        q = gh.double() * wn.double()
        dy, dya = dy + nvjp64(q, ny, ry, kind), dya + nvjp_abs(q.abs(), nya, ry, kind)
    got = sp.block_norm_bwd(y, gy, gh if nxt else None, **kw)
    p, pa = dy * s * G * wp.double(), dya * (s * G).abs() * wp.double().abs()
    check(got[0], dy, NORM_F32 * dya, dtype, "grad_x")
    check(got[1], nvjp64(p, nf, rf, kind), NORM_F32 * nvjp_abs(pa, nfa, rf, kind), dtype, "grad_f")
    check(got[3], (dy * s * G * nf).sum(0), NORM_F32 * (dya * (s * G).abs() * nfa).sum(0), "f32", "grad_w_post")
    check(got[4], (dy * G * v).sum(0), NORM_F32 * (dya * G.abs() * va).sum(0), "f32", "grad_res_scale")
    if nxt:
        check(got[5], (gh.double() * ny).sum(0), NORM_F32 * (gh.double().abs() * nya).sum(0), "f32", "grad_w_pre")


# ------------------------------------------------------------------ gated feed-forward

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("di,F,do", [(8, 16, 8), (33, 70, 5), (1000, 1200, 900)])
def test_gated_ffn_bwd_of_no_rows(di, F, do, dtype):
    """The weight gradients over no rows are zeros and their neighbours
    untouched; weights, rows and workspace may be null."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated ffn backward of no rows, null inputs, {di} x {F} x {do} {dtype}")
    bufs = [torch.full((k + 2,), 7.0, dtype=T[dtype], device="cuda") for k in (F * di, F * di, do * F)]
    to = [b.data_ptr() + b.element_size() for b in bufs]
    code = {"f32": sp.F32, "bf16": sp.BF16, "f16": sp.F16}[dtype]
    rc = sp.lib.gated_ffn_bwd(code, 0, None, di, None, None, None, None, do, 0, di, F, do, None, *to, None, 0,
                              torch.cuda.current_stream().cuda_stream)
    assert rc == sp.OK
    for b in bufs:
        assert not b[1:-1].any() and b[0] == 7 and b[-1] == 7


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [1024, 1001])
def test_gated_ffn_single_row_of_a_long_tensor(d, dtype):
    """The last position of one sequence: one row, whose stride is never used."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated ffn, one row with a row stride above 2^21, d={d} {dtype}")
    g = gen(d)
    seq, gseq = rnd(g, 1, 2500, d, dtype=dtype), rnd(g, 1, 2500, d, dtype=dtype)
    x, gy = seq[:, -1], gseq[:, -1]
    assert x.stride(0) > 1 << 21
    wg, wu = (rnd(g, 72, d, std=d ** -0.5, dtype=dtype) for _ in range(2))
    wd = rnd(g, d, 72, std=0.1, dtype=dtype)
    assert torch.equal(sp.gated_ffn_fwd(x, wg, wu, wd), sp.gated_ffn_fwd(x.clone(), wg, wu, wd))
    a, b = sp.gated_ffn_bwd(x, wg, wu, wd, gy), sp.gated_ffn_bwd(x.clone(), wg, wu, wd, gy.clone())
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("di,F,do", [(64, 128, 64), (40, 64, 200), (96, 72, 130)])
def test_gated_ffn_few_rows_as_accurate_as_many(di, F, do):
    """float32: 32 rows and more of them take different kernels, whose
    sums of few steps make the same roundings, that of the largest plane pair in
    one sum and those of the five small ones in another.  Of the some thousand
    outputs the root mean square error is the same to a few percent; with one sum
    for all six pairs it is half as much again."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated ffn float32, 32 rows alone and of 65, {di} x {F} x {do}")
    x, wg, wu, wd, _ = ffn_case(65, di, F, do, "f32", 3)
    X, G, U, D = (t.double() for t in (x, wg, wu, wd))
    ref = ((act64(X @ G.T, "silu")[0] * (X @ U.T)) @ D.T)[:32]
    few, many = ((t[:32].double() - ref).square().mean().sqrt().item()
                 for t in (sp.gated_ffn_fwd(x[:32], wg, wu, wd), sp.gated_ffn_fwd(x, wg, wu, wd)))
    print(f"[parity] rms error: few rows {few:.3e}, many {many:.3e}", flush=True)
    assert few <= 1.25 * many


def same_kind(got, ref, what):
    """Infinite where the reference is, of its sign, NaN where it is, else finite."""
    ref = ref.to(got.dtype)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN"
    inf = torch.isinf(ref)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], ref[inf]), f"{what}: infinities"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act", ["relu", "sigmoid"])
@pytest.mark.parametrize("n,di,F,do", [(5, 40, 72, 24), (64, 64, 136, 48), (90, 33, 70, 31), (700, 256, 520, 256)])
def test_gated_ffn_infinities_and_nan(n, di, F, do, act, dtype):
    """An infinity and a NaN in x, in w_down and in grad_out: what they reach is
    infinite or NaN as the formula has it, everything else as without them."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated ffn, infinities and NaN, n={n} {di} x {F} x {do} {act} {dtype}")
    x, wg, wu, wd, gy = ffn_case(n, di, F, do, dtype, n + 1)
    inf, nan = float("inf"), float("nan")

    def forward(x, wd):
        X, G, U, D = (t.double() for t in (x, wg, wu, wd))
        return (act64(X @ G.T, act)[0] * (X @ U.T)) @ D.T

    plain = sp.gated_ffn_fwd(x, wg, wu, wd, act=act)
    bad = x.clone()
    bad[1, 3], bad[2, 4], bad[n - 1, di - 1] = inf, nan, -inf
    out = sp.gated_ffn_fwd(bad, wg, wu, wd, act=act)
    same_kind(out, forward(bad, wd), "out of x")
    keep = torch.ones(n, dtype=torch.bool)
    keep[[1, 2, n - 1]] = False
    assert torch.equal(out[keep], plain[keep])
    badw = wd.clone()
    badw[2, 5], badw[do - 1, 0] = inf, nan
    out = sp.gated_ffn_fwd(x, wg, wu, badw, act=act)
    # relu's zero times an infinity is NaN; the sign of a value that is nearly zero is not asked for
    h = act64(x.double() @ wg.double().T, act)[0][:, 5] * (x.double() @ wu.double().T)[:, 5]
    clear = (h == 0) | (h.abs() > 1e-3)
    same_kind(out[clear], forward(x, badw)[clear], "out of w_down")
    keep = torch.ones(do, dtype=torch.bool)
    keep[[2, do - 1]] = False
    assert torch.equal(out[:, keep], plain[:, keep])
    # grad_out: one row of grad_x, one row of grad_w_down
    full = sp.gated_ffn_bwd(x, wg, wu, wd, gy, act=act)
    badg = gy.clone()
    badg[3, 7] = inf
    got = sp.gated_ffn_bwd(x, wg, wu, wd, badg, act=act)
    keep = torch.ones(n, dtype=torch.bool)
    keep[3] = False
    assert torch.equal(got[0][keep], full[0][keep]) and not torch.isfinite(got[0][3]).any()
    h = act64(x.double() @ wg.double().T, act)[0][3] * (x.double() @ wu.double().T)[3]
    clear = (h == 0) | (h.abs() > 1e-3)
    same_kind(got[3][7][clear], (inf * h)[clear], "grad_w_down")
    keep = torch.ones(do, dtype=torch.bool)
    keep[7] = False
    assert torch.equal(got[3][keep], full[3][keep])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_embedding_infinities_and_nan(dtype):
    """Of tokens out of range they reach nothing, of others their column only."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"embedding, infinities and NaN {dtype}")
    g = gen(8)
    for n, rows, dim in ((700, 10, 33), (700, 300, 40), (40000, 5000, 24)):
        tok = torch.randint(0, rows, (n,), generator=g, device="cuda", dtype=torch.int32)
        grad = rnd(g, n, dim, dtype=dtype)
        tok[5], tok[6] = -1, rows
        full = sp.embedding_bwd(grad, tok, rows)
        grad[5], grad[6, 2], grad[n - 1, 3], grad[8, 4] = float("nan"), float("inf"), float("inf"), float("nan")
        got = sp.embedding_bwd(grad, tok, rows)
        want = full.clone()
        want[tok[n - 1].long(), 3], want[tok[8].long(), 4] = float("inf"), float("nan")
        assert torch.equal(got.nan_to_num(7.0, 9.0, 11.0), want.nan_to_num(7.0, 9.0, 11.0))
        table = rnd(g, rows, dim, dtype=dtype)
        table[tok[0].long(), 1] = float("-inf")
        out = sp.embedding_fwd(table, tok)
        at = tok.long().clamp(0, rows - 1)
        ok = (tok >= 0) & (tok < rows)
        assert torch.equal(out, torch.where(ok[:, None], table[at], torch.zeros_like(table[at])))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,dim,kind", [(37, 64, "layer"), (9, 1000, "rms"), (5, 8192, "layer")])
def test_block_norm_infinities_and_nan(n, dim, kind, dtype):
    """A row with an infinity or a NaN spoils itself and the column sums, and
    no other row; the sums stay whole in the columns of a finite row's NaN gate."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"block norm, infinities and NaN, n={n} dim={dim} {kind} {dtype}")
    g = gen(n)
    x, f, gy, gh = (rnd(g, n, dim, dtype=dtype) for _ in range(4))
    gt = rnd(g, n, dim, dtype=dtype)
    w = 1 + rnd(g, dim, std=0.1)
    kw = dict(w_post=w, res_scale=w, w_pre=w, kind=kind)
    y0, h0 = sp.block_norm_fwd(x, f, gate=gt, **kw)
    b0 = sp.block_norm_bwd(y0, gy, gh, f, gate=gt, **kw)
    keep = torch.ones(n, dtype=torch.bool)
    keep[[1, n - 1]] = False
    bad = f.clone()
    bad[1, 3], bad[n - 1, dim - 1] = float("inf"), float("nan")
    y, h = sp.block_norm_fwd(x, bad, gate=gt, **kw)
    assert torch.equal(y[keep], y0[keep]) and torch.equal(h[keep], h0[keep])
    assert not torch.isfinite(y[n - 1]).any() and not torch.isfinite(y[1, 3])
    got = sp.block_norm_bwd(y0, gy, gh, bad, gate=gt, **kw)
    assert torch.equal(got[0], b0[0]) and all(torch.equal(p[keep], q[keep]) for p, q in zip(got[:3], b0[:3]))
    badg = gt.clone()
    badg[1, 3] = float("nan")
    got = sp.block_norm_bwd(y0, gy, gh, f, gate=badg, **kw)
    cols = torch.ones(dim, dtype=torch.bool)
    cols[3] = False
    for p, q in zip(got[3:5], b0[3:5]):
        assert torch.equal(p[cols], q[cols]) and torch.isnan(p[3])
    assert torch.equal(got[5], b0[5]) and torch.equal(got[0], b0[0])


def wide_range(n, di, F, do, how, seed):
    """float16 inputs of the feed-forward block whose hidden values leave
    float16's range and whose results do not.  "big": hidden values far past
    65504.  "small": gradients of a few 2^-24, of which the sums over many rows
    are ordinary numbers.  "mixed": runs of rows and of hidden columns of
    magnitudes from 2^-12 to 2^12 of the others."""
    x, wg, wu, wd, gy = ffn_case(n, di, F, do, "f16", seed)
    if how == "big":
        return (x * 1000).half(), wg, wu, (wd / 4096).half(), (gy / 1024).half()
    if how == "small":
        return (x * 32).half(), (wg / 32).half(), (wu / 32).half(), wd, (gy * 1.5e-7).half()
    g = gen(seed + 1)
    rows = 2.0 ** torch.randint(-3, 4, ((n + 49) // 50,), generator=g, device="cuda").repeat_interleave(50)[:n]
    cols = 2.0 ** torch.randint(-6, 7, ((F + 39) // 40,), generator=g, device="cuda").repeat_interleave(40)[:F]
    return (x * rows[:, None] * 16).half(), wg, (wu * cols[:, None] * 8).half(), (wd / 4096).half(), \
        (gy * rows.flip(0)[:, None] / 1024).half()


def wide_reference(x, wg, wu, wd, gy, act):
    """As ``ffn_reference``, of gradients times 2^40 (all are linear in grad_out), so
    that its allowance for the smallest float16 does not count, but with what a
    block loses of its small values: 2^-16 of the bounds that give its exponent,
    here over all blocks."""
    up = 2.0 ** 40
    (out, eout), grads = ffn_reference(x, wg, wu, wd, gy.double() * up, act, "f16")
    X, G, U, D, Y = (t.double() for t in (x, wg, wu, wd, gy))
    mg, mu, md = (t.abs().max().item() for t in (X @ G.T, X @ U.T, Y @ D))
    mg = 1.0 if act == "sigmoid" else mg
    n, F = x.shape[0], wg.shape[0]
    fh, fg, fu = (2.0 ** -16 * t for t in (mg * mu, 1.13 * md * mu, md * mg))
    one = torch.ones(n, F, dtype=torch.float64, device="cuda")
    more = (fg * (one @ G.abs()) + fu * (one @ U.abs()), fg * (one.T @ X.abs()), fu * (one.T @ X.abs()),
            fh * (Y.abs().T @ one))
    return (out, eout + fh * D.abs().sum(1)), [(r / up, e / up + m) for (r, e), m in zip(grads, more)]


@pytest.mark.parametrize("how", ["big", "small", "mixed"])
@pytest.mark.parametrize("act", ["relu", "sigmoid"])
@pytest.mark.parametrize("n,di,F,do", [(1, 64, 200, 40), (20, 64, 200, 40), (40, 33, 1000, 65), (64, 128, 72, 48),
                                       (65, 64, 200, 40), (700, 64, 300, 40), (130, 322, 853, 257), (70, 200, 3001, 65),
                                       (5000, 65, 70, 33), (300, 20, 8000, 640), (4100, 1030, 1032, 1100),
                                       (4096, 72, 2048, 64), (2048, 4096, 136, 4096), (17000, 16, 72, 24),
                                       (70, 24, 8500, 16), (5, 24, 8500, 40)])
def test_gated_ffn_float16_range(n, di, F, do, act, how):
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated ffn float16, {how} hidden values, n={n} {di} x {F} x {do} {act}")
    x, wg, wu, wd, gy = wide_range(n, di, F, do, how, n + F)
    (out, eout), grads = wide_reference(x, wg, wu, wd, gy, act)
    got = sp.gated_ffn_fwd(x, wg, wu, wd, act=act)
    check(got, out, eout, "f16", "out")
    back = sp.gated_ffn_bwd(x, wg, wu, wd, gy, act=act)
    for name, a, (r, e) in zip(("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down"), back, grads):
        fits = r.abs() < 60000
        check(torch.where(fits, a, 0), torch.where(fits, r, 0), torch.where(fits, e, 0), "f16", name)
    assert torch.equal(got, sp.gated_ffn_fwd(x, wg, wu, wd, act=act))
    assert all(torch.equal(p, q) for p, q in zip(back, sp.gated_ffn_bwd(x, wg, wu, wd, gy, act=act)))


@pytest.mark.parametrize("n", [40, 500])
def test_gated_ffn_float16_infinities_beside_large_and_small_blocks(n):
    """An infinity in a block of zeros, and beside finite values that need an exponent."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated ffn float16, infinities in scaled blocks, n={n}")
    x, wg, wu, wd, gy = wide_range(n, 64, 200, 40, "mixed", 3)
    keep = torch.ones(n, dtype=torch.bool)
    plain = sp.gated_ffn_fwd(x, wg, wu, wd, act="relu")
    for rest in (1.0, 0.0):
        bad = x * rest
        bad[7, 5] = float("inf")
        keep[7] = False
        X, G, U, D = (t.double() for t in (bad, wg, wu, wd))
        ref = (act64(X @ G.T, "relu")[0] * (X @ U.T)) @ D.T
        out = sp.gated_ffn_fwd(bad, wg, wu, wd, act="relu")
        same_kind(out, ref, "out")
        assert torch.equal(out[keep], plain[keep] * rest)


# ------------------------------------------------------------------ embedding gradient

@pytest.mark.parametrize("n,rows,dim", [(3, 1 << 20, 5), (524287, 5000, 3), (524288, 5000, 3), (2100000, 17, 2),
                                        (600001, 300000, 4), (700000, (1 << 20) + 5, 3), (32768, 1 << 17, 9),
                                        (32769, 1 << 17, 9), (32768, (1 << 17) + 1, 9), (32768, 17, 8)])
def test_embedding_gradient_at_its_limits(n, rows, dim):
    """The ends of the one-launch ordering (32768 tokens, 2^17 rows), three
    passes of the radix sort (2^20 rows), and its workgroups' counts added up by
    themselves and by a kernel of its own (from 524288 tokens)."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"embedding gradient at its limits, n={n} rows={rows} dim={dim}")
    g = gen(n + rows)
    tok, grad = tokens_of(g, n, rows, torch.int32), rnd(g, n, dim)
    tok[-1], grad[-1] = rows - 1, 1.0
    ok = (tok >= 0) & (tok < rows)
    at, src = tok.long().clamp(0, rows - 1), grad.double() * ok[:, None]
    ref = torch.zeros(rows, dim, dtype=torch.float64, device="cuda").index_add_(0, at, src)
    mag = torch.zeros(rows, dim, dtype=torch.float64, device="cuda").index_add_(0, at, src.abs())
    count = torch.zeros(rows, dtype=torch.float64, device="cuda").index_add_(0, at, ok.double())
    d = sp.embedding_bwd(grad, tok, rows)
    check(d, ref, (count[:, None] + 2) * E24 * mag, "f32", "grad_table")
    assert torch.equal(sp.embedding_bwd(grad, tok, rows), d)


def test_embedding_of_more_than_a_launch():
    """A launch has fewer than 2^32 threads, a list and a table may need more."""
    need_gpu()
    import segmented_polynomials_amd as sp
    n = (1 << 28) + 5
    announce(f"embedding gradient of {n} tokens, one gradient row read by all")
    tok = torch.arange(n, device="cuda", dtype=torch.int32) % 40000
    d = sp.embedding_bwd(torch.ones(1, 1, device="cuda").expand(n, 1), tok, 40000)
    want = torch.full((40000, 1), float(n // 40000), device="cuda")  # whole numbers below 2^24 are exact
    want[:n % 40000] += 1
    assert torch.equal(d, want)
    del tok, d
    rows = (1 << 28) + 3
    announce(f"embedding gradient into {rows} rows")
    tok = torch.tensor([0, 5, rows - 1, rows - 1, 1 << 27, (1 << 26) - 1, 1 << 26, rows], device="cuda", dtype=torch.int32)
    d = sp.embedding_bwd(torch.ones(8, 2, device="cuda", dtype=torch.bfloat16), tok, rows)
    at = torch.nonzero(d[:, 0])[:, 0].tolist()
    assert at == [0, 5, (1 << 26) - 1, 1 << 26, 1 << 27, rows - 1] and torch.equal(d[:, 0], d[:, 1])
    assert d[at, 0].tolist() == [1, 1, 1, 1, 1, 2]


# ------------------------------------------------------------------ accuracy of the feed-forward block

@pytest.mark.parametrize("shape", acc.SHAPES_F32)
def test_gated_ffn_float32_accuracy(shape):
    """All 24 bits of long sums: fewer plane pairs miss this bound (tests/test_ffn_accuracy.py)."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated ffn float32 accuracy {shape}")
    x, wg, wu, wd, gy = acc.inputs(*shape, 1, "cuda")
    ref = acc.block(*(t.double() for t in (x, wg, wu, wd, gy)))
    bound = acc.float32_rms(*shape)
    for name, a, r in zip(acc.NAMES, (sp.gated_ffn_fwd(x, wg, wu, wd), *sp.gated_ffn_bwd(x, wg, wu, wd, gy)), ref):
        worst = acc.rms_error(a, r) / bound[name]
        print(f"[parity] {name}: {worst:.3f} of the rms bound", flush=True)
        assert worst <= 1, name


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", acc.SHAPES_16)
def test_gated_ffn_16_bit_roundings(shape, dtype):
    """h, dg and du are rounded to 16 bits, nothing else before the outputs (dh is not)."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated ffn roundings {shape} {dtype}")
    t = T[dtype]
    x, wg, wu, wd, gy = acc.inputs(*shape, 2, "cuda", t)
    ref = acc.block(*(v.double() for v in (x, wg, wu, wd, gy)), hidden=lambda v: v.to(t).double())
    for name, a, r in zip(acc.NAMES, (sp.gated_ffn_fwd(x, wg, wu, wd), *sp.gated_ffn_bwd(x, wg, wu, wd, gy)), ref):
        share = acc.unequal(a, r, t)
        print(f"[parity] {name}: {share:.4f} of the elements rounded another way", flush=True)
        assert share <= acc.UNEQUAL, name


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [65, 90, 500])
def test_gated_ffn_bwd_infinity_in_rows_that_overlap(n, dtype):
    """One gradient row read by all, and rows eight elements apart: the sum over
    the rows ends with the last, also where a row past it would be memory of others."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated ffn backward, overlapping gradient rows with an infinity, n={n} {dtype}")
    x, wg, wu, wd, gy = ffn_case(n, 64, 72, 40, dtype, 5)
    x, wu = x.abs() + 0.1, wu.abs() + 0.1  # hidden values are positive: infinity times them is infinity
    flat = gy.flatten()[:(n - 1) * 8 + 40].clone()
    flat[-1] = float("inf")
    one = gy[:1].clone()
    one[0, 5] = float("inf")
    for rows in (one.expand(n, 40), flat.as_strided((n, 40), (8, 1))):
        a = sp.gated_ffn_bwd(x, wg, wu, wd, rows, act="sigmoid")
        b = sp.gated_ffn_bwd(x, wg, wu, wd, rows.clone(memory_format=torch.contiguous_format), act="sigmoid")
        assert torch.isinf(b[3]).any() and torch.isfinite(b[3]).any()
        assert all(torch.equal(p.nan_to_num(7.0, 9.0, 11.0), q.nan_to_num(7.0, 9.0, 11.0)) for p, q in zip(a, b))
