"""Dense layer: infinities and NaN in the rows, the weight and the bias under
slopes, in every form of the forward and the backward.  What the definition
makes zero is zero, and what they do not reach is, bit for bit, what it is
without them."""

import pytest
import torch

from tests._gpu import announce, need_gpu
from tests.test_gpu_dense import case

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# few rows (two forms), products again of few rows and in shares, tiles of 64 and 128 rows, one pass over the rows;
# widths of d_out that end inside a chunk of eight, a block of 32 or a tile
FORMS = [(3, 72, 40), (3, 72, 33), (12, 600, 33), (40, 3000, 65), (300, 72, 33), (300, 72, 40), (700, 130, 853),
         (9000, 200, 300), (150, 64, 40), (150, 40, 33), (2000, 64, 40), (2000, 40, 33), (2000, 20, 7)]


def rows_without(t, *at):
    keep = torch.ones(t.shape[0], dtype=torch.bool, device="cuda")
    keep[list(at)] = False
    return t[keep]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,do", FORMS)
def test_infinite_rows_under_sigmoid(n, di, do, dtype):
    """A row whose products are all infinite has slopes of zero: its gradient
    is zero, and the others' sums are those without it."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dense gradient: an infinite row under sigmoid {n} {di} {do} {dtype}")
    x, w, b, _, g = case(n, di, do, dtype, 6)
    y, h = x.clone(), g.clone()
    h[2] = 0
    for bad in (INF, -INF):
        y[2, 5] = bad
        dx, dw, db = sp.dense_bwd(y, w, g, bias=b, act="sigmoid")
        ex, ew, eb = sp.dense_bwd(x, w, h, bias=b, act="sigmoid")
        assert not dx[2].any() and torch.equal(dx, ex) and torch.equal(db, eb)
        assert torch.equal(rows_without(dw.T, 5), rows_without(ew.T, 5)) and torch.isnan(dw[:, 5]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,do", FORMS)
def test_row_with_nan_or_infinity(n, di, do, dtype):
    """NaN: relu's slope is zero (z > 0 is false), sigmoid's NaN.  An infinity
    under relu: slopes of one and zero by the weight's sign."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dense gradient: a row with NaN or an infinity {n} {di} {do} {dtype}")
    x, w, b, _, g = case(n, di, do, dtype, 6)
    y, h = x.clone(), g.clone()
    h[2] = 0
    y[2, 5] = NAN
    dx, dw, db = sp.dense_bwd(y, w, g, bias=b, act="relu")
    ex, ew, eb = sp.dense_bwd(x, w, h, bias=b, act="relu")
    assert torch.equal(dx, ex) and torch.equal(db, eb)
    assert torch.equal(rows_without(dw.T, 5), rows_without(ew.T, 5)) and torch.isnan(dw[:, 5]).all()
    dx, dw, db = sp.dense_bwd(y, w, g, bias=b, act="sigmoid")
    ex = sp.dense_bwd(x, w, g, bias=b, act="sigmoid")[0]
    assert torch.isnan(dx[2]).all() and torch.isnan(dw).all() and torch.isnan(db).all()
    if dtype != "f16":  # a block's power of two may change with its largest value
        assert torch.equal(rows_without(dx, 2), rows_without(ex, 2))
    for bad in (INF, -INF):
        y[2, 5] = bad
        dx, dw, db = sp.dense_bwd(y, w, g, bias=b, act="relu")
        d = g[2].double() * (w[:, 5].double() * bad > 0)  # values of the type, held as they are
        ref, terms = d @ w.double(), d.abs() @ w.double().abs()
        lim = (do + 64) * 2.0 ** -24 * terms + torch.finfo(x.dtype).eps / 2 * ref.abs() + 2.0 ** -24
        assert ((dx[2].double() - ref).abs() <= lim).all()
        assert torch.isfinite(dx).all() and torch.isfinite(db).all() and torch.isfinite(rows_without(dw.T, 5)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,do", FORMS)
def test_infinite_weight_under_sigmoid(n, di, do, dtype):
    """A column whose products are all infinite has slopes of zero: its weight's
    and its bias's gradients are zero."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dense gradient: an infinite weight under sigmoid {n} {di} {do} {dtype}")
    x, w, b, _, g = case(n, di, do, dtype, 6)
    x[:, 5] = x[:, 5].abs() + 0.5
    v, h = w.clone(), g.clone()
    h[:, 3] = 0
    ex, ew, eb = sp.dense_bwd(x, w, h, bias=b, act="sigmoid")
    for bad in (INF, -INF):
        v[3, 5] = bad
        out = sp.dense_fwd(x, v, bias=b, act="sigmoid")
        assert (out[:, 3] == (1 if bad > 0 else 0)).all()
        assert torch.equal(rows_without(out.T, 3), rows_without(sp.dense_fwd(x, w, bias=b, act="sigmoid").T, 3))
        dx, dw, db = sp.dense_bwd(x, v, g, bias=b, act="sigmoid")
        assert torch.equal(dw, ew) and torch.equal(db, eb)
        assert torch.equal(rows_without(dx.T, 5), rows_without(ex.T, 5)) and torch.isnan(dx[:, 5]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,do", FORMS)
def test_infinities_and_nan_in_the_bias(n, di, do, dtype):
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dense gradient: infinities and NaN in the bias {n} {di} {do} {dtype}")
    x, w, b, _, g = case(n, di, do, dtype, 6)
    h, c = g.clone(), b.clone()
    h[:, 3] = 0
    for act in ("sigmoid", "relu"):
        none = sp.dense_bwd(x, w, h, bias=b, act=act)
        for bad in (INF, -INF):
            c[3] = bad
            out = sp.dense_fwd(x, w, bias=c, act=act)
            assert (out[:, 3] == (0 if bad < 0 else 1 if act == "sigmoid" else INF)).all()
            got = sp.dense_bwd(x, w, g, bias=c, act=act)
            if act == "relu" and bad > 0:  # slopes of one: the bias's gradient is that of no activation
                assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
                ref = g[:, 3].double()
                lim = (n + 64) * 2.0 ** -24 * ref.abs().sum() + torch.finfo(b.dtype).eps / 2 * ref.sum().abs()
                assert (got[2][3].double() - ref.sum()).abs() <= lim
            else:
                assert all(torch.equal(p, q) for p, q in zip(got, none))
        c[3] = NAN
        out = sp.dense_fwd(x, w, bias=c, act=act)
        assert torch.isnan(out[:, 3]).all()
        assert torch.equal(rows_without(out.T, 3), rows_without(sp.dense_fwd(x, w, bias=b, act=act).T, 3))
        dx, dw, db = sp.dense_bwd(x, w, g, bias=c, act=act)
        if act == "relu":  # z > 0 is false
            assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), none))
        else:
            assert torch.isnan(dx).all() and torch.isnan(dw[3]).all() and torch.isnan(db[3])
            assert torch.equal(rows_without(db, 3), rows_without(none[2], 3)) and torch.isfinite(rows_without(dw, 3)).all()


@pytest.mark.parametrize("n,di,do,dtype", [(3, 72, 40, "f32"), (40, 64, 72, "bf16"), (40, 64, 72, "f32"), (40, 520, 72, "f16"),
                                           (40, 520, 72, "f32"), (5, 4096, 40, "bf16")])
def test_output_rows_far_apart(n, di, do, dtype):
    """The residual's and the output's rows may be any distance apart; those of x
    and grad_out are refused past 2^21 elements."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dense: rows of the output far apart {n} {di} {do} {dtype}")
    x, w, b, res, g = case(n, di, do, dtype, 8)
    stride = (1 << 21) + 24
    held = torch.empty(n * stride, dtype=x.dtype, device="cuda")
    to = torch.as_strided(held, (n, do), (stride, 1), 5)
    to.copy_(res)
    sp.dense_fwd(x, w, bias=b, act="silu", residual=to, out=to)
    assert torch.equal(to, sp.dense_fwd(x, w, bias=b, act="silu", residual=res))
    with pytest.raises(sp.SegpolyError):
        sp.dense_bwd(x, w, to, bias=b, act="silu")
    with pytest.raises(sp.SegpolyError):
        sp.dense_fwd(torch.as_strided(held, (n, di), (stride, 1)), w, bias=b)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("n,di,do", FORMS + [(66000, 64, 16)])
def test_products_are_whole(n, di, do, dtype):
    """(1 + 2^-8)^2 - (1 + 2^-7) is 2^-16 exactly: the square's last bit, past what one bfloat16 part of a factor
    holds, counts in the output and in both gradients."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dense: whole products {n} {di} {do} {dtype}")
    t = {"f32": torch.float32, "f16": torch.float16}[dtype]
    one, two = 1 + 2.0 ** -8, 1 + 2.0 ** -7
    x, w, g = (torch.zeros(s, dtype=t, device="cuda") for s in ((n, di), (do, di), (n, do)))
    x[1, 2], x[1, 3], w[4, 2], w[4, 3] = one, two, one, -1
    out = sp.dense_fwd(x, w)
    assert out[1, 4].item() == 2.0 ** -16 and out.count_nonzero() == 1
    x.zero_(), w.zero_()
    g[1, 2], g[1, 3], w[2, 4], w[3, 4] = one, two, one, -1
    dx = sp.dense_bwd(x, w, g, need_dw=False)[0]
    assert dx[1, 4].item() == 2.0 ** -16 and dx.count_nonzero() == 1
    g.zero_(), w.zero_()
    g[1, 4], g[2, 4], x[1, 2], x[2, 2] = one, two, one, -1
    dw = sp.dense_bwd(x, w, g, need_dx=False)[1]
    assert dw[4, 2].item() == 2.0 ** -16 and dw.count_nonzero() == 1


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,do", FORMS + [(3000, 192, 1024), (20, 500, 64)])
def test_weight_with_nan_or_infinity(n, di, do, dtype):
    """Without an activation: the weight's element reaches its column of the
    output and of grad_x, nothing else."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"dense: a weight with NaN or an infinity {n} {di} {do} {dtype}")
    x, w, b, res, g = case(n, di, do, dtype, 6)
    x[:, 5] = x[:, 5].abs() + 0.5
    g[:, 3] = g[:, 3].abs() + 0.5
    clean, (cx, cw, cb) = sp.dense_fwd(x, w, bias=b, residual=res), sp.dense_bwd(x, w, g, bias=b)
    v = w.clone()
    for bad in (NAN, INF, -INF):
        v[3, 5] = bad
        same = torch.isnan if bad != bad else lambda t: t == bad
        out, (dx, dw, db) = sp.dense_fwd(x, v, bias=b, residual=res), sp.dense_bwd(x, v, g, bias=b)
        assert same(out[:, 3]).all() and torch.equal(rows_without(out.T, 3), rows_without(clean.T, 3))
        assert same(dx[:, 5]).all() and torch.equal(rows_without(dx.T, 5), rows_without(cx.T, 5))
        assert torch.equal(dw, cw) and torch.equal(db, cb)
