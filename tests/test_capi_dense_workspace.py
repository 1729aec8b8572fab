"""Workspace of the dense layer by the form that a call takes, on the host: the
sizes name the form (one that a moved rule leaves untested shows here), and
ask for no space that the form does not write."""

import pytest

import segmented_polynomials_amd as sp

BYTES = {sp.F32: 4, sp.BF16: 2, sp.F16: 2}
ALL = [sp.F32, sp.BF16, sp.F16]


def up(v, to):
    return (v + to - 1) // to * to


def taken(*counts):
    """Bytes of float32 arrays, each at a multiple of 256."""
    return sum(up(4 * c, 256) for c in counts)


def shares(d_in, d_out):
    """Of the sum of few rows' products: for columns too few to fill the card."""
    groups = (d_out + 15) // 16
    most = 1 if groups > 64 else min(256 // groups, d_in // 512)
    return 1 if most < 2 else -(-d_in // up(-(-d_in // most), 64))


def packed(dtype, *shapes):
    return 0 if dtype == sp.F32 else sum(up(rows * up(width, 8) * 2, 256) for rows, width in shapes)


def held(dtype, n, d_out):
    """The gradient before the activation, of all rows."""
    if dtype == sp.F32:
        return up(n * up(d_out, 4) * 4, 256)
    blocks = up((n + 63) // 64 * ((d_out + 31) // 32) * 4, 256) if dtype == sp.F16 else 0
    return up(n * up(d_out, 64) * 2, 256) + blocks


@pytest.mark.parametrize("dtype", ALL)
def test_forward(dtype):
    # few rows: with one share, and with several
    for n, di, do in ((1, 8, 8), (16, 4096, 4096), (3, 1024, 4096), (16, 128, 64)):
        assert sp.dense_workspace(dtype, "silu", n, di, do) == 0
    for n, di, do in ((5, 8192, 64), (1, 1024, 33), (16, 1000, 1024)):
        s = shares(di, do)
        assert sp.dense_workspace(dtype, "silu", n, di, do) == (taken(s * n * up(do, 4)) if s > 1 else 0)
    # many rows of few columns: none
    for n, di, do in ((600000, 64, 64), (33, 128, 1000), (40, 31, 5000)):
        assert sp.dense_workspace(dtype, "silu", n, di, do) == 0
    # tiles that fill the card: copies of 16-bit operands alone
    for n, di, do in ((8192, 2048, 5632), (20000, 512, 512)):
        assert sp.dense_workspace(dtype, "gelu", n, di, do) == packed(dtype, (n, di), (do, di))


@pytest.mark.parametrize("dtype", ALL)
def test_backward_of_few_rows_and_in_one_pass(dtype):
    for n, di, do in ((1, 264, 33), (3, 72, 40), (4, 4096, 4096)):
        v = 4 if n > 2 else 16 // BYTES[dtype]
        lanes = 16
        while lanes < 64 and lanes * v < di:
            lanes *= 2
        most = max(1, 1024 // -(-di // (lanes * v)))
        parts = -(-do // up(max(-(-do // most), 256 // lanes * 4), 4))
        rows, sums = taken(n * up(do, 4)), taken(shares(di, do) * n * up(do, 4))
        assert sp.dense_workspace(dtype, "silu", n, di, do, True) == rows + sums + taken(parts * n * up(di, 4))
        assert sp.dense_workspace(dtype, "none", n, di, do, True) == rows + taken(parts * n * up(di, 4))
    for n, di, do in ((128 if dtype == sp.F32 else 1024, 64, 64), (600000, 64, 40), (5000, 7, 33)):
        blocks = min(-(-n // 16), 256)
        for act in ("none", "silu"):
            assert sp.dense_workspace(dtype, act, n, di, do, True) == taken(blocks * do * up(di, 4), blocks * up(do, 4))


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("n,di,do", [(600000, 64, 896), (8192, 2048, 5632), (100000, 128, 128), (20162, 64, 896)])
def test_backward_in_tiles(n, di, do, dtype):
    """Copies, the gradient before the activation, its column sums, and shares
    of the weight's gradient: at most a card's workgroups of 128 x 128 or 64 x 64
    each.  Nothing as large as all rows in float32 beside them."""
    size = sp.dense_workspace(dtype, "silu", n, di, do, True)
    fixed = packed(dtype, (n, di), (do, di)) + held(dtype, n, do) + taken(((n + 63) // 64 * 2 + 2) * up(do, 4))
    assert fixed <= size <= fixed + taken(512 * 128 * 128 + 768 * 64 * 64)
    none = sp.dense_workspace(dtype, "none", n, di, do, True)
    assert none <= packed(dtype, (n, di), (do, di), (n, do)) + taken(4096 * up(do, 4)) + taken(512 * 128 * 128 + 768 * 64 * 64)


@pytest.mark.parametrize("dtype", [sp.BF16, sp.F16])
def test_forward_rules_of_16_bit_rows(dtype):
    """Both sides of the rules: the streaming form asks for nothing, the rows'
    form with one share neither, tiles for their operands' copies."""
    copies = lambda n, di, do: packed(dtype, (n, di), (do, di))
    none = [(400, 255, 256), (200000, 255, 64), (400, 127, 512), (5000, 63, 512), (8000, 31, 1000), (1000, 192, 1024),
            (50000, 256, 256), (2000, 256, 248), (2000, 184, 1024), (20000, 250, 1020), (100000, 62, 255),
            (20000, 64, 250), (400, 256, 250), (70000, 255, 120), (70000, 31, 190), (500000, 255, 190),  # streaming
            (17, 64, 64), (32, 128, 1024), (32, 2048, 4096), (32, 1024, 8192), (24, 8190, 8192)]         # few rows
    for n, di, do in none:
        assert sp.dense_workspace(dtype, "silu", n, di, do) == 0, (n, di, do)
    for n, di, do in ((32, 2048, 512), (32, 8192, 512)):
        assert sp.dense_workspace(dtype, "silu", n, di, do) == taken(shares(di, do) * n * do)
    for n, di, do in ((4200, 255, 256), (17000, 127, 512), (17000, 63, 520), (9000, 31, 1000), (1100, 192, 1024),
                      (4100, 256, 256), (40000, 62, 1024), (1100, 192, 1023), (5000, 256, 255), (20000, 128, 1023),
                      (70000, 255, 200), (70000, 31, 260)):
        assert sp.dense_workspace(dtype, "silu", n, di, do) == copies(n, di, do) > 0, (n, di, do)
    for n, di, do in ((24, 4096, 1600), (32, 2048, 4104)):  # tiles, whose sums are shared out
        assert sp.dense_workspace(dtype, "silu", n, di, do) > copies(n, di, do)


def test_forward_rules_of_float32_rows():
    assert sp.dense_workspace(sp.F32, "silu", 17, 1000, 256) == 0  # one share
    for n, di, do in ((32, 1024, 512), (32, 2048, 512), (17, 2048, 1024)):
        assert sp.dense_workspace(sp.F32, "silu", n, di, do) == taken(shares(di, do) * n * do)
    assert sp.dense_workspace(sp.F32, "silu", 32, 2048, 1040) != taken(shares(2048, 1040) * 32 * 1040)
    for n, di, do in ((32, 64, 4096), (5000, 63, 512), (20000, 256, 1024)):  # streaming, and tiles that fill the card
        assert sp.dense_workspace(sp.F32, "silu", n, di, do) == 0
