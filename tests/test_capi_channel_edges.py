"""Host side of the invariant-channel operators at the ends of their ranges:
as in ``test_capi_channel_host`` every call fails, or does nothing, before a
kernel is launched, and no pointer is read."""

import ctypes

import pytest

import segmented_polynomials_amd as sp

P = 4096          # a non-null address, 256-byte aligned


def size(fn, *args):
    v = ctypes.c_size_t()
    rc = fn(*args, ctypes.byref(v))
    return rc, v.value


@pytest.mark.parametrize("dtype", [sp.F32, sp.BF16, sp.F16])
def test_gated_ffn_bwd_of_no_rows_needs_no_input(dtype):
    """No workspace, and with only grad_x asked for nothing to do."""
    assert size(sp.lib.gated_ffn_workspace, dtype, 0, 8, 16, 8, 1) == (sp.OK, 0)
    assert sp.lib.gated_ffn_bwd(dtype, 0, None, 8, None, None, None, None, 8, 0, 8, 16, 8, P, None, None, None, None, 0,
                                None) == sp.OK
    # what is refused with rows still is
    assert sp.lib.gated_ffn_bwd(dtype, 0, None, 8, None, None, None, None, 8, 0, 8, 16, 8, P, P, None, None, None, 0,
                                None) == sp.E_INVALID
    assert sp.lib.gated_ffn_bwd(dtype, 0, P, 8, P, None, P, P, 8, 3, 8, 16, 8, P, None, None, None, P, 1 << 30,
                                None) == sp.E_INVALID


def test_gated_ffn_row_stride_of_a_single_row():
    """Never used, so never too large; the call then fails for its workspace."""
    for n, what in ((1, "null workspace"), (2, "bad row stride")):
        assert sp.lib.gated_ffn_fwd(sp.BF16, 0, P, 1 << 40, P, P, P, n, 8, 16, 8, P, 8, None, 0, None) == sp.E_INVALID
        assert what in sp.lib.segpoly_last_error().decode()
        assert sp.lib.gated_ffn_bwd(sp.BF16, 0, P, 1 << 40, P, P, P, P, 1 << 40, n, 8, 16, 8, P, P, P, P, None, 0,
                                    None) == sp.E_INVALID
        assert what in sp.lib.segpoly_last_error().decode()


def misaligned(fn, args, at, by):
    a = list(args)
    a[at] = P + by
    return fn(*a) == sp.E_INVALID and "misaligned" in sp.lib.segpoly_last_error().decode()


@pytest.mark.parametrize("dtype,off", [(sp.F32, 2), (sp.BF16, 1), (sp.F16, 1)])
def test_buffers_off_their_elements_are_refused(dtype, off):
    """Buffers of the rows' type by half an element, parameters and tokens by
    two bytes; no other argument is at fault, and none is launched."""
    small = 0  # of the workspace: refused afterwards, were the alignment not
    emb = (dtype, P, 5, 8, P, sp.I64, 3, 1.0, P, 8, None)
    assert all(misaligned(sp.lib.embedding_fwd, emb, i, off) for i in (1, 8))
    assert misaligned(sp.lib.embedding_fwd, emb, 4, 4)
    emb = (dtype, P, 8, P, sp.I32, 3, 5, 8, 1.0, P, P, small, None)
    assert all(misaligned(sp.lib.embedding_bwd, emb, i, off) for i in (1, 9))
    assert misaligned(sp.lib.embedding_bwd, emb, 3, 2)
    norm = (dtype, 0, 2, 0, P, 8, P, 8, P, 8, P, P, P, 1e-6, 3, 8, P, P, None)
    assert all(misaligned(sp.lib.block_norm_fwd, norm, i, off) for i in (4, 6, 8, 16, 17))
    assert all(misaligned(sp.lib.block_norm_fwd, norm, i, 2) for i in (10, 11, 12))
    norm = (dtype, 0, 2, 0, P, 8, P, 8, P, 8, P, 8, P, 8, P, P, P, 1e-6, 3, 8, P, P, P, P, P, P, P, small, None)
    assert all(misaligned(sp.lib.block_norm_bwd, norm, i, off) for i in (4, 6, 8, 10, 12, 20, 21, 22))
    assert all(misaligned(sp.lib.block_norm_bwd, norm, i, 2) for i in (14, 15, 16, 23, 24, 25))
    ffn = (dtype, 0, P, 8, P, P, P, 3, 8, 16, 8, P, 8, P, small, None)
    assert all(misaligned(sp.lib.gated_ffn_fwd, ffn, i, off) for i in (2, 4, 5, 6, 11))
    ffn = (dtype, 0, P, 8, P, P, P, P, 8, 3, 8, 16, 8, P, P, P, P, P, small, None)
    assert all(misaligned(sp.lib.gated_ffn_bwd, ffn, i, off) for i in (2, 4, 5, 6, 7, 13, 14, 15, 16))


@pytest.mark.parametrize("n,rows,dim", [(100000, 40000, 70), (32769, 5000, 1), (1 << 20, 1 << 21, 24), (1 << 26, 300, 7)])
def test_embedding_workspace_holds_every_part(n, rows, dim):
    """Sorted keys and positions twice, 4096 tokens' counts of the digits and the
    total, the row ranges, and one float32 row of a multiple of eight columns per
    16 positions."""
    digits = rows.bit_length()
    passes = -(-digits // 10)
    counts = 1 << -(-digits // passes)
    need = 16 * n + 4 * counts * (-(-n // 4096) + 1) + 4 * (rows + 1) + 4 * (n // 16) * (-(-dim // 8) * 8)
    got = size(sp.lib.embedding_bwd_workspace, n, rows, dim)
    assert got[0] == sp.OK and need <= got[1] <= need + 7 * 256 and got[1] % 256 == 0
