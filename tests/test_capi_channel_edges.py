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
