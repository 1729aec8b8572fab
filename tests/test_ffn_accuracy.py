"""The accuracy bounds of the gated feed-forward block tell the forms that are
meant from worse ones: the worse forms are computed here, on the CPU."""

import pytest
import torch

from tests import _ffn_accuracy as acc


@pytest.mark.parametrize("shape", acc.SHAPES_F32)
def test_float32_bound_needs_all_plane_pairs(shape):
    t = acc.inputs(*shape, 1, "cpu")
    ref = acc.block(*(v.double() for v in t))
    bound = acc.float32_rms(*shape)
    held = lambda v: v.float().double()
    for pairs, meant in ((acc.ALL_PAIRS, True), (acc.ALL_PAIRS[:4], False), (acc.ALL_PAIRS[:3], False),
                         (acc.ALL_PAIRS[:1], False)):
        got = acc.block(*(v.double() for v in t), product=acc.planes_product(pairs), hidden=held)
        for name, a, r in zip(acc.NAMES, got, ref):
            assert (acc.rms_error(a, r) <= bound[name]) == meant, (name, len(pairs))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", acc.SHAPES_16[:3])
def test_16_bit_bound_tells_a_rounded_hidden_gradient(shape, dtype):
    t = [v.double() for v in acc.inputs(*shape, 2, "cpu", dtype)]
    held = lambda v: v.to(dtype).double()
    ref = acc.block(*t, hidden=held)
    for name, a, r in zip(acc.NAMES[1:4], acc.block(*t, hidden=held, dh_held=held)[1:4], ref[1:4]):
        assert acc.unequal(a, r, dtype) > 2 * acc.UNEQUAL, name
    # float32's own roundings stay below the bound
    for name, a, r in zip(acc.NAMES, acc.block(*(v.float() for v in t), hidden=lambda v: v.to(dtype).float()), ref):
        assert acc.unequal(a, r, dtype) <= acc.UNEQUAL, name
