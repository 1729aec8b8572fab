"""Gated feed-forward: rows with infinities, hidden widths that end inside a
chunk of eight."""

import pytest
import torch

from tests._gpu import announce, need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,di,hidden,do", [(5, 40, 33, 24), (40, 40, 33, 24), (300, 72, 133, 40), (300, 72, 136, 40),
                                            (3000, 128, 259, 130)])
def test_infinite_row(n, di, hidden, do, dtype):
    """All weights positive: an infinity in a row makes its hidden values and
    its outputs infinite, and leaves the others as they are."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"gated feed-forward: an infinite row {n} {di} {hidden} {do} {dtype}")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.randn(n, di, generator=gen, device="cuda").to(dtype)
    wg, wu, wd = ((torch.rand(s, generator=gen, device="cuda") * 0.1 + 0.01).to(dtype)
                  for s in ((hidden, di), (hidden, di), (do, hidden)))
    y = x.clone()
    y[2, 5] = float("inf")
    keep = torch.arange(n, device="cuda") != 2
    for act in ("silu", "gelu", "relu", "sigmoid"):
        clean, out = sp.gated_ffn_fwd(x, wg, wu, wd, act=act), sp.gated_ffn_fwd(y, wg, wu, wd, act=act)
        assert (out[2] == float("inf")).all(), act
        assert torch.equal(out[keep], clean[keep]), act
