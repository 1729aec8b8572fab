"""Dense layer: every form on rows of wider tensors, with outputs that are not
asked for, and on both sides of the rules between the forms (which form a
shape takes is held by its workspace, test_capi_dense_workspace.py)."""

import pytest

from tests import test_gpu_dense as dense
from tests._gpu import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,do", [(1, 264, 33), (3, 72, 40), (4, 130, 70), (2, 65, 9),       # few rows
                                     (12, 600, 40), (24, 1030, 72),                             # products of few rows
                                     (2000, 40, 33), (2000, 64, 64), (1100, 5, 3),              # one pass
                                     (300, 600, 33), (2000, 129, 72), (2000, 255, 256)])        # shares, tiles
def test_strides_and_parts(n, di, do, dtype, act):
    dense.test_strides_and_parts(n, di, do, dtype, act)


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,di,do", [
    # 17 to 32 rows
    (17, 64, 64), (32, 128, 1024), (24, 2048, 512), (32, 4096, 1024), (32, 8192, 512), (24, 4096, 1600), (32, 2048, 4104),
    (30, 2046, 4100), (21, 2047, 2050), (20, 1000, 8200), (20, 126, 4100), (20, 2000, 1040),
    # 16-bit rows of the streaming form, and of tiles
    (400, 255, 256), (9000, 255, 64), (400, 127, 512), (5000, 63, 512), (1000, 192, 1024), (50000, 256, 256), (2000, 184, 1024),
    (5000, 250, 1020), (400, 256, 250), (4200, 255, 256), (17000, 127, 512), (9000, 31, 1000), (1100, 192, 1024),
    (4100, 256, 256), (40000, 62, 1024), (1100, 192, 1023), (5000, 256, 255), (66000, 31, 190),
    # float32 rows of the streaming form, and of tiles
    (1000, 128, 130), (8200, 62, 1024), (66000, 64, 16), (66000, 64, 20), (16000, 61, 36), (9000, 64, 2003)])
def test_both_sides_of_the_rules(n, di, do, dtype, act):
    need_gpu()
    dense.run(n, di, do, dtype, act, 13)
