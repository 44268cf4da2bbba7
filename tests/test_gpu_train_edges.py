"""Edge calls of the gated block and of the cross entropy head on the GPU."""

import pytest
import torch

import tile_partitioned_dense_amd as tg
from test_gpu_glu import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    with tg.TileGemm(0) as handle:
        yield handle


@pytest.mark.parametrize("rows", [1, 3])
def test_columns_apart_are_refused(g, rows):
    """A view whose columns are not consecutive, of one row as of several: the
    call is refused and writes nothing."""
    K, F = 64, 16
    w = torch.randn(2 * F, K, device=DEV).bfloat16()
    x, h = torch.randn(rows, K, device=DEV).bfloat16(), torch.zeros(rows, F, device=DEV)
    wide_x, wide_h = torch.randn(K, 8, device=DEV).bfloat16(), torch.zeros(F, 8, device=DEV)
    bad_x, bad_h = wide_x[:, :rows].t(), wide_h[:, :rows].t()
    for gate in tg.Gate:
        assert tg.tile_gemm_run_glu(g.handle, bad_x, w.t(), h, gate=gate, check=False) == tg.Status.ERR_BAD_STRIDE
        assert tg.tile_gemm_run_glu(g.handle, x, w.t(), bad_h, gate=gate, check=False) == tg.Status.ERR_BAD_STRIDE
    torch.cuda.synchronize()
    assert not bool(h.any()) and not bool(wide_h.any())
