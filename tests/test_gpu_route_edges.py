"""The routing's gradient where scores saturate, and routing, places and sums at
their largest sizes."""

import pytest
import torch

import tile_partitioned_dense_amd as tg

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    with tg.TileGemm(0) as gg:
        yield gg


@pytest.mark.parametrize("E", [16, 64, 200, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_sigmoid_gradient_of_saturated_scores(g, E, dtype):
    """s (1 - s) of a score next to 1 is its exponential's, not a difference that
    rounds away: right relative to itself, rounded once."""
    T = 40
    logits = torch.linspace(-80, 80, T * E).view(T, E).to(dtype)
    ids = torch.arange(T)[:, None].mul(7).add(torch.tensor([0, 1, E // 2, E - 1])).remainder(E).to(I32)
    dw = torch.randn(T, 4, generator=torch.Generator().manual_seed(E))
    d = torch.zeros(T, E, dtype=dtype, device="cuda")
    g.route_backward(logits.cuda(), ids.cuda(), dw.cuda(), d, score=tg.Score.SIGMOID, renormalize=False, scale=2.0)
    e = torch.exp(-logits.double().abs())
    want = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, ids.long(), 2.0 * dw.double())
    want = want * e / (1 + e) ** 2
    got = d.cpu().double()
    # (its 64-bit operations are off by 1e-13 at the most; what cancels in `want` does in the kernel's sum)
    assert bool(((got - want).abs() <= (torch.finfo(dtype).eps / 2 + 2.0 ** -40) * want.abs()).all())
