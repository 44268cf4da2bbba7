"""Few tokens: the two gradients of a call share a launch, and up to 64 rows
form the loss gradient's constants where it is stored. On both sides of those
limits, against the 64-bit references and against each gradient by itself."""
import pytest
import torch

import tile_partitioned_dense_amd as tg
from test_gpu_glu import DEV, put, strided
from train_helpers import HALF, Glu, Xent, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    with tg.TileGemm(0) as handle:
        yield handle


def like(t):
    return strided(*t.shape, 8, float("nan"))[1]


def tokens(T, K, seed):
    gen = torch.Generator().manual_seed(seed)
    return gen, torch.randn(T, K, generator=gen).bfloat16()


@pytest.mark.parametrize("T", [1, 15, 32, 33, 64, 65, 128, 129])
@pytest.mark.parametrize("K,F", [(264, 136), (1000, 1368), (1031, 40)])
def test_gated_block(g, T, K, F):
    gen, x = tokens(T, K, 61)
    w = (torch.randn(2 * F, K, generator=gen) * K ** -0.5).bfloat16()
    dh = torch.randn(T, F, generator=gen).bfloat16()
    ref = Glu(x, w, None, "SILU", dh)
    xd, wd, hd = put(x, 8), put(w, 8), put(dh, 8)
    both = like(xd), like(wd)
    g.glu_backward(xd, wd.t(), hd, dA=both[0], dB=both[1].t())
    close(both[0], ref.dx, ref.dx_err, True, "dx")
    close(both[1], ref.dw, ref.dw_err, True, "dw")
    dx, dw = like(xd), like(wd)
    g.glu_backward(xd, wd.t(), hd, dA=dx)
    g.glu_backward(xd, wd.t(), hd, dB=dw.t())
    assert torch.equal(dx, both[0]) and torch.equal(dw, both[1])


@pytest.mark.parametrize("T", [1, 31, 32, 33, 63, 64, 65, 128, 129])
@pytest.mark.parametrize("K,V,piece", [(264, 1000, 0), (264, 1000, 300), (65, 777, 0), (1032, 4100, 1100)])
@pytest.mark.parametrize("ignored", [0.0, 0.4])
def test_cross_entropy(g, T, K, V, piece, ignored):
    gen, x = tokens(T, K, 62)
    w = (torch.randn(V, K, generator=gen) * (2 * K ** -0.5)).bfloat16()
    t = torch.randint(0, V, (T,), generator=gen)
    t = torch.where(torch.rand(T, generator=gen) < ignored, 3, t)
    d = torch.randn(T, generator=gen) / T
    opts = dict(ignore_index=3, label_smoothing=0.1, z_loss=1e-3)
    ref = Xent(x, w, t, ignore=3, smoothing=0.1, z_loss=1e-3, dloss=d)
    xd, wd, td, dd = put(x, 8), put(w, 8), t.to(DEV, torch.int32), d.to(DEV)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    g.xent(xd, wd.t(), td, loss, lse, **opts)
    close(loss, ref.loss, ref.loss_err, False, "loss")
    both = like(xd), like(wd)
    g.xent_backward(xd, wd.t(), td, lse, dd, dA=both[0], dB=both[1].t(), piece=piece, **opts)
    close(both[0], ref.dx, ref.dx_err, True, "dx")
    close(both[1], ref.dw, ref.dw_err, True, "dw")
    dx, dw = like(xd), like(wd)
    g.xent_backward(xd, wd.t(), td, lse, dd, dA=dx, piece=piece, **opts)
    g.xent_backward(xd, wd.t(), td, lse, dd, dB=dw.t(), piece=piece, **opts)
    assert torch.equal(dx, both[0]) and torch.equal(dw, both[1])


@pytest.mark.parametrize("T", [40, 64, 65])
def test_unknown_targets_and_extremes(g, T):
    """Unknown targets are NaN in their rows only, ignored rows exact zeros (an
    infinite or NaN loss gradient there counts for nothing), no row at all left
    gives zeros, an infinite loss gradient its own row only."""
    K, V = 64, 300
    gen, x = tokens(T, K, 63)
    w = (torch.randn(V, K, generator=gen) * K ** -0.5).bfloat16()
    t = torch.randint(0, V, (T,), generator=gen)
    d = torch.rand(T, generator=gen) + 0.5
    t[3], t[4], t[5], t[T - 1] = V, -7, -100, -100
    d[5], d[T - 1] = float("inf"), float("nan")
    xd, wd, td, dd = put(x), put(w), t.to(DEV), d.to(DEV)
    lse = torch.empty(T, device=DEV)
    g.xent(xd, wd.t(), td, None, lse)
    keep = [i for i in range(T) if i not in (3, 4, 5, T - 1)]
    ref = Xent(x[keep], w, t[keep], dloss=d[keep])
    dx = torch.empty_like(xd)
    g.xent_backward(xd, wd.t(), td, lse, dd, dA=dx)
    assert bool(dx[3:5].isnan().all()) and not bool(dx[5].any()) and not bool(dx[T - 1].any())
    close(dx[keep], ref.dx, ref.dx_err, True, "dx")
    td.fill_(-100)
    dw = torch.empty_like(wd)
    g.xent_backward(xd, wd.t(), td, lse, dd, dA=dx, dB=dw.t())
    assert not bool(dx.any()) and not bool(dw.any())
    td.copy_(torch.randint(0, V, (T,), generator=gen))
    dd.fill_(1.0)
    dd[7] = float("inf")
    g.xent_backward(xd, wd.t(), td, lse, dd, dA=dx)
    others = [i for i in range(T) if i != 7]
    assert bool(dx[others].isfinite().all()) and not bool(dx[7].isfinite().all())


def test_captured_and_replayed(g):
    """Forward and both gradients in one graph, replayed with new inputs."""
    T, K, V, F = 48, 264, 1000, 136
    gen, x = tokens(T, K, 64)
    xd = put(x)
    w = put((torch.randn(V, K, generator=gen) * K ** -0.5).bfloat16())
    wg = put((torch.randn(2 * F, K, generator=gen) * K ** -0.5).bfloat16())
    dh = put(torch.randn(T, F, generator=gen).bfloat16())
    t = torch.randint(0, V, (T,), generator=gen).to(DEV)
    d = torch.rand(T, generator=gen).to(DEV)

    def step():
        loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        out = [loss, torch.empty_like(xd), torch.empty_like(w), torch.empty_like(xd), torch.empty_like(wg)]
        g.xent(xd, w.t(), t, loss, lse)
        g.xent_backward(xd, w.t(), t, lse, d, dA=out[1], dB=out[2].t())
        g.glu_backward(xd, wg.t(), dh, dA=out[3], dB=out[4].t())
        return out

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        xd.copy_(torch.randn(T, K, generator=gen).bfloat16())
        t.copy_(torch.randint(0, V, (T,), generator=gen))
        d.copy_(torch.rand(T, generator=gen))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("T", [40, 200, 600])
@pytest.mark.parametrize("V", [601, 1026])
def test_columns_past_a_ragged_vocabulary(g, T, V):
    """Logits of about -200 throughout: the zero logits of columns that are none
    would have exponentials past all bounds, and rows past the last token
    likewise; neither reaches a gradient.

    The gradients are held to their bounds element by element only. close()'s
    rule for the 2-norm takes a result for as large as its terms; here dx = G w
    with w = -3 +- 0.1 and rows of G that sum to zero keeps 0.1 of its terms'
    3, so G's rounding, at most HALF of a term, is up to 30 HALF of the result."""
    K = 64
    gen = torch.Generator().manual_seed(65)
    x = (1.0 + 0.1 * torch.randn(T, K, generator=gen)).bfloat16()
    w = (-3.0 + 0.1 * torch.randn(V, K, generator=gen)).bfloat16()
    t = torch.randint(0, V, (T,), generator=gen)
    d = torch.rand(T, generator=gen) / T
    ref = Xent(x, w, t, dloss=d)
    assert float(ref.lse.max()) < -150
    xd, wd, td = put(x), put(w), t.to(DEV)
    lse = torch.empty(T, device=DEV)
    g.xent(xd, wd.t(), td, None, lse)
    close(lse, ref.lse, ref.lse_err, False, "lse")
    dx, dw = like(xd), like(wd)
    g.xent_backward(xd, wd.t(), td, lse, d.to(DEV), dA=dx, dB=dw.t())
    for got, want, err in ((dx, ref.dx, ref.dx_err), (dw, ref.dw, ref.dw_err)):
        err = err + HALF * (want.abs() + err) + 2.0 ** -133
        assert bool(((got.double().cpu() - want).abs() <= err).all())
