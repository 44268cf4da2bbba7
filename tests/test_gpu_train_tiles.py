"""Every compiled kernel of the gated block and the cross entropy head, each on
the smallest of a list of shapes for which the planner takes it."""

import functools

import pytest
import torch

import tile_partitioned_dense_amd as tg
from test_gpu_glu import DEV, integers, put
from train_helpers import GATES, Glu, Xent, close

pytestmark = pytest.mark.gpu
N_TILES = 9  # five tiles, four stream configurations
ROWS = (40, 70, 130, 200, 300, 520, 770, 1030, 1300, 1540, 2050)
COLS = (64, 144, 272, 528, 784, 1040, 2064, 3600, 4112, 5008, 6160, 8208)
DEPTHS = {tg.TrainProduct.LOGITS: (72, 100), tg.TrainProduct.GATED: (72, 100),
          tg.TrainProduct.GRADIENT: (80, 144, 528, 1040, 4112, 10256)}


@pytest.fixture(scope="module")
def g():
    with tg.TileGemm(0) as handle:
        yield handle


@functools.lru_cache(None)
def shapes():
    """{(product, tile, split): (M, N, K)}, the smallest of each."""
    found = {}
    for product, depths in DEPTHS.items():
        for M in ROWS:
            for N in COLS:
                for K in depths:
                    p = tg.tile_gemm_plan_train(M, N, K, product)
                    key = (product, p.config, p.k_split > 1)
                    if key not in found or M * N * (K + 200) < found[key][0]:
                        found[key] = (M * N * (K + 200), (M, N, K))
    return {k: v[1] for k, v in found.items()}


def shape(*key):
    assert key in shapes(), f"no listed shape is planned to {key}: add one"
    return shapes()[key]


@pytest.mark.parametrize("tile", range(N_TILES))
def test_logits(g, tile):
    T, V, K = shape(tg.TrainProduct.LOGITS, tile, False)
    gen = torch.Generator().manual_seed(tile)
    V += 3  # no whole chunk at the end; a few columns do not change the plan
    assert tg.tile_gemm_plan_train(T, V, K, tg.TrainProduct.LOGITS).config == tile
    x = torch.randn(T, K, generator=gen).bfloat16()
    w = (torch.randn(V, K, generator=gen) * 2 * K ** -0.5).bfloat16()
    t = torch.randint(0, V, (T,), generator=gen)
    t[::5] = -100
    d = torch.rand(T, generator=gen) / T
    ref = Xent(x, w, t, smoothing=0.1, z_loss=1e-3, dloss=d)
    xd, wd, td = put(x), put(w), t.to(DEV)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    opts = dict(label_smoothing=0.1, z_loss=1e-3)
    g.xent(xd, wd.t(), td, loss, lse, **opts)
    close(lse, ref.lse, ref.lse_err, False, "lse")
    close(loss, ref.loss, ref.loss_err, False, "loss")
    dx, dw = put(x), put(w)
    g.xent_backward(xd, wd.t(), td, lse, d.to(DEV), dA=dx, dB=dw.t(), piece=1 << 30, **opts)
    close(dx, ref.dx, ref.dx_err, True, "dx")
    close(dw, ref.dw, ref.dw_err, True, "dw")


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("tile", [t for t in range(N_TILES) if t != 2])  # 192 columns: not gated
def test_gated(g, tile, gate):
    T, N, K = shape(tg.TrainProduct.GATED, tile, False)
    F = N // 2
    gen = torch.Generator().manual_seed(10 + tile)
    x = torch.randn(T, K, generator=gen).bfloat16()
    w = (torch.randn(N, K, generator=gen) * 2 * K ** -0.5).bfloat16()
    b = torch.randn(N, generator=gen) * 0.5
    dh = torch.randn(T, F, generator=gen).bfloat16()
    ref = Glu(x, w, b, gate, dh)
    xd, wd, bd, dhd = put(x), put(w), b.to(DEV), put(dh)
    layouts = [wd.t()] + ([put(w.T.contiguous())] if tile < 5 else [])
    for weights in layouts:
        for dt in (torch.float32, torch.bfloat16):
            h = torch.empty(T, F, dtype=dt, device=DEV)
            g.glu(xd, weights, h, gate=tg.Gate[gate], bias=bd)
            close(h, ref.h, ref.h_err, dt == torch.bfloat16, f"h {dt}")
    dx, dw, db = put(x), put(w), torch.empty(N, device=DEV)
    g.glu_backward(xd, wd.t(), dhd, dA=dx, dB=dw.t(), gate=tg.Gate[gate], bias=bd, dbias=db)
    close(db, ref.dbias, ref.dbias_err, False, "dbias")
    close(dx, ref.dx, ref.dx_err, True, "dx")
    close(dw, ref.dw, ref.dw_err, True, "dw")


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("tile", range(5))
def test_gradients_exact(g, tile, split):
    """dx's product (T x K over 2 F) on integers whose sums are exact, and dW's."""
    T, K, N = shape(tg.TrainProduct.GRADIENT, tile, split)
    F = N // 2
    x, w, dh = integers(T, K, F, 40 + tile)
    z = x.double() @ w.double().T
    dz = torch.cat([dh * z[:, F:] * (z[:, :F] > 0), dh * z[:, :F].clamp(min=0)], 1)
    dx, dw = put(x.bfloat16()), put(w.bfloat16())
    db = torch.empty(N, device=DEV)
    for _ in range(2):
        g.glu_backward(put(x.bfloat16()), put(w.bfloat16()).t(), put(dh.bfloat16()), dA=dx, dB=dw.t(),
                       gate=tg.Gate.RELU, dbias=db)
        assert torch.equal(db.cpu().double(), dz.sum(0))
        assert torch.equal(dx.cpu(), (dz @ w.double()).bfloat16())
        assert torch.equal(dw.cpu(), (dz.T @ x.double()).bfloat16())


@pytest.mark.parametrize("T", [17, 128, 129, 640])
def test_weight_gradient_lengths(g, T):
    """dW over few tokens (its own kernel up to 128) and just past them, on
    columns and rows that fill no block."""
    for K, F in ((72, 504), (1000, 40), (264, 136)):
        x, w, dh = integers(T, K, F, 60 + T)
        z = x.double() @ w.double().T
        dz = torch.cat([dh * z[:, F:] * (z[:, :F] > 0), dh * z[:, :F].clamp(min=0)], 1)
        dw = put(w.bfloat16(), 8)
        g.glu_backward(put(x.bfloat16(), 8), put(w.bfloat16()).t(), put(dh.bfloat16()), dB=dw.t(), gate=tg.Gate.RELU)
        assert torch.equal(dw.cpu(), (dz.T @ x.double()).bfloat16())


@pytest.mark.parametrize("T,K,V", [(660, 264, 22197), (320, 520, 33054), (830, 264, 33054)])
def test_last_round_of_its_own(g, T, K, V):
    """Sizes whose last round of tiles is nearly empty: the logits (first two)
    and the weight gradient (last two) go in two launches, cut at a column. The
    targets lie on both sides of every multiple of 1024 columns, and in the
    last ones."""
    gen = torch.Generator().manual_seed(70 + T)
    x = torch.randn(T, K, generator=gen).bfloat16()
    w = (torch.randn(V, K, generator=gen) * 2 * K ** -0.5).bfloat16()
    t = torch.randint(0, V, (T,), generator=gen)
    edges = torch.arange(1024, V, 1024)
    edges = torch.cat([edges, edges - 1, torch.arange(V - 120, V)])
    t[:len(edges)] = edges
    t[-1] = -100
    d = torch.rand(T, generator=gen) / T
    opts = dict(label_smoothing=0.1, z_loss=1e-3)
    ref = Xent(x, w, t, dloss=d, smoothing=0.1, z_loss=1e-3)
    xd, wd, td = put(x), put(w), t.to(DEV)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    g.xent(xd, wd.t(), td, loss, lse, **opts)
    close(lse, ref.lse, ref.lse_err, False, "lse")
    close(loss, ref.loss, ref.loss_err, False, "loss")
    dx, dw = put(x), put(w)
    g.xent_backward(xd, wd.t(), td, lse, d.to(DEV), dA=dx, dB=dw.t(), **opts)
    close(dx, ref.dx, ref.dx_err, True, "dx")
    close(dw, ref.dw, ref.dw_err, True, "dw")
