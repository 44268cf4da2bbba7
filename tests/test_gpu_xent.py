"""Cross entropy of a projection and its gradients on the GPU, against 64-bit
references."""

import math

import pytest
import torch

import tile_partitioned_dense_amd as tg
from test_gpu_glu import DEV, put, strided
from train_helpers import Xent, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    with tg.TileGemm(0) as handle:
        yield handle


def make(T, K, V, seed, ignored=0.0, scale=2.0, ignore=-100):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=gen).bfloat16()
    w = (torch.randn(V, K, generator=gen) * (scale * K ** -0.5)).bfloat16()
    t = torch.randint(0, V, (T,), generator=gen)
    t = torch.where(torch.rand(T, generator=gen) < ignored, ignore, t)
    d = torch.rand(T, generator=gen) * (torch.rand(T, generator=gen) > 0.1) / T
    return x, w, t, d


# rows: one, the stream kernel's blocks and one past them, a tile and one past
# it; odd K; vocabularies below a segment, ragged, of one column
SHAPES = [(1, 64, 1), (1, 136, 1000), (7, 72, 33), (32, 64, 257), (33, 1000, 500), (64, 128, 2051), (65, 200, 777),
          (50, 65, 300), (130, 96, 1031), (257, 328, 515), (300, 1032, 130)]


def forward(g, x, w, t, **kw):
    T = x.shape[0]
    loss, lse = (torch.full((T,), float("nan"), device=DEV) for _ in range(2))
    g.xent(x, w.t(), t, loss, lse, **kw)
    return loss, lse


@pytest.mark.parametrize("T,K,V", SHAPES)
@pytest.mark.parametrize("smoothing,z_loss,ignored", [(0.0, 0.0, 0.0), (0.1, 1e-3, 0.4), (1.0, 0.0, 1.0)])
def test_forward(g, T, K, V, smoothing, z_loss, ignored):
    x, w, t, _ = make(T, K, V, 5, ignored)
    ref = Xent(x, w, t, smoothing=smoothing, z_loss=z_loss)
    for it in (torch.int64, torch.int32):
        loss, lse = forward(g, put(x, 8), put(w, 8), t.to(DEV, it), label_smoothing=smoothing, z_loss=z_loss)
        close(lse, ref.lse, ref.lse_err, False, "lse")
        close(loss, ref.loss, ref.loss_err, False, "loss")


@pytest.mark.parametrize("T,K,V", SHAPES)
@pytest.mark.parametrize("piece", [0, 1, 300])
@pytest.mark.parametrize("smoothing,z_loss,ignored", [(0.0, 0.0, 0.0), (0.1, 1e-3, 0.4), (0.0, 0.0, 1.0)])
def test_backward(g, T, K, V, piece, smoothing, z_loss, ignored):
    if piece == 1:
        if V > 300:
            pytest.skip("a launch for each column: small vocabularies only")
        piece = 7
    x, w, t, d = make(T, K, V, 6, ignored)
    ref = Xent(x, w, t, smoothing=smoothing, z_loss=z_loss, dloss=d)
    opts = dict(label_smoothing=smoothing, z_loss=z_loss)
    xd, wd, td = put(x, 8), put(w, 8), t.to(DEV)
    _, lse = forward(g, xd, wd, td, **opts)
    sx, dx = strided(T, K, 8, float("nan"))
    sw, dw = strided(V, K, 16, float("nan"))
    g.xent_backward(xd, wd.t(), td, lse, d.to(DEV), dA=dx, dB=dw.t(), piece=piece, **opts)
    close(dx, ref.dx, ref.dx_err, True, "dx")
    close(dw, ref.dw, ref.dw_err, True, "dw")
    assert bool(sx[:, K:].isnan().all()) and bool(sw[:, K:].isnan().all())


@pytest.mark.parametrize("T,K,V", SHAPES + [(1100, 72, 2051), (40, 520, 9000), (2100, 64, 300)])
@pytest.mark.parametrize("piece", [0, 264])
def test_backward_exact_targets(g, T, K, V, piece):
    """With lse far above every logit the exponentials are exact zeros and G is
    minus dloss at the targets: dx = -dloss w[target], dw the sums of -dloss x
    over the rows of each target, exact for small integers (dloss 0, 1 or 2 over
    its largest, a power of two)."""
    gen = torch.Generator().manual_seed(7)
    x = torch.randint(-3, 4, (T, K), generator=gen).float()
    w = torch.randint(-3, 4, (V, K), generator=gen).float()
    t = torch.randint(0, V, (T,), generator=gen)
    t[torch.rand(T, generator=gen) < 0.2] = -1
    d = torch.randint(0, 3, (T,), generator=gen).float()
    keep = (t >= 0).float() * d
    at = t.clamp(min=0)
    dx = torch.empty(T, (K + 7) // 8 * 8, dtype=torch.bfloat16, device=DEV)[:, :K]
    dw = torch.empty(V, (K + 7) // 8 * 8, dtype=torch.bfloat16, device=DEV)[:, :K]
    lse = torch.full((T,), 1e30, device=DEV)
    for _ in range(2):
        g.xent_backward(put(x.bfloat16()), put(w.bfloat16()).t(), t.to(DEV), lse, d.to(DEV), dA=dx, dB=dw.t(),
                        ignore_index=-1, piece=piece)
        assert torch.equal(dx.cpu().float(), (-keep[:, None] * w[at]).bfloat16().float())
        want = torch.zeros(V, K).index_add_(0, at, -keep[:, None] * x)
        assert torch.equal(dw.cpu().float(), want.bfloat16().float())


@pytest.mark.parametrize("T,K,V", [(2048, 64, 300), (2500, 72, 1030)])
def test_many_rows(g, T, K, V):
    """From 2048 rows on, sixteen rows share a workgroup that joins segments."""
    x, w, t, _ = make(T, K, V, 16, 0.3)
    ref = Xent(x, w, t, smoothing=0.1, z_loss=1e-3)
    loss, lse = forward(g, put(x), put(w), t.to(DEV), label_smoothing=0.1, z_loss=1e-3)
    close(lse, ref.lse, ref.lse_err, False, "lse")
    close(loss, ref.loss, ref.loss_err, False, "loss")


@pytest.mark.parametrize("ignore", [0, 17, 2 ** 40, -(2 ** 63)])
def test_any_ignore_index(g, ignore):
    """The index to leave out may be a column of the vocabulary or no int32."""
    T, K, V = 90, 64, 120
    x, w, t, d = make(T, K, V, 17)
    t[::3] = ignore if abs(ignore) < 2 ** 31 else 5
    ref = Xent(x, w, t, ignore=ignore, dloss=d)
    xd, wd = put(x), put(w)
    for it in (torch.int64, torch.int32):
        td = t.to(DEV, it)
        loss, lse = forward(g, xd, wd, td, ignore_index=ignore)
        close(loss, ref.loss, ref.loss_err, False, "loss")
        dx = torch.empty_like(xd)
        g.xent_backward(xd, wd.t(), td, lse, d.to(DEV), dA=dx, ignore_index=ignore)
        close(dx, ref.dx, ref.dx_err, True, "dx")


@pytest.mark.parametrize("T", [8, 300])
def test_weights_past_four_gib(g, T):
    """A vocabulary whose weights span more than 4 GiB: rows on both sides of
    the 32-bit boundary, by the loss (targets there) and by single gradients."""
    K, V = 8192, 270000  # 4.4 GB
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    gen = torch.Generator(device=DEV).manual_seed(18)
    w = torch.empty(V, K, dtype=torch.bfloat16, device=DEV)
    for a in range(0, V, 30000):
        w[a:a + 30000] = torch.randn(min(30000, V - a), K, generator=gen, device=DEV) * K ** -0.5
    x = torch.randn(T, K, generator=gen, device=DEV).bfloat16()
    edge = 2 ** 32 // (2 * K)
    t = torch.randint(0, V, (T,), generator=gen, device=DEV)
    t[:4] = torch.tensor([edge - 1, edge, V - 1, 0], device=DEV)
    loss, lse = forward(g, x, w, t)
    want = torch.full((T,), -math.inf, device=DEV, dtype=torch.float64)
    for a in range(0, V, 30000):
        want = torch.logaddexp(want, torch.logsumexp((x.double() @ w[a:a + 30000].double().t()), 1))
    hit = (x.double() * w[t].double()).sum(1)
    # logits of about unit size over 8192 products: TAU * D is 1e-5 * 0.64 * 91
    assert float((lse.double() - want).abs().max()) <= 1e-3
    assert float((loss.double() - (want - hit)).abs().max()) <= 2e-3
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    d = torch.ones(T, device=DEV)
    g.xent_backward(x, w.t(), t, lse, d, dA=dx, dB=dw.t())
    rows = torch.tensor([0, edge - 1, edge, V - 1, V // 2], device=DEV)
    G = torch.exp(x.double() @ w[rows].double().t() - want[:, None])
    G -= (t[:, None] == rows[None]).double()
    wdw = G.t() @ x.double()
    # each of the T terms and the result rounded to bf16
    err = 2.0 ** -8 * (G.abs().t() @ x.double().abs() + wdw.abs()) + 1e-4
    assert bool(((dw[rows].double() - wdw).abs() <= err).all())
    wdx = torch.zeros(T, K, device=DEV, dtype=torch.float64)
    for a in range(0, V, 30000):
        wdx += torch.exp(x.double() @ w[a:a + 30000].double().t() - want[:, None]) @ w[a:a + 30000].double()
    wdx -= w[t].double()
    assert float((dx.double() - wdx).norm() / wdx.norm()) <= 1.5 * 2.0 ** -8


def test_large_and_tiny_logits(g):
    """Logits in the thousands of both signs: no exponential overflows."""
    T, K, V = 70, 64, 600
    x, w, t, d = make(T, K, V, 8)
    w = (w.float() * 600).bfloat16()
    ref = Xent(x, w, t, dloss=d)
    assert float(ref.lse.max()) > 1500
    xd, wd, td = put(x), put(w), t.to(DEV)
    loss, lse = forward(g, xd, wd, td)
    close(lse, ref.lse, ref.lse_err, False, "lse")
    close(loss, ref.loss, ref.loss_err, False, "loss")
    dx, dw = torch.empty_like(xd), torch.empty_like(wd)
    g.xent_backward(xd, wd.t(), td, lse, d.to(DEV), dA=dx, dB=dw.t())
    assert bool(dx.isfinite().all()) and bool(dw.isfinite().all())


def test_unknown_targets_and_masked_rows(g):
    """A target outside the vocabulary gives NaN in its row only; an ignored row
    gives an exact zero loss and gradient, also where its logits overflow."""
    T, K, V = 70, 64, 300
    for it in (torch.int64, torch.int32):
        x, w, t, _ = make(T, K, V, 9)
        t[3], t[4], t[5] = V, -7, -100
        x[5] = 3e38  # its logits overflow
        xd, wd, td = put(x), put(w), t.to(DEV, it)
        loss, lse = forward(g, xd, wd, td)
        assert bool(loss[3:5].isnan().all()) and float(loss[5]) == 0.0
        others = [i for i in range(T) if i not in (3, 4, 5)]
        assert bool(loss[others].isfinite().all())
        dx = torch.empty_like(xd)
        g.xent_backward(xd, wd.t(), td, lse, torch.ones(T, device=DEV), dA=dx)
        assert bool(dx[3:5].isnan().all()) and not bool(dx[5].any())
        assert bool(dx[others].isfinite().all())
    # a row of its own that is not finite is NaN, the others are not touched
    x, w, t, _ = make(T, K, V, 10)
    x[8, 2] = float("nan")
    loss, lse = forward(g, put(x), put(w), t.to(DEV))
    assert bool(loss[8].isnan()) and bool(lse[8].isnan()) and int(loss.isnan().sum()) == 1


def test_loss_gradient_extremes(g):
    """All loss gradients zero; one in the subnormals' reach; one infinite."""
    T, K, V = 40, 64, 200
    x, w, t, _ = make(T, K, V, 11)
    xd, wd, td = put(x), put(w), t.to(DEV)
    _, lse = forward(g, xd, wd, td)
    dx, dw = torch.empty_like(xd), torch.empty_like(wd)
    g.xent_backward(xd, wd.t(), td, lse, torch.zeros(T, device=DEV), dA=dx, dB=dw.t())
    assert not bool(dx.any()) and not bool(dw.any())
    tiny = torch.full((T,), 2.0 ** -120)
    g.xent_backward(xd, wd.t(), td, lse, tiny.to(DEV), dA=dx, dB=dw.t())
    ref = Xent(x, w, t, dloss=torch.ones(T))
    close(dx.double().cpu() * 2.0 ** 120, ref.dx, ref.dx_err + 2.0 ** -8 * ref.dx.abs() + 2.0 ** -13, False, "dx")
    big = torch.ones(T)
    big[2] = math.inf
    g.xent_backward(xd, wd.t(), td, lse, big.to(DEV), dA=dx)
    assert not bool(dx[2].isfinite().all()) and bool(dx[3:].isfinite().all())


def test_one_gradient_at_a_time(g):
    T, K, V = 150, 200, 700
    x, w, t, d = make(T, K, V, 12, 0.2)
    xd, wd, td, dd = put(x), put(w), t.to(DEV), d.to(DEV)
    _, lse = forward(g, xd, wd, td)
    dx, dw, dx1, dw1 = torch.empty_like(xd), torch.empty_like(wd), torch.empty_like(xd), torch.empty_like(wd)
    g.xent_backward(xd, wd.t(), td, lse, dd, dA=dx, dB=dw.t())
    g.xent_backward(xd, wd.t(), td, lse, dd, dA=dx1)
    g.xent_backward(xd, wd.t(), td, lse, dd, dB=dw1.t())
    assert torch.equal(dx, dx1) and torch.equal(dw, dw1)
    only = torch.empty(T, device=DEV)
    g.xent(xd, wd.t(), td, lse=only)
    assert torch.equal(only, lse)


def test_empty(g):
    K, V = 64, 100
    w = torch.randn(V, K, device=DEV).bfloat16()
    x = torch.empty(0, K, dtype=torch.bfloat16, device=DEV)
    none, t = torch.empty(0, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    g.xent(x, w.t(), t, none, none.clone())
    dw = torch.full_like(w, float("nan"))
    g.xent_backward(x, w.t(), t, none, none, dA=x.clone(), dB=dw.t())
    assert not bool(dw.any())


def test_streams_workspaces_and_graph(g):
    T, K, V = 200, 264, 1200
    x, w, t, d = make(T, K, V, 13, 0.2)
    xd, wd, td, dd = put(x), put(w), t.to(DEV), d.to(DEV)

    def outs():
        return torch.empty(T, device=DEV), torch.empty(T, device=DEV), torch.empty_like(xd), torch.empty_like(wd)

    def call(o, w1=None, w2=None, **kw):
        g.xent(xd, wd.t(), td, o[0], o[1], workspace=w1, **kw)
        g.xent_backward(xd, wd.t(), td, o[1], dd, dA=o[2], dB=o[3].t(), piece=500, workspace=w2, **kw)

    want = outs()
    call(want)
    own = outs()
    call(own, torch.empty(tg.tile_gemm_xent_workspace(g.handle, T, V, K), dtype=torch.uint8, device=DEV),
         torch.empty(tg.tile_gemm_xent_backward_workspace(g.handle, T, V, K, wd.stride(0), 500), dtype=torch.uint8,
                     device=DEV))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    side = [outs() for _ in streams]
    for s, o in zip(streams, side):
        call(o, stream=s)
    for s in streams:
        s.synchronize()
    graph, cap = torch.cuda.CUDAGraph(), outs()
    with torch.cuda.graph(graph):
        call(cap)
    for _ in range(3):
        for c in cap:
            c.fill_(float("nan"))
        graph.replay()
        eager = outs()
        call(eager)
        torch.cuda.synchronize()
        for o in (own, *side, cap, eager):
            assert all(torch.equal(a, c) for a, c in zip(o, want))


def test_step_of_block_and_head(g):
    """One training step as it is used: gated block, head, loss, both backward
    passes and an update, against autograd in 64 bits on the same bf16 values
    (h and dh rounded to bf16 where the step holds them so)."""
    T, K, F, V = 96, 128, 192, 600
    gen = torch.Generator().manual_seed(14)
    x = torch.randn(T, K, generator=gen).bfloat16()
    w1 = (torch.randn(2 * F, K, generator=gen) * K ** -0.5).bfloat16()
    w2 = (torch.randn(V, F, generator=gen) * F ** -0.5).bfloat16()
    t = torch.randint(0, V, (T,), generator=gen)
    t[::7] = -100
    n = int((t >= 0).sum())
    xd, w1d, w2d, td = x.to(DEV), w1.to(DEV), w2.to(DEV), t.to(DEV)
    h = torch.empty(T, F, dtype=torch.bfloat16, device=DEV)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    dh, dw2, dx, dw1 = torch.empty_like(h), torch.empty_like(w2d), torch.empty_like(xd), torch.empty_like(w1d)
    g.glu(xd, w1d.t(), h, gate=tg.Gate.GELU)
    g.xent(h, w2d.t(), td, loss, lse)
    g.xent_backward(h, w2d.t(), td, lse, torch.full((T,), 1.0 / n, device=DEV), dA=dh, dB=dw2.t())
    g.glu_backward(xd, w1d.t(), dh, dA=dx, dB=dw1.t(), gate=tg.Gate.GELU)
    w1d -= 0.1 * dw1

    X, W1 = x.double().requires_grad_(), w1.double().requires_grad_()
    z = X @ W1.T
    H = torch.nn.functional.gelu(z[:, :F]) * z[:, F:]
    H2, W2 = H.detach().bfloat16().double().requires_grad_(), w2.double().requires_grad_()
    L = torch.nn.functional.cross_entropy(H2 @ W2.T, t)
    L.backward()
    H.backward(H2.grad)
    assert abs(float(loss.sum()) / n - float(L)) <= 1e-3 * float(L)
    for got, want in ((dw2, W2.grad), (dh, H2.grad), (dx, X.grad), (dw1, W1.grad)):
        rel = float((got.cpu().double() - want).norm() / want.norm())
        # h's, dh's, dz's and the result's roundings, 0.58 * 2^-8 each
        assert rel <= 2.0 ** -8 * 2, rel


def test_refusals(g):
    T, K, V = 8, 64, 40
    x, w, t, d = make(T, K, V, 15)
    xd, wd, td, dd = put(x), put(w), t.to(DEV), d.to(DEV)
    loss, lse = forward(g, xd, wd, td)
    dx, dw = torch.empty_like(xd), torch.empty_like(wd)
    with pytest.raises(TypeError):
        g.xent(xd, wd.t(), td.float(), loss, lse)
    with pytest.raises(ValueError):
        g.xent(xd, wd.t(), td[:4], loss, lse)
    with pytest.raises(ValueError):
        g.xent(xd, wd.t(), t, loss, lse)
    with pytest.raises(TypeError):
        g.xent_backward(xd, wd.t(), td, lse.double(), dd, dA=dx)

    def fwd(**kw):
        a = {"A": xd, "B": wd.t(), "target": td, "loss": loss, "lse": lse} | kw
        return tg.tile_gemm_run_xent(g.handle, **a, check=False)

    def bwd(**kw):
        a = {"A": xd, "B": wd.t(), "target": td, "lse": lse, "dloss": dd, "dA": dx, "dB": dw.t()} | kw
        return tg.tile_gemm_run_xent_backward(g.handle, **a, check=False)

    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    assert fwd(loss=None, lse=None) == tg.Status.ERR_NULL_ARG
    assert fwd(lse=loss) == tg.Status.ERR_ALIAS
    assert fwd(label_smoothing=1.5) == tg.Status.ERR_BAD_SHAPE
    assert fwd(z_loss=float("nan")) == tg.Status.ERR_BAD_SHAPE
    assert fwd(B=wd.t().contiguous()) == tg.Status.ERR_BAD_STRIDE
    assert fwd(workspace=small) == tg.Status.ERR_WORKSPACE
    assert bwd(dA=None, dB=None) == tg.Status.ERR_NULL_ARG
    assert bwd(dA=xd) == tg.Status.ERR_ALIAS
    assert bwd(dB=wd.t()) == tg.Status.ERR_ALIAS
    assert bwd(workspace=small) == tg.Status.ERR_WORKSPACE
    assert bwd(piece=-1) == tg.Status.ERR_BAD_SHAPE
    torch.cuda.synchronize()
