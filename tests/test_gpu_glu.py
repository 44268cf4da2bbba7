"""Gated block and its backward pass on the GPU, against 64-bit references."""

import pytest
import torch

import tile_partitioned_dense_amd as tg
from train_helpers import GATES, Glu, close

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def g():
    with tg.TileGemm(0) as handle:
        yield handle


def strided(rows, cols, pad, fill=0.0, dtype=torch.bfloat16):
    """A rows x cols view whose rows are a multiple of 16 bytes plus `pad` apart."""
    ld = (cols + 7) // 8 * 8 + pad
    store = torch.full((max(rows, 1), ld), fill, dtype=dtype, device=DEV)
    return store, store[:rows, :cols]


def put(t, pad=0):
    _, v = strided(*t.shape, pad, dtype=t.dtype)
    v.copy_(t)
    return v


def make(T, K, F, seed, bias, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=gen).bfloat16()
    w = (torch.randn(2 * F, K, generator=gen) * (scale * K ** -0.5)).bfloat16()
    b = torch.randn(2 * F, generator=gen) * 0.5 if bias else None
    dh = torch.randn(T, F, generator=gen).bfloat16()
    return x, w, b, dh


# one token, few rows (the stream kernel's row blocks), one tile, several, ragged
SHAPES = [(1, 64, 8), (3, 72, 24), (33, 1000, 200), (64, 136, 64), (65, 200, 136), (130, 96, 264),
          (257, 328, 520), (300, 65, 128), (520, 1032, 384)]


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,K,F", [(1, 64, 8), (33, 1000, 200), (130, 96, 264)])
def test_forward(g, gate, T, K, F):
    for bias in (False, True):
        x, w, b, _ = make(T, K, F, 11, bias, 2.0)
        ref = Glu(x, w, b, gate)
        xd, wd, bd = put(x, 8), put(w), b.to(DEV) if bias else None
        for dt in (torch.float32, torch.bfloat16):
            store, h = strided(T, F, 8, float("nan"), dt)
            g.glu(xd, wd.t(), h, gate=tg.Gate[gate], bias=bd)
            close(h, ref.h, ref.h_err, dt == torch.bfloat16, f"h {gate} {dt} bias={bias}")
            assert bool(store[:, F:].isnan().all())


@pytest.mark.parametrize("T,K,F", [(5, 64, 40), (200, 120, 72)])
@pytest.mark.parametrize("gate", GATES)
def test_forward_row_major_weights(g, gate, T, K, F):
    x, w, b, _ = make(T, K, F, 12, True)
    ref = Glu(x, w, b, gate)
    h = torch.empty(T, F, device=DEV)
    g.glu(put(x), put(w.T.contiguous()), h, gate=tg.Gate[gate], bias=b.to(DEV))
    close(h, ref.h, ref.h_err, False, f"h {gate}")


def test_silu_gate_is_the_swiglu_epilogue(g):
    """The same function: bit for bit with a row-major B, where it is the same
    kernel, within both results' bounds otherwise."""
    x, w, b, _ = make(300, 328, 136, 13, True)
    ref = Glu(x, w, b, "SILU")
    xd, wd, bd = put(x), put(w), b.to(DEV)
    wr = put(w.T.contiguous())
    for weights in (wr, wd.t()):
        h, h2 = (torch.empty(300, 136, device=DEV) for _ in range(2))
        g.glu(xd, weights, h, bias=bd)
        g(xd, weights, h2, bias=bd, act=tg.Act.SWIGLU)
        close(h, ref.h, ref.h_err, False, "glu")
        close(h2, ref.h, ref.h_err, False, "swiglu")
        assert weights is not wr or torch.equal(h, h2)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,K,F", SHAPES)
def test_backward(g, gate, T, K, F):
    bias = T % 2 == 1
    x, w, b, dh = make(T, K, F, 21, bias, 1.5)
    ref = Glu(x, w, b, gate, dh)
    sx, dx = strided(T, K, 8, float("nan"))
    sw, dw = strided(2 * F, K, 16, float("nan"))
    db = torch.full((2 * F,), float("nan"), device=DEV)
    g.glu_backward(put(x, 8), put(w, 8).t(), put(dh, 16), dA=dx, dB=dw.t(), gate=tg.Gate[gate],
                   bias=b.to(DEV) if bias else None, dbias=db)
    close(db, ref.dbias, ref.dbias_err, False, "dbias")
    close(dx, ref.dx, ref.dx_err, True, "dx")
    close(dw, ref.dw, ref.dw_err, True, "dw")
    # what lies behind the rows stays as it was
    assert bool(sx[:, K:].isnan().all()) and bool(sw[:, K:].isnan().all())


def test_no_contraction(g):
    """K = 0: the gated block of the biases."""
    T, F = 5, 24
    b = torch.randn(2 * F)
    ref = Glu(torch.zeros(T, 8).bfloat16(), torch.zeros(2 * F, 8).bfloat16(), b, "GELU")
    h = torch.empty(T, F, device=DEV)
    none = torch.empty(T, 0, dtype=torch.bfloat16, device=DEV)
    g.glu(none, torch.empty(2 * F, 0, dtype=torch.bfloat16, device=DEV).t(), h, gate=tg.Gate.GELU, bias=b.to(DEV))
    close(h, ref.h, ref.h_err, False, "h")


def test_masked_rows_stay_out(g):
    """Columns and rows past the edges of a tile read the neighbours' memory or
    zeros; not even infinities there reach a result."""
    T, K, F = 70, 72, 40
    x, w, b, dh = make(T, K, F, 22, True)
    big_x = torch.full((T + 200, K), float("inf"), dtype=torch.bfloat16, device=DEV)
    big_w = torch.full((2 * F + 200, K), float("inf"), dtype=torch.bfloat16, device=DEV)
    big_d = torch.full((T + 200, F), float("inf"), dtype=torch.bfloat16, device=DEV)
    big_x[:T], big_w[:2 * F], big_d[:T] = x.to(DEV), w.to(DEV), dh.to(DEV)
    ref = Glu(x, w, b, "GELU_TANH", dh)
    dx, dw = torch.empty(T, K, dtype=torch.bfloat16, device=DEV), torch.empty(2 * F, K, dtype=torch.bfloat16, device=DEV)
    db = torch.empty(2 * F, device=DEV)
    g.glu_backward(big_x[:T], big_w[:2 * F].t(), big_d[:T], dA=dx, dB=dw.t(), dbias=db, bias=b.to(DEV),
                   gate=tg.Gate.GELU_TANH)
    close(db, ref.dbias, ref.dbias_err, False, "dbias")
    close(dx, ref.dx, ref.dx_err, True, "dx")
    close(dw, ref.dw, ref.dw_err, True, "dw")


def integers(T, K, F, seed):
    """Small integers for which every dz of a relu gate is exact in bf16: up to
    three non-zeros of +-1 in a row of x against w in -2..2, dh in -2..2."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.zeros(T, K)
    for _ in range(3):
        at = torch.randint(0, K, (T,), generator=gen)
        x[torch.arange(T), at] = torch.randint(0, 2, (T,), generator=gen) * 2.0 - 1
    w = torch.randint(-2, 3, (2 * F, K), generator=gen).float()
    dh = torch.randint(-2, 3, (T, F), generator=gen).float()
    return x, w, dh


@pytest.mark.parametrize("T,K,F", SHAPES + [(1029, 72, 1032), (70, 2056, 1000), (2100, 264, 40)])
def test_backward_exact_on_integers(g, T, K, F):
    """|z| <= 6, so dz = dh z (or dh relu(z)) is an integer of at most 12: exact in
    bf16, and every sum of their products (at most 2 * 12 * 4200 < 2^24) exact in
    fp32. The gradients are then the exact sums rounded once."""
    x, w, dh = integers(T, K, F, 31)
    z = x.double() @ w.double().T
    gate, up = z[:, :F], z[:, F:]
    dz = torch.cat([dh * up * (gate > 0), dh * gate.clamp(min=0)], 1)
    dx = torch.empty(T, (K + 7) // 8 * 8, dtype=torch.bfloat16, device=DEV)[:, :K]
    dw = torch.empty(2 * F, (K + 7) // 8 * 8, dtype=torch.bfloat16, device=DEV)[:, :K]
    db = torch.empty(2 * F, device=DEV)
    for _ in range(2):
        g.glu_backward(put(x.bfloat16()), put(w.bfloat16()).t(), put(dh.bfloat16()), dA=dx, dB=dw.t(),
                       gate=tg.Gate.RELU, dbias=db)
        assert torch.equal(db.cpu().double(), dz.sum(0))
        assert torch.equal(dx.cpu(), (dz @ w.double()).bfloat16())
        assert torch.equal(dw.cpu(), (dz.T @ x.double()).bfloat16())


def test_backward_against_differences(g):
    """The gradients' directional derivative against a central difference of the
    fp32 forward: sum(h dh) changes by 2 e <grad, d> within the fp32 results'
    errors and the gradients' bf16 roundings."""
    T, K, F = 40, 128, 48
    x, w, b, dh = make(T, K, F, 41, True)
    gen = torch.Generator().manual_seed(42)
    xd, wd, bd, dhd = put(x), put(w), b.to(DEV), put(dh)
    dx, dw, db = torch.empty_like(xd), torch.empty_like(wd), torch.empty_like(bd)
    for gate in GATES:
        if gate == "RELU":
            continue  # no derivative at its corner
        g.glu_backward(xd, wd.t(), dhd, dA=dx, dB=dw.t(), gate=tg.Gate[gate], bias=bd, dbias=db)
        e = 2.0 ** -6
        dirs = [torch.randint(-1, 2, t.shape, generator=gen).double() for t in (x, w, b)]

        def f(sign):
            ref = Glu(x.double() + sign * e * dirs[0], w.double() + sign * e * 0.1 * dirs[1],
                      b.double() + sign * e * dirs[2], gate)
            return float((ref.h * dh.double()).sum())

        slope = (f(1) - f(-1)) / (2 * e)
        parts = [dx.cpu().double() * dirs[0], dw.cpu().double() * 0.1 * dirs[1], db.cpu().double() * dirs[2]]
        got = float(sum(p.sum() for p in parts))
        size = float(sum((p ** 2).sum() for p in parts)) ** 0.5
        # roundings of the gradients in quadrature (2 HALF of each), the
        # difference's third-order term by halving the step
        e, coarse = e / 2, slope
        slope = (f(1) - f(-1)) / (2 * e)
        tol = 2 * 2.0 ** -8 * size * 3 + 2 * abs(slope - coarse)
        assert abs(got - slope) <= tol, (gate, got, slope, tol)


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("db",), ("dx", "db")])
def test_backward_of_some_gradients(g, want):
    T, K, F = 150, 200, 136
    x, w, b, dh = (t.to(DEV) for t in make(T, K, F, 51, True))
    full = {"dx": torch.empty_like(x), "dw": torch.empty_like(w), "db": torch.empty_like(b)}
    g.glu_backward(x, w.t(), dh, dA=full["dx"], dB=full["dw"].t(), dbias=full["db"], bias=b)
    part = {k: torch.empty_like(full[k]) for k in want}
    g.glu_backward(x, w.t(), dh, dA=part.get("dx"), dB=part["dw"].t() if "dw" in part else None,
                   dbias=part.get("db"), bias=b)
    for k in want:
        assert torch.equal(part[k], full[k])


def test_empty(g):
    K, F = 64, 16
    w = torch.randn(2 * F, K, device=DEV).bfloat16()
    x = torch.empty(0, K, dtype=torch.bfloat16, device=DEV)
    dw, db = torch.full_like(w, float("nan")), torch.full((2 * F,), float("nan"), device=DEV)
    g.glu_backward(x, w.t(), torch.empty(0, F, dtype=torch.bfloat16, device=DEV), dA=x.clone(), dB=dw.t(),
                   dbias=db)
    assert not bool(dw.any()) and not bool(db.any())
    x = torch.randn(5, K, device=DEV).bfloat16()
    dx = torch.full_like(x, float("nan"))
    g.glu_backward(x, torch.empty(0, K, dtype=torch.bfloat16, device=DEV).t(),
                   torch.empty(5, 0, dtype=torch.bfloat16, device=DEV), dA=dx)
    assert not bool(dx.any())


def test_streams_workspaces_and_graph(g):
    """A side stream, a caller's workspace, two calls at once with one each, and
    a captured call replayed between eager ones: all the same bits."""
    T, K, F = 300, 264, 136
    x, w, b, dh = (t.to(DEV) for t in make(T, K, F, 61, True))

    def outs():
        return torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)

    def call(o, **kw):
        g.glu_backward(x, w.t(), dh, dA=o[0], dB=o[1].t(), dbias=o[2], bias=b, gate=tg.Gate.GELU, **kw)

    want = outs()
    call(want)
    need = tg.tile_gemm_glu_backward_workspace(g.handle, T, 2 * F, K)
    own = outs()
    call(own, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
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
        for t in cap:
            t.fill_(float("nan"))
        graph.replay()
        eager = outs()
        call(eager)
        torch.cuda.synchronize()
        for o in (own, *side, cap, eager):
            assert all(torch.equal(a, c) for a, c in zip(o, want))


def test_refusals(g):
    T, K, F = 8, 64, 16
    x, w, b, dh = (t.to(DEV) for t in make(T, K, F, 71, True))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    run = g.glu_backward
    with pytest.raises(TypeError):
        run(x.float(), w.t(), dh, dA=dx)
    with pytest.raises(ValueError):
        run(x, w.t(), dh[:, :8], dA=dx)
    with pytest.raises(ValueError):
        run(x.cpu(), w.t(), dh, dA=dx)
    with pytest.raises(ValueError):
        run(x, w.t(), dh, dA=dx, dbias=b[:4])

    def status(**kw):
        a = {"A": x, "B": w.t(), "dC": dh, "dA": dx, "dB": dw.t()} | kw
        return tg.tile_gemm_run_glu_backward(g.handle, **a, check=False)

    assert status(B=w.t().contiguous()) == tg.Status.ERR_BAD_STRIDE
    assert status(dA=x) == tg.Status.ERR_ALIAS
    assert status(dB=w.t()) == tg.Status.ERR_ALIAS
    assert status(dA=None, dB=None) == tg.Status.ERR_NULL_ARG
    assert status(gate=9) == tg.Status.ERR_EPILOGUE
    assert status(workspace=torch.empty(16, dtype=torch.uint8, device=DEV)) == tg.Status.ERR_WORKSPACE
    odd = torch.empty(T, K + 4, dtype=torch.bfloat16, device=DEV)[:, :K]
    assert status(A=odd) == tg.Status.ERR_MISALIGNED
    assert tg.tile_gemm_run_glu(g.handle, x, w.t(), torch.empty(T, F, device=DEV), gate=5,
                                check=False) == tg.Status.ERR_EPILOGUE
    torch.cuda.synchronize()
