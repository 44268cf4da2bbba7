"""Edge calls of the gated block and of the cross entropy head on the GPU."""

import math

import pytest
import torch

import tile_partitioned_dense_amd as tg
from test_gpu_glu import DEV, put
from train_helpers import EVAL, GATES, HALF, TAU, Glu, Xent, act_slope, close

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


def masked_head(T, K, V, masked, seed):
    """x, w and targets of a head whose columns `masked` have logit -inf, by a
    last value of 1 in x and of -inf in their weights (0 in the others'), and
    the reference over the other columns, their numbers in `kept`."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=gen).bfloat16()
    w = (torch.randn(V, K, generator=gen) * 2 * K ** -0.5).bfloat16()
    x[:, -1], w[:, -1] = 1.0, 0.0
    w[masked, -1] = -float("inf")
    kept = torch.ones(V, dtype=torch.bool)
    kept[masked] = False
    kept = kept.nonzero()[:, 0]
    at = torch.randint(0, len(kept), (T,), generator=gen)
    d = torch.rand(T, generator=gen)
    return x, w, kept[at], d, kept, Xent(x, w[kept], at, dloss=d)


# one to many tokens: 32-column segments, then those of 64 to 128 columns
@pytest.mark.parametrize("T,K,V", [(1, 64, 33), (7, 72, 65), (40, 64, 1300), (300, 72, 4129), (1300, 72, 6161),
                                   (2050, 72, 8209), (50, 65, 300), (700, 65, 900)])
@pytest.mark.parametrize("which", ["last", "first segments", "last segments", "all but one"])
def test_columns_of_minus_infinity(g, T, K, V, which):
    """Logits of -inf count for nothing, alone in the last segment of a row as
    well as over whole segments; the gradients of their weights are zero."""
    wide = min(V - 1, 256)
    masked = {"last": [V - 1], "first segments": list(range(wide)), "last segments": list(range(V - wide, V)),
              "all but one": [v for v in range(V) if v != V // 2]}[which]
    x, w, t, d, kept, ref = masked_head(T, K, V, masked, 3)
    xd, wd, td = put(x), put(w), t.to(DEV)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    g.xent(xd, wd.t(), td, loss, lse)
    close(lse, ref.lse, ref.lse_err, False, "lse")
    close(loss, ref.loss, ref.loss_err, False, "loss")
    dx, dw = put(torch.zeros_like(x)), put(torch.zeros_like(w))
    g.xent_backward(xd, wd.t(), td, lse, d.to(DEV), dA=dx, dB=dw.t())
    # (the last value of dx is the sum over 0 * -inf)
    close(dx[:, :-1], ref.dx[:, :-1], ref.dx_err[:, :-1], True, "dx")
    close(dw[kept.to(DEV)], ref.dw, ref.dw_err, True, "dw")
    assert not bool(dw[masked].any())


@pytest.mark.parametrize("T,K,V", [(1, 64, 33), (40, 64, 1300), (300, 72, 4129), (1300, 72, 6161), (700, 65, 900)])
@pytest.mark.parametrize("lowest", [torch.finfo(torch.bfloat16).min, -2e38, -1e30, -1e10, -1e9])
def test_columns_of_the_lowest_value(g, T, K, V, lowest):
    """Logits of the type's lowest value, whose multiples overflow, and of other
    large negative values, whose multiples are rounded by more than any exponent,
    count for nothing like those of -inf, whole segments of them too."""
    for masked in ([V - 1], list(range(min(V - 1, 256))), [v for v in range(V) if v != V // 2]):
        x, w, t, d, kept, ref = masked_head(T, K, V, masked, 9)
        w[masked, -1] = lowest
        xd, wd, td = put(x), put(w), t.to(DEV)
        loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        g.xent(xd, wd.t(), td, loss, lse)
        close(lse, ref.lse, ref.lse_err, False, "lse")
        close(loss, ref.loss, ref.loss_err, False, "loss")
        dx, dw = put(torch.zeros_like(x)), put(torch.zeros_like(w))
        g.xent_backward(xd, wd.t(), td, lse, d.to(DEV), dA=dx, dB=dw.t())
        close(dx, ref.dx, ref.dx_err, True, "dx")
        close(dw[kept.to(DEV)], ref.dw, ref.dw_err, True, "dw")
        assert not bool(dw[masked].any())


@pytest.mark.parametrize("T,K,V", [(6, 64, 300), (70, 72, 1300), (300, 72, 2051)])
@pytest.mark.parametrize("lowest", [torch.finfo(torch.bfloat16).min, -1e30, -1e10])
def test_rows_of_the_lowest_value(g, T, K, V, lowest):
    """Rows of which nothing is left (every third): all logits are the same large
    negative value, so the loss is log V and lse that value, the sum of V of them
    to the last place; every column's e^(l - lse) is 1 by that lse, and the
    gradients are those of the formula, without an infinity."""
    gen = torch.Generator().manual_seed(10)
    x = torch.randn(T, K, generator=gen).bfloat16()
    w = (torch.randn(V, K, generator=gen) * 2 * K ** -0.5).bfloat16()
    t = torch.randint(0, V, (T,), generator=gen)
    d = torch.rand(T, generator=gen)
    out = torch.zeros(T, dtype=torch.bool)
    out[::3] = True
    x[:, -1], x[out], w[:, -1] = 0.0, 0.0, 0.0
    ref = Xent(x, w, t, dloss=d)
    x[out, -1], w[:, -1] = 1.0, lowest
    one = float(w[0, -1].float())
    xd, wd, td = put(x), put(w), t.to(DEV)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    g.xent(xd, wd.t(), td, loss, lse)
    assert bool((lse.cpu()[out] == one).all())
    assert float((loss.cpu()[out].double() - math.log(V)).abs().max()) <= EVAL * math.log(V)
    close(lse[~out.to(DEV)], ref.lse[~out], ref.lse_err[~out], False, "lse")
    close(loss[~out.to(DEV)], ref.loss[~out], ref.loss_err[~out], False, "loss")
    dx, dw = put(torch.zeros_like(x)), put(torch.zeros_like(w))
    g.xent_backward(xd, wd.t(), td, lse, d.to(DEV), dA=dx, dB=dw.t())
    close(dx[~out.to(DEV), :-1], ref.dx[~out, :-1], ref.dx_err[~out, :-1], True, "dx")
    # G = d (1 - [target]) in those rows, held in bf16
    G = d[out].double()[:, None] * (1 - torch.nn.functional.one_hot(t[out], V).double())
    w64 = w.double()[:, :-1]
    err = HALF * G.abs() @ w64.abs() + TAU * G.abs() @ w64.abs()
    close(dx[out.to(DEV), :-1], G @ w64, err, True, "dx of the masked rows")
    # x is zero in those rows but for its last value
    close(dw[:, :-1], ref.dw[:, :-1], ref.dw_err[:, :-1], True, "dw")
    close(dw[:, -1], G.sum(0), (HALF + TAU) * G.sum(0), True, "dw of the last value")


@pytest.mark.parametrize("T,V", [(5, 300), (200, 2000)])
def test_rows_of_infinities(g, T, V):
    """A row whose logits are all -inf has a log-sum-exp of -inf, one with a
    logit of inf one of inf; the other rows do not see it."""
    K = 64
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(T, K, generator=gen).bfloat16()
    w = (torch.randn(V, K, generator=gen) * K ** -0.5).bfloat16()
    x[:, -2:] = 0.0
    w[:, -1], w[:, -2] = 1.0, 0.0
    w[V // 3, -2] = 1.0
    t = torch.randint(0, V, (T,), generator=gen)
    want = Xent(x, w, t)
    x[1, -1], x[3, -2] = -float("inf"), 3e38
    x[3, :-2], w[V // 3, -2] = 0.0, 3e38
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    g.xent(put(x), put(w).t(), t.to(DEV), loss, lse)
    assert float(lse[1]) == -float("inf") and float(lse[3]) == float("inf")
    others = [i for i in range(T) if i not in (1, 3)]
    close(lse[others], want.lse[others], want.lse_err[others], False, "lse")
    close(loss[others], want.loss[others], want.loss_err[others], False, "loss")


@pytest.mark.parametrize("T,V", [(1, 40), (30, 1300), (300, 4129), (1300, 6161), (2050, 8209)])
def test_nearly_certain_tokens(g, T, V):
    """Logits given exactly: the target's m of 20 to 127.5, one that is 2 to 20
    below it, the others 1000 below. The loss log(1 + e^-(2 to 20)) is never
    negative and off by at most 2^-21: the maximum's exponential is 1, the
    other's is at most e^-2 and within 2^-19 of itself (2^-23 for the hardware's,
    two roundings of an exponent of at most 29, and a product), and the sums, two
    joins of segments and the logarithm add half a unit in the last place of a
    value below 2, 2^-24, each."""
    K = 64
    gen = torch.Generator().manual_seed(5)
    top = 20 + 0.5 * torch.randint(0, 216, (K,), generator=gen)
    gap = torch.randint(2, 21, (K,), generator=gen)
    hit = torch.randint(0, V, (K,), generator=gen)
    near = (hit + torch.randint(1, V, (K,), generator=gen)) % V
    w = (top - 1000).expand(V, K).clone()
    w[hit, torch.arange(K)], w[near, torch.arange(K)] = top, top - gap
    k = torch.randint(0, K, (T,), generator=gen)  # a token takes one column of w
    x = torch.nn.functional.one_hot(k, K).bfloat16()
    assert torch.equal(w.bfloat16()[hit, torch.arange(K)].float(), top)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    g.xent(put(x), put(w.bfloat16()).t(), hit[k].to(DEV), loss, lse)
    want = torch.log1p(torch.exp(-gap.double()))[k]
    off = (loss.cpu().double() - want).abs().max()
    assert float(loss.min()) >= 0 and float(off) <= 2.0 ** -21, (float(loss.min()), float(off))


@pytest.mark.parametrize("gate", ["RELU", "SIGMOID"])
@pytest.mark.parametrize("T,K,F", [(1, 64, 16), (33, 136, 200), (300, 72, 1032), (1300, 72, 4112)])
def test_units_switched_off(g, gate, T, K, F):
    """A gate bias of -inf gives zeros in its column of h and of both gradients
    of the pre-activations, one of NaN NaN in its column of h alone. The
    reference has -1e4 in the place of -inf: no difference in 64 bits, but for
    the error bounds, which the exact zeros stand for here."""
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(T, K, generator=gen).bfloat16()
    w = (torch.randn(2 * F, K, generator=gen) * K ** -0.5).bfloat16()
    b = torch.randn(2 * F, generator=gen)
    dh = torch.randn(T, F, generator=gen).bfloat16()
    off = torch.arange(0, F, 3)
    b[off] = -1e4
    ref = Glu(x, w, b, gate, dh)
    on = torch.ones(F, dtype=torch.bool)
    on[off] = False
    b[off] = -float("inf")
    xd, wd, bd = put(x), put(w), b.to(DEV)
    for weights in (wd.t(), put(w.T.contiguous())):
        for dt in (torch.float32, torch.bfloat16):
            h = torch.full((T, F), float("nan"), device=DEV, dtype=dt)
            g.glu(xd, weights, h, gate=tg.Gate[gate], bias=bd)
            assert not bool(h[:, off].any())
            close(h[:, on], ref.h[:, on], ref.h_err[:, on], dt == torch.bfloat16, "h")
    dx, dw, db = torch.empty_like(xd), torch.empty_like(wd), torch.empty_like(bd)
    g.glu_backward(xd, wd.t(), put(dh), dA=dx, dB=dw.t(), dbias=db, gate=tg.Gate[gate], bias=bd)
    both = torch.cat([off, F + off])
    assert not bool(db[both].any()) and not bool(dw[both].any())
    keep = torch.cat([on, on])
    close(db[keep], ref.dbias[keep], ref.dbias_err[keep], False, "dbias")
    close(dw[keep], ref.dw[keep], ref.dw_err[keep], True, "dw")
    close(dx, ref.dx, ref.dx_err, True, "dx")
    b[1] = float("nan")
    g.glu(xd, wd.t(), h, gate=tg.Gate[gate], bias=b.to(DEV))
    assert bool(h[:, 1].isnan().all()) and int(h.isnan().sum()) == T


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T", [4, 300])
def test_largest_preactivations(g, gate, T):
    """Gate pre-activations of up to 3e38, whose squares and cubes overflow:
    gates are 0 or z (or 1) there and their slopes 0 or 1 (or 0). x is zero, so
    the pre-activations are the biases; up is 1 and dh 1/4 in four rows, so h is
    the gate and dbias slope and gate."""
    K, size = 64, torch.tensor([20.0, 1e3, 1e10, 1e13, 1.7e19, 5e19, 1e20, 3e38])
    z = torch.cat([size, -size]).repeat(20)
    F = len(z)
    b = torch.cat([z, torch.ones(F)])
    x, w = torch.zeros(T, K).bfloat16(), torch.zeros(2 * F, K).bfloat16()
    dh = torch.zeros(T, F).bfloat16()
    dh[:4] = 0.25
    act, slope = act_slope(z.double(), gate)
    xd, wd, bd = put(x), put(w), b.to(DEV)
    h, db = torch.empty(T, F, device=DEV), torch.empty(2 * F, device=DEV)
    g.glu(xd, wd.t(), h, gate=tg.Gate[gate], bias=bd)
    g.glu_backward(xd, wd.t(), put(dh), dbias=db, gate=tg.Gate[gate], bias=bd)
    # e^-20 is 2e-9: what gate and slope are off their limits at 20 already
    close(h, act.expand(T, F), EVAL * act.abs() + 1e-7, False, "h")
    close(db, torch.cat([slope, act]), EVAL * torch.cat([slope, act]).abs() + 1e-6, False, "dbias")


@pytest.mark.parametrize("pitch", [0, 3, 8, 2 ** 31 + 4, 2 ** 40])
@pytest.mark.parametrize("K", [65, 72, 1032])
def test_one_row_of_any_stride(g, pitch, K):
    """A single row of x, dC and the results has no row stride that counts."""
    V, F = 1300, 200
    gen = torch.Generator(device=DEV).manual_seed(7)
    ld = (K + 7) // 8 * 8
    w = (torch.randn(V, ld, generator=gen, device=DEV) * K ** -0.5).bfloat16()[:, :K]
    w2 = w[:2 * F]
    x = torch.randn(ld, generator=gen, device=DEV).bfloat16()[:K]
    dh = torch.randn(F, generator=gen, device=DEV).bfloat16()
    t, d = torch.tensor([V // 2], device=DEV), torch.ones(1, device=DEV)

    def row(v, apart):
        return v.as_strided((1, len(v)), (apart, 1))

    def run(apart):
        o = [torch.full((n,), float("nan"), device=DEV) for n in (1, 1, 2 * F)]
        r = [torch.full((n,), float("nan"), dtype=torch.bfloat16, device=DEV) for n in (F, ld, ld)]
        m = [torch.full((n, ld), float("nan"), dtype=torch.bfloat16, device=DEV)[:, :K] for n in (V, 2 * F)]
        xr = row(x, apart)
        g.xent(xr, w.t(), t, o[0], o[1])
        g.xent_backward(xr, w.t(), t, o[1], d, dA=row(r[1][:K], apart), dB=m[0].t())
        g.glu(xr, w2.t(), row(r[0], apart), gate=tg.Gate.GELU)
        g.glu_backward(xr, w2.t(), row(dh, apart), dA=row(r[2][:K], apart), dB=m[1].t(), dbias=o[2], gate=tg.Gate.GELU)
        return o + [r[0], r[1][:K], r[2][:K]] + m

    for a, b in zip(run(pitch), run(ld)):
        assert bool(b.isfinite().all()) and torch.equal(a, b)


@pytest.mark.parametrize("T,K,V", [(1, 64, 1), (1, 136, 50), (33, 72, 40), (70, 65, 33), (300, 72, 21)])
def test_pieces_of_one_column(g, T, K, V):
    """The smallest pieces of a vocabulary: a column at a time."""
    gen = torch.Generator().manual_seed(8)
    x = torch.randn(T, K, generator=gen).bfloat16()
    w = (torch.randn(V, K, generator=gen) * 2 * K ** -0.5).bfloat16()
    t = torch.randint(0, V, (T,), generator=gen)
    t[1::5] = -100
    d = torch.rand(T, generator=gen)
    ref = Xent(x, w, t, smoothing=0.1, z_loss=1e-3, dloss=d)
    opts = dict(label_smoothing=0.1, z_loss=1e-3)
    xd, wd, td = put(x), put(w), t.to(DEV)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    g.xent(xd, wd.t(), td, loss, lse, **opts)
    dx, dw = put(torch.zeros_like(x)), put(torch.zeros_like(w))
    g.xent_backward(xd, wd.t(), td, lse, d.to(DEV), dA=dx, dB=dw.t(), piece=1, **opts)
    close(dx, ref.dx, ref.dx_err, True, "dx")
    close(dw, ref.dw, ref.dw_err, True, "dw")
