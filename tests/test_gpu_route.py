"""Routing to experts, its gradient, the tokens' order by expert and the
weighted sum of the experts' rows, against plain 64-bit references; and the
whole of it with the E4M3 products, as it is used."""

import pytest
import torch

import block_helpers as bh
import tile_partitioned_dense_amd as tg

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
I32 = torch.int32


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    with tg.TileGemm(0) as gg:
        yield gg


def gen(seed):
    return torch.Generator().manual_seed(seed)


def run_route(g, logits, k, **kw):
    T = logits.shape[0]
    ids = torch.full((T, k), -9, dtype=I32, device="cuda")
    w = torch.full((T, k), NAN, device="cuda")
    bias = kw.pop("bias", None)
    g.route(logits.cuda(), ids, w, bias=None if bias is None else bias.cuda(), **kw)
    return ids.cpu(), w.cpu()


def check_route(g, logits, k, score="SOFTMAX", **kw):
    want_ids, want_w = bh.route(logits, k, score, **{"renorm" if n == "renormalize" else n: v for n, v in kw.items()})
    ids, w = run_route(g, logits, k, score=tg.Score[score], **kw)
    assert torch.equal(ids.long(), want_ids)
    # 64-bit scores, rounded once
    assert bool(((w.double() - want_w).abs() <= 2.0 ** -24 * 1.01 * want_w.abs() + 2.0 ** -149).all())


@pytest.mark.parametrize("score", ["SOFTMAX", "SIGMOID"])
@pytest.mark.parametrize("T,E,k,kw", [
    (1, 1, 1, {}),
    (1, 8, 2, dict(renormalize=False)),
    (7, 60, 6, dict(scale=2.5)),
    (33, 64, 8, dict(groups=8, top_groups=3)),
    (20, 65, 5, {}),
    (9, 128, 32, dict(renormalize=False, scale=-1.5)),
    (30, 256, 8, dict(groups=8, top_groups=4, scale=2.5)),
    (17, 96, 6, dict(groups=3, top_groups=2, group_top=1)),
    (5, 12, 4, dict(groups=6, top_groups=2)),
    (5, 6, 3, dict(groups=6, top_groups=4)),                   # groups of one
    (11, 320, 10, dict(groups=64, top_groups=5)),
    (6, 513, 7, {}),
    (3, 1024, 16, dict(groups=4, top_groups=1)),
    (4, 24, 24, {}),                                           # all of them
])
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("bias", [False, True], ids=["plain", "bias"])
def test_route(g, T, E, k, kw, score, bf16, bias):
    r = gen(T * 1000 + E + k)
    logits = torch.randn(T, E, generator=r) * 2
    logits = logits.bfloat16() if bf16 else logits  # (bf16: equal logits among them)
    check_route(g, logits, k, score, **kw, **(dict(bias=torch.randn(E, generator=r) * 0.1) if bias else {}))


@pytest.mark.parametrize("score", ["SOFTMAX", "SIGMOID"])
@pytest.mark.parametrize("groups", [1, 4])
def test_close_and_equal_scores(g, score, groups):
    """Equal logits by index; neighbours in fp32, whose scores are equal there, by their order."""
    logits = torch.zeros(6, 64)
    logits[1] = 3.0
    logits[2] = torch.nextafter(torch.tensor(2.0), torch.tensor(3.0))
    logits[2, 40] = torch.nextafter(logits[2, 0], torch.tensor(3.0))
    logits[3, ::3] = -0.0
    logits[4] = torch.arange(64) % 5
    logits[5] = 20.0
    logits[5, 63] = torch.nextafter(torch.tensor(20.0), torch.tensor(30.0))
    check_route(g, logits, 6, score, groups=groups, top_groups=max(1, groups // 2))


@pytest.mark.parametrize("score", ["SOFTMAX", "SIGMOID"])
@pytest.mark.parametrize("groups", [1, 3])
def test_masked_logits(g, score, groups):
    """-inf (experts that are switched off), NaN, the largest values, whole rows of them."""
    r = gen(3)
    logits = torch.randn(12, 48, generator=r)
    logits[0, 5:40] = -INF
    logits[1, 3:] = -INF          # fewer than k left: the others by index
    logits[2] = -INF
    logits[3, 7] = NAN
    logits[4] = NAN
    logits[5, 9] = INF
    logits[6, [4, 44]] = INF
    logits[7] = INF
    logits[8] = -3.4e38
    logits[9, 2] = 3.4e38
    logits[10, :24] = -1e30
    logits[11, 0], logits[11, 1] = INF, -INF
    for renorm in (True, False):
        check_route(g, logits, 6, score, groups=groups, top_groups=groups - groups // 3, renormalize=renorm)
    bias = torch.randn(48, generator=r)
    bias[3], bias[4], bias[5] = INF, -INF, NAN
    check_route(g, logits, 6, score, groups=groups, top_groups=groups - groups // 3, bias=bias)


def test_strided_logits(g):
    wide = torch.randn(40, 100, generator=gen(8))
    for t in (wide, wide.bfloat16()):
        ids, w = run_route(g, t[:, :33], 4)
        want = run_route(g, t[:, :33].contiguous(), 4)
        on_gpu = t.cuda()[:, :33]
        a, b = torch.empty(40, 4, dtype=I32, device="cuda"), torch.empty(40, 4, device="cuda")
        g.route(on_gpu, a, b)
        assert torch.equal(a.cpu(), want[0]) and torch.equal(b.cpu(), want[1]) and torch.equal(ids, want[0])


# ------------------------------------------------------------------ gradient

GRAD = [(1, 1, 1), (3, 8, 2), (20, 60, 6), (9, 160, 8), (5, 513, 4), (4, 1024, 32)]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["SOFTMAX", "SIGMOID"])
@pytest.mark.parametrize("T,E,k", GRAD)
@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
def test_route_backward(g, T, E, k, score, renorm, bf16):
    r = gen(T + E + k)
    logits = torch.randn(T, E, generator=r) * 2
    logits = logits.bfloat16() if bf16 else logits
    ids, _ = bh.route(logits, k, score)
    dw = torch.randn(T, k, generator=r)
    want = bh.route_grad(logits, ids, dw, score, renorm, 2.5)
    whole = torch.full((T, E + 3), NAN, dtype=logits.dtype, device="cuda")
    g.route_backward(logits.cuda(), ids.to(I32).cuda(), dw.cuda(), whole[:, :E], score=tg.Score[score],
                     renormalize=renorm, scale=2.5)
    # 64-bit arithmetic (2^-48 of the largest term where terms cancel), rounded once
    err = 2.0 ** -48 * 2.5 * dw.double().abs().sum(1, keepdim=True) + 2.0 ** -24 * 1.01 * want.abs() + 2.0 ** -149
    bh.close(whole[:, :E], want, err.expand_as(want), bf16, "dlogits")
    assert bool(whole[:, E:].isnan().all())


@pytest.mark.parametrize("score", ["SOFTMAX", "SIGMOID"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(g, score, renorm):
    """Central differences of the formula's weights with step 2^-17 in 64 bits: off by
    step^2 / 6 times a third derivative (below 30 here: products of at most four
    scores over a sum above 0.1) and 2^-52 / step of rounding."""
    T, E, k, h = 4, 10, 3, 2.0 ** -17
    r = gen(4)
    logits = torch.randn(T, E, generator=r)
    ids, _ = bh.route(logits, k, score)
    dw = torch.randn(T, k, generator=r)

    def value(l):
        s = torch.softmax(l, 1) if score == "SOFTMAX" else torch.sigmoid(l)
        w = s.gather(1, ids)
        return ((w / w.sum(1, keepdim=True) if renorm else w) * dw.double()).sum(1)
    want = torch.empty(T, E, dtype=torch.float64)
    for e in range(E):
        step = torch.zeros(T, E, dtype=torch.float64)
        step[:, e] = h
        want[:, e] = (value(logits.double() + step) - value(logits.double() - step)) / (2 * h)
    out = torch.empty(T, E, device="cuda")
    g.route_backward(logits.cuda(), ids.to(I32).cuda(), dw.cuda(), out, score=tg.Score[score], renormalize=renorm)
    err = (5 * h * h + 2.0 ** -50 / h) * dw.double().abs().sum(1, keepdim=True) + 2.0 ** -23 * want.abs()
    bh.close(out, want, err, False, "dlogits")


@pytest.mark.parametrize("score", ["SOFTMAX", "SIGMOID"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_masked_places(g, score, renorm):
    """Ids outside the experts, one named twice, rows without a score."""
    r = gen(5)
    logits = torch.randn(8, 20, generator=r)
    logits[2, 3], logits[3], logits[4, 7] = -INF, -INF, NAN
    logits[6] = -800.0
    ids = torch.randint(0, 20, (8, 4), generator=r)
    ids[0, 1], ids[1, 2], ids[5] = -1, 20, -1
    ids[7] = 6
    ids[2, 0], ids[4, 0] = 3, 7
    dw = torch.randn(8, 4, generator=r)
    want = bh.route_grad(logits, ids, dw, score, renorm, 1.0)
    assert bool(want.isfinite().all())
    out = torch.full((8, 20), NAN, device="cuda")
    g.route_backward(logits.cuda(), ids.to(I32).cuda(), dw.cuda(), out, score=tg.Score[score], renormalize=renorm)
    err = 2.0 ** -44 * dw.double().abs().sum(1, keepdim=True) + 2.0 ** -23 * want.abs()
    bh.close(out, want, err.expand_as(want), False, "dlogits")


# -------------------------------------------------------------------- places

@pytest.mark.parametrize("T,k,E,first", [
    (0, 2, 5, 0), (1, 1, 1, 0), (1, 8, 64, 0), (8, 4, 64, 0), (100, 3, 7, 2), (512, 2, 1024, 0), (1024, 4, 33, 0),
    (1025, 4, 256, 64), (3000, 8, 160, 0), (9000, 8, 1024, 100), (150000, 1, 12, 3), (40001, 6, 300, 0),
])
def test_place(g, T, k, E, first):
    print(f"[place {T}x{k} over {E} from {first}]", flush=True)
    r = gen(T + k)
    ids = torch.randint(-2, first + E + 3, (T, k), generator=r).to(I32)
    if T > 4:
        ids[1] = first            # one expert named by every place of a token
        ids[T // 2:T // 2 + 3] = first + E - 1
    want = bh.place(ids, first, E)
    for rows_too, places_too in ((True, True), (False, True), (True, False)):
        off = torch.full((E + 1,), -7, dtype=I32, device="cuda")
        rows = torch.full((T * k,), -7, dtype=I32, device="cuda") if rows_too else None
        places = torch.full((T, k), -7, dtype=I32, device="cuda") if places_too else None
        g.place(ids.cuda(), off, rows, places, first=first)
        assert torch.equal(off.cpu(), want[0])
        assert rows is None or torch.equal(rows.cpu(), want[1])
        assert places is None or torch.equal(places.cpu(), want[2])


@pytest.mark.parametrize("T", [500, 5000])
def test_place_extremes(g, T):
    """Every entry of one expert, none here, and the int32 range's ends."""
    for value in (3, -1, 2 ** 31 - 1, -2 ** 31):
        ids = torch.full((T, 2), value, dtype=I32)
        want = bh.place(ids, 0, 16)
        off, rows, places = (torch.empty(17, dtype=I32, device="cuda"), torch.empty(2 * T, dtype=I32, device="cuda"),
                             torch.empty(T, 2, dtype=I32, device="cuda"))
        g.place(ids.cuda(), off, rows, places)
        for got, w in zip((off, rows, places), want):
            assert torch.equal(got.cpu(), w)


# ------------------------------------------------------------------- combine

@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("T,k,N,z_rows", [(1, 1, 1, 1), (3, 2, 8, 5), (24, 8, 2048, 192), (50, 5, 131, 90),
                                          (7, 64, 40, 300), (200, 3, 1000, 0), (300, 1, 520, 300)])
def test_combine(g, T, k, N, z_rows, bf16):
    r = gen(T + N)
    ld = (N + 7) // 8 * 8 + 8
    z = torch.full((z_rows + 1, ld), NAN)
    z[:z_rows, :N] = torch.randn(z_rows, N, generator=r)
    z = z.bfloat16().cuda()[:z_rows, :N]
    places = torch.randint(-2, z_rows + 2, (T, k), generator=r).to(I32)
    places[0, 0] = 2 ** 31 - 1
    w = torch.randn(T, k, generator=r)
    on = (places >= 0) & (places < z_rows)
    for weights in (w, None):
        f = torch.where(on, (w if weights is not None else torch.ones(T, k)).double(), 0.0)
        rows = (z.cpu().double()[torch.where(on, places, 0).long()] if z_rows
                else torch.zeros(T, k, N, dtype=torch.float64))
        want = (f[:, :, None] * rows).sum(1)
        err = 2.0 ** -24 * (k + 1) * (f.abs()[:, :, None] * rows.abs()).sum(1)
        whole = torch.full((T + 1, ld), NAN, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
        g.combine(z, places.cuda(), None if weights is None else weights.cuda(), whole[:T, :N])
        bh.close(whole[:T, :N], want, err, bf16, "y")
        assert bool(whole[T].isnan().all()) and bool(whole[:, N:].isnan().all())


# -------------------------------------------------------------- as it is used

def layer(g, x, wr, w1, s1, w2, s2, k, first=0, options={}):
    """A router and its experts over x, the experts of w1 on this device."""
    T, K = x.shape
    E, F2 = w1.shape[0], w1.shape[1]
    e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    logits = e(T, wr.shape[0], dtype=torch.float32)
    g(x, wr.t(), logits)
    ids, weights = e(T, k, dtype=I32), e(T, k, dtype=torch.float32)
    g.route(logits, ids, weights, **options)
    off, rows, places = e(E + 1, dtype=I32), e(T * k, dtype=I32), e(T, k, dtype=I32)
    g.place(ids, off, rows, places, first=first)
    q1, t1 = e(T * k, K, dtype=bh.FP8), bh.row_scales(T * k, K, "cuda")
    g.quantize(x, q1, t1, rows=rows)
    z = e(T * k, F2)
    g.fp8_experts(q1, w1, z, t1, s1, off)
    q2, t2 = e(T * k, F2 // 2, dtype=bh.FP8), bh.row_scales(T * k, F2 // 2, "cuda")
    g.quantize(z, q2, t2, gate=tg.Gate.SILU)
    out = e(T * k, K)
    g.fp8_experts(q2, w2, out, t2, s2, off)
    y = e(T, K)
    g.combine(out, places, weights, y)
    return dict(logits=logits, ids=ids, weights=weights, y=y, q1=q1, t1=t1, z=z, q2=q2, t2=t2, out=out, places=places)


def weights_of(g, E, N, K, seed):
    w = (torch.randn(E, N, K, generator=gen(seed)) * K ** -0.5).bfloat16().cuda()
    q, s = torch.empty(E, N, K, dtype=bh.FP8, device="cuda"), torch.empty(E, bh.blocks(N), bh.blocks(K), device="cuda")
    for i in range(E):
        g.quantize(w[i], q[i], s[i], form=tg.Quant.BLOCKS)
    return q, s


@pytest.mark.parametrize("T,first,here,options", [
    (1, 0, 12, {}),
    (37, 0, 12, dict(score=tg.Score.SIGMOID, groups=4, top_groups=2, scale=2.5)),
    (300, 3, 7, dict(renormalize=False)),
])
def test_experts_of_a_layer(g, T, first, here, options):
    """Each step of the layer against 64 bits on the values it was given, and the
    captured layer, replayed on other values, against the eager one."""
    E, K, F, k = 12, 272, 144, 3
    r = gen(T)
    x = torch.randn(T, K, generator=r).bfloat16().cuda()
    wr = (torch.randn(E, K, generator=r) * 2 * K ** -0.5).bfloat16().cuda()
    w1, s1 = weights_of(g, here, 2 * F, K, 1)
    w2, s2 = weights_of(g, here, K, F, 2)
    v = layer(g, x, wr, w1, s1, w2, s2, k, first, options)
    torch.cuda.synchronize()
    want_ids, want_w = bh.route(v["logits"].cpu(), k, options.get("score", tg.Score.SOFTMAX).name,
                                groups=options.get("groups", 1), top_groups=options.get("top_groups", 1),
                                renorm=options.get("renormalize", True), scale=options.get("scale", 1.0))
    ids = v["ids"].cpu().long()
    assert torch.equal(ids, want_ids)
    # token by token over the quantized values that the products read
    y = torch.zeros(T, K, dtype=torch.float64)
    size = torch.zeros(T, K, dtype=torch.float64)
    places = v["places"].cpu()
    host = {n: v[n].cpu() for n in ("q1", "t1", "z", "q2", "t2", "out")}
    for t in range(T):
        for j in range(k):
            p, e = int(places[t, j]), int(ids[t, j]) - first
            assert (p >= 0) == (0 <= e < here)
            if p < 0:
                continue
            at = slice(p, p + 1)
            z, err = bh.product(host["q1"][at], host["t1"][at], w1[e].cpu(), s1[e].cpu())
            bh.close(host["z"][at], z, err, True, "first product")
            o, err = bh.product(host["q2"][at], host["t2"][at], w2[e].cpu(), s2[e].cpu())
            bh.close(host["out"][at], o, err, True, "second product")
            y[t] += want_w[t, j] * host["out"][p].double()
            size[t] += (want_w[t, j] * host["out"][p].double()).abs()
    bh.close(v["y"], y, 2.0 ** -21 * size, True, "y")

    graph, x2 = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph):
        captured = layer(g, x2, wr, w1, s1, w2, s2, k, first, options)
    for n in range(3):
        x2.copy_(x.roll(n + 1, 0) * (1 + n))
        eager = layer(g, x2, wr, w1, s1, w2, s2, k, first, options)
        captured["y"].fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured["y"], eager["y"]) and torch.equal(captured["ids"], eager["ids"])


def test_two_streams(g):
    """The same calls at once on two streams, each with its own workspace."""
    r = gen(77)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ids = [torch.randint(0, 64, (6000, 4), generator=r).to(I32).cuda() for _ in streams]
    outs = [(torch.empty(65, dtype=I32, device="cuda"), torch.empty(24000, dtype=I32, device="cuda"),
             torch.empty(6000, 4, dtype=I32, device="cuda")) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, i, o in zip(streams, ids, outs):
            g.place(i, *o, stream=s)
    torch.cuda.synchronize()
    for i, o in zip(ids, outs):
        for got, want in zip(o, bh.place(i.cpu(), 0, 64)):
            assert torch.equal(got.cpu(), want)


def test_binding_refusals(g):
    e = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    l, ids, w = e(10, 16), e(10, 2, dtype=I32), e(10, 2)
    for args, kw, error in (((l.half(), ids, w), {}, TypeError), ((l[:9], ids, w), {}, ValueError),
                            ((l.t(), ids, w), {}, ValueError), ((l, ids.long(), w), {}, TypeError),
                            ((l, ids, w[:, :1]), {}, ValueError), ((l, ids, w.t().contiguous().t()), {}, ValueError),
                            ((l, ids, w), dict(bias=e(15)), ValueError), ((l.cpu(), ids, w), {}, ValueError),
                            ((l, ids, w), dict(groups=3), tg.TileGemmError),
                            ((l, ids, w), dict(scale=NAN), tg.TileGemmError)):
        with pytest.raises(error):
            g.route(*args, **kw)
    for args, error in (((l, ids, w, l.bfloat16()), TypeError), ((l, ids, w, l), tg.TileGemmError),
                        ((l, ids, w, e(10, 15)), ValueError), ((l, ids, ids, e(10, 16)), TypeError)):
        with pytest.raises(error):
            g.route_backward(*args)
    off = e(17, dtype=I32)
    for args, kw, error in (((ids, off[:1]), {}, ValueError), ((ids, e(17)), {}, TypeError),
                            ((ids, off, e(19, dtype=I32)), {}, ValueError),
                            ((ids, off, None, e(2, 10, dtype=I32)), {}, ValueError),
                            ((ids, off), dict(first=-1), tg.TileGemmError)):
        with pytest.raises(error):
            g.place(*args, **kw)
    z, y = e(20, 64, dtype=torch.bfloat16), e(10, 64)
    for args, error in (((z.float(), ids, w, y), TypeError), ((z, ids, w, y[:9]), ValueError),
                        ((z, ids, w, y.half()), TypeError), ((z, ids, w[:9], y), ValueError),
                        ((z.t(), ids, w, e(10, 20)), ValueError), ((z[:, :60], ids, w, y[:, :62]), ValueError)):
        with pytest.raises(error):
            g.combine(*args)
