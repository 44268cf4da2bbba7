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


def test_most_tokens(g):
    """T at its largest: ids and weights of 2^25 - 1 tokens, their gradient."""
    T, E, k = (1 << 25) - 1, 4, 1
    logits = torch.zeros(T, E, device="cuda")
    best = torch.arange(T, device="cuda") % E
    logits.scatter_(1, best[:, None], 1.0)
    ids, w = torch.full((T, k), -9, dtype=I32, device="cuda"), torch.zeros(T, k, device="cuda")
    g.route(logits, ids, w, renormalize=False)
    assert torch.equal(ids[:, 0].long(), best)
    p = float(torch.softmax(torch.tensor([1.0, 0, 0, 0], dtype=torch.float64), 0)[0])
    assert bool(((w.double() - p).abs() <= 2.0 ** -24).all())
    d = torch.full_like(logits, float("nan"))
    g.route_backward(logits, ids, torch.ones_like(w), d, renormalize=False)
    assert bool(((d.gather(1, best[:, None]).double() - p * (1 - p)).abs() <= 2.0 ** -24).all())
    assert bool((d.sum(1).abs() <= 2.0 ** -22).all())


def test_most_entries_placed(g):
    """n at its largest, 2^31 - 1 entries of 7 experts, two of them elsewhere."""
    n, E, first = (1 << 31) - 1, 5, 1
    ids = (torch.arange(n, device="cuda", dtype=I32) % 7).view(n, 1)
    off, places = torch.empty(E + 1, dtype=I32, device="cuda"), torch.empty(n, 1, dtype=I32, device="cuda")
    rows = torch.empty(n, dtype=I32, device="cuda")
    g.place(ids, off, rows, places, first=first)
    counts = [(n - e + 6) // 7 for e in range(7)]
    want = [0]
    for e in range(first, first + E):
        want.append(want[-1] + counts[e])
    assert off.tolist() == want
    step = 1 << 27
    start = torch.tensor([0] + want[:E] + [0], device="cuda")
    for lo in range(0, n, step):
        at = torch.arange(lo, min(lo + step, n), device="cuda")
        e = at % 7
        here = (e >= first) & (e < first + E)
        p = torch.where(here, start[e] + at // 7, -1)
        assert torch.equal(places[at, 0].long(), p)
        assert torch.equal(rows[p[here]].long(), at[here])
        behind = at[at >= want[-1]]
        assert bool((rows[behind] == -1).all())


def test_most_sums(g):
    """The most tokens, and the most values of one call that they allow."""
    T, N, k, R = (1 << 22) - 1, 1023 * 8, 2, 5
    z = (torch.arange(R * N, device="cuda") % 251 - 125).bfloat16().view(R, N)
    places = torch.stack([torch.arange(T, device="cuda") % R, torch.full((T,), -1, device="cuda")], 1).to(I32)
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    g.combine(z, places, None, y)
    for r in range(R):
        mine = y[r::R]
        for lo in range(0, len(mine), 1 << 18):
            assert bool((mine[lo:lo + (1 << 18)] == z[r]).all())
