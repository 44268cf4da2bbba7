"""Operands whose rows lie far apart: views into tensors of nearly 4 GiB, such
as the last token of every sequence of a batch. Results have to be those of the
same call on a contiguous copy, bit for bit: a launch plan does not depend on
the row strides of x."""

import pytest
import torch

import tile_partitioned_dense_amd as tg
from test_gpu_glu import DEV

pytestmark = pytest.mark.gpu
SPAN = 2 ** 32  # bytes an operand may span (exclusive)


@pytest.fixture(scope="module")
def g():
    with tg.TileGemm(0) as handle:
        yield handle


def far(t, pitch):
    """A view with the values of t, its rows `pitch` elements apart and NaN
    everywhere between them."""
    rows, cols = t.shape
    assert pitch % 8 == 0 and ((rows - 1) * pitch + cols) * 2 < SPAN
    store = torch.full(((rows - 1) * pitch + (cols + 7) // 8 * 8,), float("nan"), dtype=torch.bfloat16, device=DEV)
    view = store.as_strided((rows, cols), (pitch, 1))
    view.copy_(t)
    return view


def widest(rows, cols):
    """The largest pitch that an operand of this many rows may have."""
    return ((SPAN // 2 - cols - 8) // (rows - 1)) // 8 * 8


def values(T, K, N, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, K, generator=gen, device=DEV).bfloat16()
    w = (torch.randn(N, K, generator=gen, device=DEV) * K ** -0.5).bfloat16()
    return gen, x, w


def head(g, x, w, t, d):
    """Loss, log-sum-exp and both gradients."""
    T, K = x.shape
    o = [torch.full((T,), float("nan"), device=DEV) for _ in range(2)]
    o += [torch.full((r, (K + 7) // 8 * 8), float("nan"), dtype=torch.bfloat16, device=DEV)[:, :K]
          for r in (T, w.shape[0])]
    g.xent(x, w.t(), t, o[0], o[1])
    g.xent_backward(x, w.t(), t, o[1], d, dA=o[2], dB=o[3].t())
    return o


def block(g, x, w, dh, gate):
    """Forward result and all three gradients."""
    T, K = x.shape
    F2 = w.shape[0]
    o = [torch.full(s, float("nan"), dtype=torch.bfloat16, device=DEV) for s in ((T, F2 // 2), (T, K), (F2, K))]
    o.append(torch.full((F2,), float("nan"), device=DEV))
    g.glu(x, w.t(), o[0], gate=gate)
    g.glu_backward(x, w.t(), dh, dA=o[1], dB=o[2].t(), gate=gate, dbias=o[3])
    return o


def same(got, want):
    for i, (a, b) in enumerate(zip(got, want)):
        assert bool(b.isfinite().all()), i
        assert torch.equal(a, b), f"output {i}: {int((a != b).sum())} of {b.numel()} differ"


# Rows of x past 2 GiB from the start of a tile's panel, with a contraction that
# ends inside a tile's step: (48, ...) in the weight gradient, which contracts
# the 48 tokens on 256 x 160 tiles, (200, ...) in the logits or pre-activations,
# which contract the width on 128-row and on 256-row tiles.
@pytest.mark.parametrize("T,K,V,pitch", [(48, 136, 40000, 2 ** 25), (200, 72, 20000, 10 * 2 ** 20),
                                         (200, 520, 50257, 2 ** 23), (200, 2056, 9000, 10 * 2 ** 20)])
def test_far_rows_of_x_head(g, T, K, V, pitch):
    gen, x, w = values(T, K, V, 1)
    t = torch.randint(0, V, (T,), generator=gen, device=DEV)
    d = torch.rand(T, generator=gen, device=DEV)
    same(head(g, far(x, pitch), w, t, d), head(g, x, w, t, d))


@pytest.mark.parametrize("T,K,F,pitch", [(48, 136, 20000, 2 ** 25), (200, 136, 10000, 10 * 2 ** 20),
                                         (200, 136, 25136, 2 ** 23), (200, 520, 20000, 2 ** 23)])
def test_far_rows_of_x_block(g, T, K, F, pitch):
    gen, x, w = values(T, K, 2 * F, 2)
    dh = torch.randn(T, F, generator=gen, device=DEV).bfloat16()
    for gate in (tg.Gate.SILU, tg.Gate.GELU_TANH):
        same(block(g, far(x, pitch), w, dh, gate), block(g, x, w, dh, gate))


# The up half of a weight of nearly 4 GiB begins 2 GiB behind the gate half.
@pytest.mark.parametrize("T,K,F", [(2000, 72, 1024), (8000, 72, 1024)])
def test_far_up_half(g, T, K, F):
    gen, x, w = values(T, K, 2 * F, 3)
    dh = torch.randn(T, F, generator=gen, device=DEV).bfloat16()
    same(block(g, x, far(w, 2 ** 20), dh, tg.Gate.GELU), block(g, x, w, dh, tg.Gate.GELU))


# Rows of a row-major weight past 2 GiB, on 128-row tiles (steps of 32 rows) and
# on 256-row tiles (steps of 64).
@pytest.mark.parametrize("T,K,F,pitch", [(200, 24, 1000, 2 ** 26), (4096, 56, 2048, 2 ** 25)])
def test_far_rows_of_a_row_major_weight(g, T, K, F, pitch):
    _, x, w = values(T, K, 2 * F, 4)
    wr = w.t().contiguous()
    for gate in (tg.Gate.GELU, tg.Gate.RELU):
        h = [torch.full((T, F), float("nan"), device=DEV) for _ in range(2)]
        g.glu(x, far(wr, pitch), h[0], gate=gate)
        g.glu(x, wr, h[1], gate=gate)
        same(h[:1], h[1:])


# The step of a contraction that ends inside it names rows past the last one,
# whose 32-bit offsets wrap to the NaN between the first rows where rows lie as
# far apart as they may: the contractions over tokens (a weight gradient) and
# over a row-major weight's rows. (48 tokens span so near to 4 GiB that their
# step goes through registers, 63 take 128-row tiles.)
@pytest.mark.parametrize("T,K,V", [(36, 136, 40000), (48, 136, 40000), (63, 264, 40000)])
def test_farthest_tokens(g, T, K, V):
    gen, x, w = values(T, K, V, 6)
    t = torch.randint(0, V, (T,), generator=gen, device=DEV)
    d = torch.rand(T, generator=gen, device=DEV)
    same(head(g, far(x, widest(T, K)), w, t, d), head(g, x, w, t, d))
    gen, x, w = values(T, K, V, 7)
    dh = torch.randn(T, V // 2, generator=gen, device=DEV).bfloat16()
    same(block(g, far(x, widest(T, K)), w, dh, tg.Gate.SILU), block(g, x, w, dh, tg.Gate.SILU))


@pytest.mark.parametrize("T,K,F", [(200, 24, 1000), (4096, 56, 2048), (4096, 40, 2048), (300, 8, 512)])
def test_farthest_rows_of_a_row_major_weight(g, T, K, F):
    _, x, w = values(T, K, 2 * F, 8)
    wr = w.t().contiguous()
    h = [torch.full((T, F), float("nan"), device=DEV) for _ in range(2)]
    g.glu(x, far(wr, widest(K, 2 * F)), h[0], gate=tg.Gate.GELU)
    g.glu(x, wr, h[1], gate=tg.Gate.GELU)
    same(h[:1], h[1:])


# Weights of a vocabulary with the widest rows allowed (8 MiB apart).
@pytest.mark.parametrize("T,K,V", [(200, 72, 500), (2000, 328, 500)])
def test_far_rows_of_a_vocabulary(g, T, K, V):
    gen, x, w = values(T, K, V, 5)
    t = torch.randint(0, V, (T,), generator=gen, device=DEV)
    d = torch.rand(T, generator=gen, device=DEV)
    got = head(g, x, far(w, 2 ** 22 - 8), t, d)
    want = head(g, x, w, t, d)
    # the pieces of the vocabulary follow its stride, and with them the sums
    g.xent_backward(x, w.t(), t, want[1], d, dA=want[2], dB=want[3].t(), piece=256)
    same(got, want)
