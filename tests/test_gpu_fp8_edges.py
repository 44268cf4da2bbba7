"""E4M3 products and the quantization at the ends of their ranges: bad values
behind an activation, gates far out on their tails."""

import pytest
import torch

import block_helpers as bh
import tile_partitioned_dense_amd as tg

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    with tg.TileGemm(0) as gg:
        yield gg


def gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K,many", [(20, 300, 272, False), (2050, 4105, 144, True)])
@pytest.mark.parametrize("act", ["NONE", "RELU", "SIGMOID", "TANH", "SILU"])
def test_nan_passes_every_activation(g, M, N, K, many, dtype, act):
    """A row with a NaN scale, one with a NaN code, one whose block held an
    infinity when it was quantized, and the columns of a NaN scale are NaN
    behind any activation, on both kernels; the others are not."""
    p = tg.tile_gemm_plan_fp8(M, N, K, 0, tg.Dtype(int(dtype is torch.bfloat16)))
    assert (p.config < 4) == many
    print(f"[fp8 nan {M}x{N}x{K} {dtype} {act}]", flush=True)
    x = torch.randn(M, K, generator=gen(M)).bfloat16()
    x[4, K - 2] = INF
    q, s = torch.empty(M, K, dtype=torch.uint8, device="cuda"), bh.row_scales(M, K, "cuda")
    g.quantize(x.cuda(), q, s)
    b, sb = bh.codes(gen(N), N, K), torch.full((bh.blocks(N), bh.blocks(K)), 1e-3)
    s[3, 1], sb[1, 0] = NAN, NAN
    q[M - 1, 0] = 0xff
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[3] = bad[4] = bad[M - 1] = True
    bad[:, 128:256] = True
    for bias in (None, torch.randn(N, generator=gen(1)).cuda()):
        c = torch.zeros(M, (N + 7) // 8 * 8, dtype=dtype, device="cuda")[:, :N]
        g.fp8(q, b.cuda(), c, s, sb.cuda(), bias=bias, act=tg.Act[act])
        assert torch.equal(c.isnan().cpu(), bad)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(20, 300, 272), (2050, 4105, 144)])
def test_infinite_scale_and_relu(g, M, N, K, dtype):
    """relu of a row with an infinite scale: infinity, or 0 for minus infinity."""
    a, b = bh.codes(gen(M), M, K), torch.full((N, K), 1.0).to(bh.FP8)
    s = bh.row_scales(M, K, "cuda")
    s.fill_(1.0)
    s[3, 0] = s[7, 0] = INF
    a[3, :128], a[7, :128] = 2.0, -2.0
    c = torch.zeros(M, (N + 7) // 8 * 8, dtype=dtype, device="cuda")[:, :N]
    g.fp8(a.cuda(), b.cuda(), c, s, torch.ones(bh.blocks(N), bh.blocks(K), device="cuda"), act=tg.Act.RELU)
    assert bool((c[3] == INF).all()) and bool((c[7] == 0).all())


# (gate, the largest relative error of its value in fp32): the exponential's
# argument is off by a few of its roundings, 2^-24 of it each -- one for silu and
# gelu (z^2 / 2 of a bf16 value is exact), six for gelu_tanh -- and by half a step
# of the hardware's exponential, EVAL at most together with the rest
TAILS = [("SILU", lambda z: bh.EVAL + 2.0 ** -24 * z.abs()),
         ("GELU", lambda z: bh.EVAL + 2.0 ** -24 * z * z / 2),
         ("GELU_TANH", lambda z: bh.EVAL + 6 * 2.0 ** -24 * 1.6 * (z.abs() + 0.045 * z.abs() ** 3)),
         ("SIGMOID", lambda z: bh.EVAL + 2.0 ** -24 * z.abs())]


def gate64(z, gate):
    if gate == "GELU":
        return z * 0.5 * torch.special.erfc(-z * 0.5 ** 0.5)
    if gate == "GELU_TANH":
        y = 2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)
        return z * torch.sigmoid(y)
    return torch.sigmoid(z) * (z if gate == "SILU" else 1.0)


@pytest.mark.parametrize("gate,bound", TAILS, ids=[t[0] for t in TAILS])
def test_scales_of_gates_on_their_tails(g, gate, bound):
    """A block whose gates all lie at one value, from 9 down to -9: its scale is
    that value's, to the precision of fp32, however small it is."""
    z = torch.arange(-9.0, 9.0, 1 / 16).bfloat16()
    z = z[(z.double() * (7.0 if gate == "GELU_TANH" else 1.0)).abs() <= 45]  # (2^-100 and less counts as that)
    M, K = len(z), 128
    x = torch.cat([z[:, None].expand(M, K), torch.ones(M, K)], 1).bfloat16().cuda()
    q, s = torch.empty(M, K, dtype=bh.FP8, device="cuda"), bh.row_scales(M, K, "cuda")
    g.quantize(x, q, s, gate=tg.Gate[gate])
    want = gate64(z.double(), gate).abs().clamp(min=2.0 ** -100) / 448
    off = (s[:, 0].cpu().double() - want).abs() / want
    # (two more roundings: of the value and of its division by 448)
    over = off > bound(z.double()) + 2.0 ** -23
    assert not bool(over.any()), [(float(z[i]), float(off[i])) for i in over.nonzero()[:8, 0]]


# -------------------------------------------------------------- the longest axes

def small(seed, *shape):
    """Codes of -1, 0 and 1: sums of 2^22 products are exact in fp32."""
    r = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=r, device="cuda").float().to(bh.FP8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [((1 << 22) - 1, 5, 16), (3, (1 << 22) - 13, 16), (200, (1 << 18) - 3, 16),
                                   (5, 40, (1 << 22) - 16), (300, 520, (1 << 20) - 112)])
def test_longest_axes(g, M, N, K, dtype):
    print(f"[fp8 longest {M}x{N}x{K} {dtype}]", flush=True)
    a, b = small(1, M, K), small(2, N, K)
    sa, sb = torch.ones(bh.blocks(K), M, device="cuda").t(), torch.ones(bh.blocks(N), bh.blocks(K), device="cuda")
    sa[M - 1], sb[bh.blocks(N) - 1] = 2.0, 4.0
    want = a.float() @ b.float().T.contiguous()
    want[M - 1] *= 2
    want[:, (N - 1) // 128 * 128:] *= 4
    c = torch.full((M, (N + 7) // 8 * 8), NAN, dtype=dtype, device="cuda")
    g.fp8(a, b, c[:, :N], sa, sb)
    assert torch.equal(c[:, :N], want.to(dtype)) and bool(c[:, N:].isnan().all())
    c.fill_(NAN)
    cut = M // 3
    off = torch.tensor([0, cut, cut, M], dtype=torch.int32, device="cuda")
    g.fp8_experts(a, b.float().mul(-1).to(bh.FP8).expand(3, N, K).contiguous(), c[:, :N], sa,
                  sb.expand(3, *sb.shape).contiguous(), off)
    assert torch.equal(c[:, :N], (-want).to(dtype)) and bool(c[:, N:].isnan().all())


def test_quantize_longest_rows(g):
    K = (1 << 22) - 16
    x = (torch.arange(K, device="cuda") // 128 % 61 + 1).bfloat16().view(1, K).repeat(2, 1)
    q, s = torch.zeros(2, K, dtype=torch.uint8, device="cuda"), bh.row_scales(2, K, "cuda")
    g.quantize(x, q, s)
    assert bool((q == 0x7e).all())
    assert torch.equal(s, (x[:, ::128].double() / 448).float())
