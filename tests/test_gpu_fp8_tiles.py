"""Every compiled tile of the E4M3 products, one weight and rows sorted by
expert, on operands as they come: general scales, rows further apart than they
are long, K that ends inside a block, columns that fill no chunk, a bias and each
activation, NaN scales and codes, and the same call again. The shapes are
taken from the plan, so that a changed plan changes them too."""

import pytest
import torch

import block_helpers as bh
import tile_partitioned_dense_amd as tg

NAN = float("nan")
N_CONFIGS, N_TILE = 15, 4  # compiled tiles; those of the kernel for many rows
ROWS = (7, 20, 45, 70, 150, 300, 500, 700, 1030, 2050, 4100)
COLS = (9, 42, 131, 265, 530, 1031, 2057, 4105, 8201, 28691)
DEPTH = (144, 272, 400, 528, 784, 1040, 1552, 2064, 4112)
DTYPES = (torch.bfloat16, torch.float32)
EXPERTS = 6
_shapes = {}


def plan(M, N, K, experts, dtype, cus=256):
    return tg.tile_gemm_plan_fp8(M, N, K, experts, tg.Dtype(int(dtype is torch.bfloat16)), cus)


def shapes(experts):
    """{(configuration, dtype): the smallest shape planned to it that has more than one stage}."""
    if experts not in _shapes:
        found = _shapes[experts] = {}
        for dtype in DTYPES:
            for M in ROWS:
                for N in COLS:
                    for K in DEPTH:
                        p = plan(M, N, K, experts, dtype)
                        old = found.get((p.config, dtype))
                        if K > p.bk and (old is None or M * N * K < old[0] * old[1] * old[2]):
                            found[p.config, dtype] = (M, N, K)
    return _shapes[experts]


@pytest.mark.parametrize("experts", [0, EXPERTS])
def test_shapes_reach_every_tile(experts):
    """(an fp32 result has no 256 x 256 tile)"""
    want = {(c, t) for c in range(N_CONFIGS) for t in DTYPES} - {(0, torch.float32)}
    assert set(shapes(experts)) == want
    for (c, t), (M, N, K) in shapes(experts).items():
        assert N % 4 and K % 128


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    with tg.TileGemm(0) as gg:
        yield gg


CASES = [(c, t, e) for c in range(N_CONFIGS) for t in DTYPES for e in (0, EXPERTS) if (c, t) != (0, torch.float32)]


def case_id(c):
    return f"{c[0]}-{'bf16' if c[1] is torch.bfloat16 else 'fp32'}-{c[2]}"


@pytest.fixture(params=CASES, ids=case_id)
def case(request, g):
    """Configuration, type, experts, and operands on the GPU, padded with NaN on every side."""
    config, dtype, experts = request.param
    M, N, K = shapes(experts)[config, dtype]
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert plan(M, N, K, experts, dtype, cus).config == config
    print(f"[fp8 {config}: {M}x{N}x{K} {dtype} {experts}]", flush=True)
    return Case(config, dtype, experts, M, N, K)


class Case:
    def __init__(self, config, dtype, experts, M, N, K):
        self.config, self.dtype, self.experts, self.M, self.N, self.K = config, dtype, experts, M, N, K
        r = torch.Generator(device="cuda").manual_seed(1000 * M + 10 * N + K + config)
        E, kb, nb = max(experts, 1), bh.blocks(K), bh.blocks(N)

        def codes(*shape):
            return (torch.randn(*shape, generator=r, device="cuda") * 100).clamp(-448, 448).to(bh.FP8)
        a = torch.full((M + 9, K + 16), 0x7f, dtype=torch.uint8, device="cuda").view(bh.FP8)
        b = torch.full((E, N + 5, K + 48), 0x7f, dtype=torch.uint8, device="cuda").view(bh.FP8)
        sa = torch.full((kb, M + 7), NAN, device="cuda")
        sb = torch.full((E, nb, kb + 3), NAN, device="cuda")
        a[:M, :K], b[:, :N, :K] = codes(M, K), codes(E, N, K)
        sa[:, :M] = torch.rand(kb, M, generator=r, device="cuda") * 0.02 + 0.001
        sb[:, :, :kb] = torch.rand(E, nb, kb, generator=r, device="cuda") * 0.001 + 0.0001
        self.a, self.b, self.sa, self.sb = a[:M, :K], b[:, :N, :K], sa.t()[:M], sb[:, :, :kb]
        self.bias = torch.randn(N, generator=r, device="cuda")
        cuts = sorted([0, M // 50, M // 50, M - M // 5 - M // 50, M - M // 5 - min(M // 50, 1), M - M // 5, M])
        self.cuts = cuts if experts else [0, M]
        self.offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")

    def run(self, g, **epilogue):
        """The whole output, with NaN around the result, and the result."""
        whole = torch.full((self.M + 2, (self.N + 7) // 8 * 8 + 8), NAN, dtype=self.dtype, device="cuda")
        c = whole[1:self.M + 1, :self.N]
        if self.experts:
            g.fp8_experts(self.a, self.b, c, self.sa, self.sb, self.offsets)
        else:
            g.fp8(self.a, self.b[0], c, self.sa, self.sb[0], **epilogue)
        keep = torch.ones_like(whole, dtype=torch.bool)
        keep[1:self.M + 1, :self.N] = False
        assert bool(whole[keep].isnan().all())
        return c

    def reference(self):
        """The products in 64 bits and their bound (block_helpers; a run's largest
        product is at most the product of its largest values)."""
        def wide(q, s, high):
            s = s.double().repeat_interleave(128, -1)[..., :self.K]
            return q.double() * (s.repeat_interleave(high, -2)[..., :q.shape[-2], :] if high > 1 else s)

        def tops(v):
            return torch.nn.functional.pad(v.abs(), (0, -self.K % 8)).view(v.shape[0], -1, 8).amax(2)
        x, want, err = wide(self.a, self.sa, 1), [], []
        for e, (lo, hi) in enumerate(zip(self.cuts, self.cuts[1:])):
            if hi == lo:
                continue
            y, z = wide(self.b[e], self.sb[e], 128), x[lo:hi]
            want.append(z @ y.T)
            err.append(bh.TAU * (z.abs() @ y.abs().T))
            if self.dtype is torch.bfloat16:
                err[-1] += 7 * 2.0 ** -13 * (tops(z) @ tops(y).T)
        return torch.cat(want), torch.cat(err)


@pytest.mark.gpu
def test_general_operands(g, case):
    """Against 64 bits, and bit for bit the same again."""
    want, err = case.reference()
    c = case.run(g)
    bh.close(c, want.cpu(), err.cpu(), case.dtype is torch.bfloat16, "c")
    for _ in range(2):
        assert torch.equal(case.run(g), c)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["NONE", "RELU", "SIGMOID", "TANH", "SILU"])
@pytest.mark.parametrize("case", [c for c in CASES if not c[2]], indirect=True, ids=case_id)
def test_bias_and_activation(g, case, act):
    """(of one weight; the experts' product has neither)"""
    want, err = case.reference()
    assert float(want.abs().amax()) > 1.0  # (both ends of the activation)
    want = want + case.bias.double()
    err = err + 2.0 ** -23 * want.abs()
    y = bh.ACTS[act](want)
    if act != "NONE":
        err = bh.LIP[act] * err + bh.EVAL * y.abs() + 2.0 ** -22
    c = case.run(g, bias=case.bias, act=tg.Act[act])
    bh.close(c, y.cpu(), err.cpu(), case.dtype is torch.bfloat16, act)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "fp32"])
def test_bias_without_products(g, dtype):
    """K = 0 on the tiles for many rows: act(bias), of a width that fills no chunk."""
    M, N = 6100, 15398
    assert plan(M, N, 0, 0, dtype).config < N_TILE
    bias, e = torch.randn(N, device="cuda"), torch.empty
    c = e(M, (N + 7) // 8 * 8, dtype=dtype, device="cuda")[:, :N]
    for act, f in ((tg.Act.NONE, lambda v: v), (tg.Act.RELU, lambda v: v.clamp(min=0))):
        g.fp8(e(M, 0, dtype=bh.FP8, device="cuda"), e(N, 0, dtype=bh.FP8, device="cuda"), c.fill_(NAN),
              e(M, 0, device="cuda"), e(bh.blocks(N), 0, device="cuda"), bias=bias, act=act)
        assert torch.equal(c, f(bias).to(dtype).expand(M, N))


@pytest.mark.gpu
def test_bad_scales_and_codes(g, case):
    """A NaN scale or code reaches its row or its 128 columns of one weight, an
    infinite scale its row, and no other value."""
    M, N = case.M, case.N
    want, err = case.reference()
    bad = torch.zeros(M, N, dtype=torch.bool)
    case.sa[3, 1] = NAN
    case.a.view(torch.uint8)[5, case.K - 1] = 0x7f
    bad[3] = bad[5] = True
    case.sa[M - 1, 0] = float("inf")
    lo, hi = case.cuts[-2:]
    if N > 128 and hi > lo:
        case.sb[len(case.cuts) - 2, 1, 1] = NAN  # of the last expert (or the one weight)
        bad[lo:hi, 128:256] = True
    c = case.run(g).cpu()
    assert bool(c[bad].isnan().all())
    assert not bool(c[M - 1].isfinite().any())
    bad[M - 1] = True
    bh.close(c.float().masked_fill(bad, 0), want.cpu().masked_fill(bad, 0), err.cpu(),
             case.dtype is torch.bfloat16, "the others")
