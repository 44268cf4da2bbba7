"""The E4M3 products with block scales, for one weight and for rows sorted by
expert, and the quantization, against plain 64-bit references."""

import ctypes

import pytest
import torch

import block_helpers as bh
import tile_partitioned_dense_amd as tg

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    with tg.TileGemm(0) as gg:
        yield gg


def gen(seed):
    return torch.Generator().manual_seed(seed)


def padded(t, pad, fill):
    """t on the GPU with `pad` values behind each row."""
    rows, cols = t.shape
    out = torch.full((rows, cols + pad), fill, dtype=torch.float32).to(t.dtype)
    if out.dtype == bh.FP8:
        out = torch.full((rows, cols + pad), 0x7f, dtype=torch.uint8).view(bh.FP8)  # NaN codes
    out[:, :cols] = t
    return out.cuda()[:, :cols]


def to_row_scales(s, pad=0):
    out = bh.row_scales(s.shape[0], s.shape[1] * 128, "cuda", pad)
    out.copy_(s)
    return out


def out_like(M, N, dtype, pad=8, fill=NAN):
    ld = (N + 7) // 8 * 8 + pad
    whole = torch.full((M + 2, ld), fill, dtype=dtype, device="cuda")
    return whole, whole[1:M + 1, :N]


def untouched(whole, c):
    """Everything of `whole` outside c is still NaN."""
    keep = torch.ones_like(whole, dtype=torch.bool)
    keep[1:c.shape[0] + 1, :c.shape[1]] = False
    return bool(whole[keep].isnan().all())


def operands(M, N, K, seed=0, lead=()):
    r = gen(1000 * M + 10 * N + K + seed)
    a, b = bh.codes(r, M, K), bh.codes(r, *lead, N, K)
    sa = torch.rand(M, bh.blocks(K), generator=r) * 0.02 + 0.001
    sb = torch.rand(*lead, bh.blocks(N), bh.blocks(K), generator=r) * 0.02 + 0.001
    return a, sa, b, sb


SHAPES = [
    (1, 1, 16), (1, 64, 128), (3, 130, 144), (16, 200, 528), (17, 129, 2064), (32, 1000, 1024), (33, 260, 4112),
    (64, 128, 256), (65, 300, 400), (129, 500, 2064), (200, 257, 128), (256, 256, 16), (300, 1030, 1296),
    (513, 770, 640),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(g, M, N, K, dtype):
    print(f"[fp8 {M}x{N}x{K} {dtype}]", flush=True)
    a, sa, b, sb = operands(M, N, K)
    want, err = bh.product(a, sa, b, sb, fp32=dtype == torch.float32)
    whole, c = out_like(M, N, dtype)
    # NaN codes and scales behind every row: nothing past K or M reaches a result
    g.fp8(padded(a, 16, NAN), padded(b, 48, NAN), c, to_row_scales(sa, 5), padded(sb, 3, NAN))
    bh.close(c, want, err, dtype == torch.bfloat16, "c")
    assert untouched(whole, c)


N_CONFIGS = 15  # compiled tiles


def smallest_shapes(experts):
    """{(configuration, dtype): the smallest shape (M, N, K) that is planned to it}, odd ones."""
    found = {}
    for dtype in (torch.bfloat16, torch.float32):
        for M in (1, 7, 20, 45, 70, 150, 300, 500, 700, 1030, 2050, 4100):
            for N in (9, 40, 130, 264, 530, 1030, 2056, 4104, 8200, 28690):
                for K in (16, 144, 272, 528, 1040, 2064, 4112, 8208):
                    c = tg.tile_gemm_plan_fp8(M, N, K, experts, tg.Dtype(int(dtype is torch.bfloat16))).config
                    old = found.get((c, dtype))
                    if old is None or M * N * K < old[0] * old[1] * old[2]:
                        found[c, dtype] = (M, N, K)
    return found


def integers(seed, *shape):
    return torch.randint(-3, 4, shape, generator=gen(seed)).float().to(bh.FP8)


def powers(seed, *shape):
    return (2.0 ** torch.randint(-2, 3, shape, generator=gen(seed))).float()


def wide(q, s, high):
    """As bh.widen, in fp32 on the GPU: exact here."""
    return (q.cuda().float() * s.cuda().repeat_interleave(128, -1)[..., :q.shape[-1]].repeat_interleave(
        high, -2)[..., :q.shape[-2], :])


@pytest.mark.parametrize("config", range(N_CONFIGS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_every_tile(g, config, dtype):
    """Each compiled tile on the smallest shape planned to it: integers and
    scales that are powers of two, whose sums are exact in any order."""
    shape = smallest_shapes(0).get((config, dtype))
    if shape is None:
        assert (config, dtype) == (0, torch.float32)
        return
    M, N, K = shape
    for K in (K, K + 112):  # and one that ends inside a block
        print(f"[fp8 {config}: {M}x{N}x{K} {dtype}]", flush=True)
        a, b, sa, sb = (integers(K, M, K), integers(K + 1, N, K), powers(K, M, bh.blocks(K)),
                        powers(K + 1, bh.blocks(N), bh.blocks(K)))
        want = wide(a, sa, 1).double() @ wide(b, sb, 128).double().T
        whole, c = out_like(M, N, dtype)
        g.fp8(a.cuda(), b.cuda(), c, to_row_scales(sa), sb.cuda())
        assert torch.equal(c.double(), want.to(dtype).double())
        assert untouched(whole, c)


@pytest.mark.parametrize("K", [0, 16, 128, 272, 528, 800, 1056])
@pytest.mark.parametrize("M", [5, 20])
def test_rounds_of_few_rows(g, M, K):
    """Three rounds of tiles and more, of one stage, of a few, of none: stages
    of the tiles behind are loaded while a tile is in use."""
    N = 98354
    print(f"[fp8 rounds {M}x{N}x{K}]", flush=True)
    a, b, sa, sb = (integers(1, M, K), integers(2, N, K), powers(3, M, bh.blocks(K)),
                    powers(4, bh.blocks(N), bh.blocks(K)))
    want = wide(a, sa, 1).double() @ wide(b, sb, 128).double().T if K else torch.zeros(M, N, device="cuda").double()
    for dtype in (torch.bfloat16, torch.float32):
        whole, c = out_like(M, N, dtype)
        g.fp8(a.cuda(), b.cuda(), c, to_row_scales(sa), sb.cuda())
        assert torch.equal(c.double(), want.to(dtype).double())
        assert untouched(whole, c)


@pytest.mark.parametrize("K", [0, 16, 144, 272, 400])
@pytest.mark.parametrize("M,N", [(2300, 15400), (1100, 28690), (6100, 4104), (1100, 15400), (6100, 8200)])
def test_rounds_of_large_tiles(g, M, N, K):
    """Two rounds of the large tiles and more, of one stage to four: the last
    stages of a tile load the first of the next. Once with one weight, once with
    experts of which one has a row, one none, and none ends with a tile."""
    print(f"[fp8 rounds of tiles {M}x{N}x{K}]", flush=True)
    off = [0, M // 3, M // 3, M // 3 + 1, M - M // 7, M - 2]
    a, b, sa, sb = (integers(1, M, K), integers(2, 5, N, K), powers(3, M, bh.blocks(K)),
                    powers(4, 5, bh.blocks(N), bh.blocks(K)))
    ad, sad, bd, sbd = a.cuda(), to_row_scales(sa), b.cuda(), sb.cuda()
    x = wide(a, sa, 1) if K else torch.zeros(M, 1, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        for experts in (False, True):
            whole, c = out_like(M, N, dtype)
            if experts:
                g.fp8_experts(ad, bd, c, sad, sbd, torch.tensor(off, dtype=torch.int32).cuda())
            else:
                g.fp8(ad, bd[0], c, sad, sbd[0])
            for e, (lo, hi) in enumerate(zip(off, off[1:]) if experts else [(0, M)]):
                y = wide(b[e], sb[e], 128) if K else torch.zeros(N, 1, device="cuda")
                # (sums of at most 400 products of up to 9 * 16, in steps of 1 / 16: exact in fp32)
                assert torch.equal(c[lo:hi], (x[lo:hi] @ y.T.contiguous()).to(dtype)), (dtype, e)
            assert untouched(whole, c[:M - 2] if experts else c)


@pytest.mark.parametrize("K", [0, 16, 272, 528, 800])
@pytest.mark.parametrize("rows", [3, 20, 40])
def test_rounds_of_experts(g, rows, K):
    """The same with 40 experts of about `rows` rows, every third one with none."""
    E, N = 40, 4098
    sizes = [0 if e % 3 == 1 else rows + e % 5 - 2 for e in range(E)]
    off = torch.tensor([0] + sizes).cumsum(0)
    M = int(off[-1]) + 3
    print(f"[experts rounds {M}x{N}x{K}]", flush=True)
    a, b, sa, sb = (integers(1, M, K), integers(2, E, N, K), powers(3, M, bh.blocks(K)),
                    powers(4, E, bh.blocks(N), bh.blocks(K)))
    for dtype in (torch.bfloat16, torch.float32):
        whole, c = out_like(M, N, dtype)
        g.fp8_experts(a.cuda(), b.cuda(), c, to_row_scales(sa), sb.cuda(), off.int().cuda())
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            if hi > lo:
                want = (wide(a[lo:hi], sa[lo:hi], 1).double() @ wide(b[e], sb[e], 128).double().T if K
                        else torch.zeros(hi - lo, N, device="cuda").double())
                assert torch.equal(c[lo:hi].double(), want.to(dtype).double()), e
        assert untouched(whole, c[:int(off[-1])])


@pytest.mark.parametrize("config", range(N_CONFIGS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_every_tile_of_experts(g, config, dtype):
    """The same with 6 experts: one with most of the rows, a row, none."""
    shape = smallest_shapes(6).get((config, dtype))
    if shape is None:
        assert (config, dtype) == (0, torch.float32)
        return
    M, N, K = shape
    print(f"[experts {config}: {M}x{N}x{K} {dtype}]", flush=True)
    cuts = sorted([0, M // 50, M // 50, M - M // 5 - M // 50, M - M // 5 - min(M // 50, 1), M - M // 5, M])
    a, b = integers(1, M, K), integers(2, 6, N, K)
    sa, sb = powers(3, M, bh.blocks(K)), powers(4, 6, bh.blocks(N), bh.blocks(K))
    whole, c = out_like(M, N, dtype)
    g.fp8_experts(a.cuda(), b.cuda(), c, to_row_scales(sa), sb.cuda(), torch.tensor(cuts, dtype=torch.int32).cuda())
    for e in range(6):
        rows = slice(cuts[e], cuts[e + 1])
        want = wide(a[rows], sa[rows], 1).double() @ wide(b[e], sb[e], 128).double().T
        assert torch.equal(c[rows].double(), want.to(dtype).double()), e
    assert untouched(whole, c)


@pytest.mark.parametrize("K", [16, 128, 272, 1424])
def test_large_tile(g, K):
    """Many tiles of the large kernels, ragged at every edge."""
    M, N = 4100, 2042
    print(f"[fp8 {M}x{N}x{K}]", flush=True)
    a, b, sa, sb = (integers(K, M, K), integers(K + 1, N, K), powers(K, M, bh.blocks(K)),
                    powers(K + 1, bh.blocks(N), bh.blocks(K)))
    want = wide(a, sa, 1).double() @ wide(b, sb, 128).double().T
    for dtype in (torch.bfloat16, torch.float32):
        whole, c = out_like(M, N, dtype)
        g.fp8(a.cuda(), b.cuda(), c, to_row_scales(sa), sb.cuda())
        assert torch.equal(c.double(), want.to(dtype).double())
        assert untouched(whole, c)


@pytest.mark.parametrize("M", [1, 16, 32, 64, 100, 300])
def test_exact_every_tile(g, M):
    N, K = 264, 400
    r = gen(M)
    a = torch.randint(-3, 4, (M, K), generator=r).float().to(bh.FP8)
    b = torch.randint(-3, 4, (N, K), generator=r).float().to(bh.FP8)
    sa = (2.0 ** torch.randint(-2, 3, (M, 4), generator=r)).float()
    sb = (2.0 ** torch.randint(-2, 3, (3, 4), generator=r)).float()
    want = bh.widen(a, sa, 1) @ bh.widen(b, sb, 128).T
    for dtype in (torch.bfloat16, torch.float32):
        _, c = out_like(M, N, dtype)
        g.fp8(a.cuda().view(torch.uint8), b.cuda().view(torch.uint8), c, to_row_scales(sa), sb.cuda())
        assert torch.equal(c.cpu().double(), want.to(dtype).double())


@pytest.mark.parametrize("act", ["NONE", "RELU", "SIGMOID", "TANH", "SILU"])
@pytest.mark.parametrize("M,N,K,dtype", [(5, 136, 272, torch.bfloat16), (200, 200, 256, torch.float32),
                                         (0, 8, 16, torch.float32)])
def test_bias_and_act(g, M, N, K, dtype, act):
    a, sa, b, sb = operands(M, N, K)
    bias = torch.randn(N, generator=gen(N))
    sb = sb * 0.05
    want, err = bh.product(a, sa, b, sb, bias, act, dtype == torch.float32)
    whole, c = out_like(M, N, dtype)
    g.fp8(a.cuda(), b.cuda(), c, to_row_scales(sa), sb.cuda(), bias=bias.cuda(), act=tg.Act[act])
    bh.close(c, want, err, dtype == torch.bfloat16, act)
    assert untouched(whole, c)


@pytest.mark.parametrize("M", [3, 70, 300])
def test_no_k(g, M):
    """K = 0 stores act(bias)."""
    bias = torch.randn(40, device="cuda")
    _, c = out_like(M, 40, torch.float32)
    e = torch.empty
    g.fp8(e(M, 0, dtype=bh.FP8, device="cuda"), e(40, 0, dtype=bh.FP8, device="cuda"), c,
          e(M, 0, device="cuda"), e(1, 0, device="cuda"), bias=bias, act=tg.Act.RELU)
    assert torch.equal(c, bias.clamp(min=0).expand(M, 40))


@pytest.mark.parametrize("M,N", [(20, 300), (300, 520)])
def test_bad_scales_stay_with_their_rows(g, M, N):
    """NaN and infinite scales (a block that held such values) reach their rows and columns only."""
    K = 400
    a, sa, b, sb = operands(M, N, K)
    sa[3, 1], sa[M - 1, 3], sb[1, 2] = NAN, float("inf"), NAN
    clean_a, clean_b = sa.clone(), sb.clone()
    clean_a[3, 1] = clean_a[M - 1, 3] = clean_b[1, 2] = 1.0
    want, err = bh.product(a, clean_a, b, clean_b)
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[3] = True
    bad[:, 128:256] = True
    _, c = out_like(M, N, torch.bfloat16)
    g.fp8(a.cuda(), b.cuda(), c, to_row_scales(sa), sb.cuda())
    c = c.cpu()
    assert bool(c[bad].isnan().all())
    assert not bool(c[M - 1].isfinite().any())
    bad[M - 1] = True
    bh.close(c.float().masked_fill(bad, 0), want.masked_fill(bad, 0), err, True, "the others")


def test_nan_codes(g):
    """A NaN value reaches its row only."""
    a, sa, b, sb = operands(40, 72, 272)
    raw = a.view(torch.uint8)
    raw[7, 270] = 0x7f
    _, c = out_like(40, 72, torch.float32)
    g.fp8(a.cuda(), b.cuda(), c, to_row_scales(sa), sb.cuda())
    assert bool(c[7].isnan().all()) and not bool(torch.cat([c[:7], c[8:]]).isnan().any())


# ------------------------------------------------------------------- experts

def run_experts(g, sizes, N, K, dtype, M=None, start=0, seed=0):
    ends = [start]
    for n in sizes:
        ends.append(ends[-1] + n)
    M = ends[-1] if M is None else M
    a, sa, b, sb = operands(M, N, K, seed, (len(sizes),))
    whole, c = out_like(M, N, dtype)
    g.fp8_experts(padded(a, 16, NAN), b.cuda(), c, to_row_scales(sa, 3), sb.cuda(),
                  torch.tensor(ends, dtype=torch.int32, device="cuda"))
    got = c.cpu()
    assert bool(got[:start].isnan().all()) and bool(got[ends[-1]:].isnan().all())  # left as they were
    assert untouched(whole, c)
    for e, n in enumerate(sizes):
        if n:
            at = slice(ends[e], ends[e + 1])
            want, err = bh.product(a[at], sa[at], b[e], sb[e], fp32=dtype == torch.float32)
            bh.close(got[at], want, err, dtype == torch.bfloat16, f"expert {e}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("sizes,N,K,more", [
    ([1], 16, 16, {}),
    ([0, 3, 0, 0, 1, 0], 136, 272, {}),
    ([2, 0, 5, 9, 1, 1, 30, 0], 200, 400, dict(M=60, start=4)),
    ([0, 0, 0], 64, 128, dict(M=5)),                       # no expert has rows
    ([33, 1, 90, 0, 17, 60], 264, 528, {}),
    ([300, 0, 129, 7, 256], 392, 272, {}),
    ([700, 650, 0], 520, 400, dict(M=1401)),
    ([1] * 200 + [0] * 300 + [2] * 100, 48, 144, {}),
    ([1] * 1024, 24, 16, {}),
])
def test_experts(g, sizes, N, K, more, dtype):
    print(f"[experts {len(sizes)} {sum(sizes)}x{N}x{K} {dtype}]", flush=True)
    run_experts(g, sizes, N, K, dtype, **more)


@pytest.mark.parametrize("total", [40, 160, 400, 1000, 5000])
def test_experts_of_different_sizes(g, total):
    """A few rows of one expert beside many of another."""
    run_experts(g, [1, 0, total - 20, 0, 19, 0, 0, 0], 136, 144, torch.bfloat16, seed=total)


def test_experts_bad_offsets(g):
    """Offsets are cut to the rows there are; where they decrease an expert is empty."""
    M, N, K = 50, 72, 144
    a, sa, b, sb = operands(M, N, K, 0, (5,))
    _, c = out_like(M, N, torch.float32)
    off = torch.tensor([-7, 10, 5, 20, 60, 2000000000], dtype=torch.int32, device="cuda")
    g.fp8_experts(a.cuda(), b.cuda(), c, to_row_scales(sa), sb.cuda(), off)
    got = c.cpu()
    # expert 0: rows 0..9; 1: none; 2: rows 5..19 (5..9 either's); 3: 20..49; 4: none left
    for e, (lo, hi) in {0: (0, 5), 2: (10, 20), 3: (20, 50)}.items():
        want, err = bh.product(a[lo:hi], sa[lo:hi], b[e], sb[e], fp32=True)
        bh.close(got[lo:hi], want, err, False, f"expert {e}")
    assert bool(got.isfinite().all())


def test_experts_zigzag_offsets(g):
    """Every other expert claims all rows: far more row tiles than the output
    has. Any expert's result or none in a row, nothing outside of C."""
    M, N, K, E = 300, 72, 144, 200
    a, _, _, _ = operands(M, N, K)
    one, sa = torch.full((E, N, K), 1.0).to(bh.FP8).cuda(), to_row_scales(torch.ones(M, 2))
    whole, c = out_like(M, N, torch.float32)
    off = torch.tensor(([0, M] * E)[:E + 1], dtype=torch.int32, device="cuda")
    g.fp8_experts(a.cuda(), one, c, sa, torch.ones(E, 1, 2, device="cuda"), off)
    want = a.double().sum(1, keepdim=True).expand(M, N)
    got = c.cpu().double()
    near = (got - want).abs() <= bh.TAU * a.double().abs().sum(1, keepdim=True)
    assert bool((near | got.isnan()).all()) and untouched(whole, c)


def test_single_rows_and_blocks_of_any_stride(g):
    """The stride of a single row, or of a single block's scales, is not looked at."""
    for M, N, K in ((1, 300, 128), (70, 128, 112), (300, 100, 16), (1, 28690, 16)):
        a, sa, b, sb = operands(M, N, K)
        want, err = bh.product(a, sa, b, sb, fp32=True)
        s = tg.Fp8Strides(a_stride=-5 if M == 1 else K, b_stride=K, c_stride=-9 if M == 1 else N,
                          a_scale_stride=-(1 << 40), b_scale_stride=-3 if N <= 128 else 1)
        ad, bd, sad, sbd, c = (a.cuda(), b.cuda(), sa.t().contiguous().cuda(), sb.cuda(),
                               torch.full((M, N), NAN, device="cuda"))
        status = tg.load_library().tile_gemm_run_fp8(
            g.handle, ad.data_ptr(), bd.data_ptr(), c.data_ptr(), M, N, K, ctypes.byref(s), sad.data_ptr(),
            sbd.data_ptr(), 0, None, 0, torch.cuda.current_stream().cuda_stream)
        assert status == 0, tg.last_error_detail()
        bh.close(c, want, err, False, f"{M}x{N}x{K}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("config", [0, 1, 2])
def test_far_rows(g, config, dtype):
    """Rows of C as far apart as they may be: a tile of 256 of them spans 4 GiB."""
    shape = smallest_shapes(0).get((config, dtype))
    if shape is None:
        assert (config, dtype) == (0, torch.float32)
        return
    M, N, K = shape
    print(f"[fp8 far {config}: {M}x{N}x{K} {dtype}]", flush=True)
    a, b, sa, sb = (integers(1, M, K), integers(2, N, K), powers(3, M, bh.blocks(K)),
                    powers(4, bh.blocks(N), bh.blocks(K)))
    want = wide(a, sa, 1).double() @ wide(b, sb, 128).double().T
    c = torch.empty(M, (1 << 22) - 8, dtype=dtype, device="cuda")[:, :N]
    c.fill_(NAN)
    g.fp8(a.cuda(), b.cuda(), c, to_row_scales(sa), sb.cuda())
    assert torch.equal(c.double(), want.to(dtype).double())


def test_expert_matrices_past_4_gib(g):
    """The last experts' matrices and scales, 4 GiB and more behind the first's."""
    E, N, K = 40, 8192, 16384
    b = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    sb = torch.ones(E, 64, 128, device="cuda")
    b[E - 1, N - 1, 100:132] = 0x38  # 1.0
    b[E - 1, 5, 16000] = 0x40        # 2.0
    sb[E - 1, 63, 0], sb[E - 1, 63, 1] = 2.0, 4.0
    a = torch.full((7, K), 0x38, dtype=torch.uint8, device="cuda")
    sa = to_row_scales(torch.ones(7, 128))
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[E] = 7
    c = torch.full((7, N), NAN, device="cuda")
    g.fp8_experts(a, b, c, sa, sb, off.cuda())
    want = torch.zeros(7, N)
    want[:, N - 1] = 28 * 2.0 + 4 * 4.0
    want[:, 5] = 2.0
    assert torch.equal(c.cpu(), want)


# -------------------------------------------------------------- quantization

def rows_of(x, seed=0):
    return torch.randn(*x, generator=gen(seed)) * torch.randn(x[0], 1, generator=gen(seed + 1)).exp()


@pytest.mark.parametrize("M,K", [(1, 16), (1, 8192), (5, 144), (16, 512), (17, 528), (130, 1040), (33, 4096)])
def test_quantize_rows(g, M, K):
    x = rows_of((M, K)).bfloat16()
    want_q, want_s = bh.quantize(x.float(), 1)
    xd = padded(x, 8, NAN)
    whole = torch.full((M, K + 16), 0x7e, dtype=torch.uint8, device="cuda")
    s = bh.row_scales(M, K, "cuda", 3)
    g.quantize(xd, whole[:, :K], s)
    assert torch.equal(whole[:, :K].cpu(), want_q.view(torch.uint8))
    assert torch.equal(s.cpu(), want_s)
    assert bool((whole[:, K:] == 0x7e).all()) and bool(s.t().storage_offset() == 0)


@pytest.mark.parametrize("M,K", [(1, 16), (128, 128), (300, 272), (129, 1040), (64, 400)])
def test_quantize_blocks(g, M, K):
    x = rows_of((M, K), 3).bfloat16()
    want_q, want_s = bh.quantize(x.float(), 128)
    q = torch.empty(M, K, dtype=bh.FP8, device="cuda")
    s = torch.full((bh.blocks(M), bh.blocks(K) + 2), NAN, device="cuda")
    g.quantize(padded(x, 8, NAN), q, s[:, :bh.blocks(K)], form=tg.Quant.BLOCKS)
    assert torch.equal(q.cpu().view(torch.uint8), want_q.view(torch.uint8))
    assert torch.equal(s.cpu()[:, :bh.blocks(K)], want_s) and bool(s[:, bh.blocks(K):].isnan().all())


@pytest.mark.parametrize("form", ["ROWS", "BLOCKS"])
def test_quantize_special_values(g, form):
    """Zeros, tiny and largest values; a NaN or infinity is its block's scale."""
    x = torch.zeros(256, 384)
    x[0, 0], x[1, 3], x[2, 7] = 1e-38, 2.0 ** -126, -3e38
    x[130, 5], x[140, 250], x[200, 300] = NAN, float("inf"), float("-inf")
    x[130, 9], x[140, 251] = 7.0, 3.0
    x = x.bfloat16()
    q = torch.empty(256, 384, dtype=bh.FP8, device="cuda")
    if form == "ROWS":
        s, high = bh.row_scales(256, 384, "cuda"), 1
    else:
        s, high = torch.empty(2, 3, device="cuda"), 128
    g.quantize(x.cuda(), q, s, form=tg.Quant[form])
    q, s = q.cpu().float(), s.cpu()
    want_q, want_s = bh.quantize(x.float(), high)
    finite = want_s.isfinite()
    assert torch.equal(s[finite], want_s[finite]) and bool((s[finite] > 0).all())
    wide = finite.repeat_interleave(high, 0).repeat_interleave(128, 1)
    assert torch.equal(q[wide], want_q.float()[wide])
    b = lambda r, c: (r // high, c // 128)  # noqa: E731
    assert s[b(130, 5)].isnan() and s[b(140, 250)] == float("inf") and s[b(200, 300)] == float("inf")
    # a product that reads such a block is not finite
    c = torch.empty(256, 128, device="cuda")
    if form == "ROWS":
        one = torch.full((128, 384), 1.0).to(bh.FP8).cuda()
        g.fp8(q.to(bh.FP8).cuda(), one, c, to_row_scales(s), torch.ones(1, 3, device="cuda"))
        bad = ~c.cpu().isfinite()
        assert bool(bad[[130, 140, 200]].all()) and int(bad.any(1).sum()) == 3


def test_quantize_gathered(g):
    """Rows by number, one of them twice; a number that is no row leaves its
    row and scales as they were."""
    x = rows_of((21, 272), 5).bfloat16()
    rows = torch.tensor([20, 0, -1, 7, 7, 21, 3, 2000000000, -2000000000, 1] * 5, dtype=torch.int32)
    want_q, want_s = bh.quantize(x.float(), 1)
    q = torch.full((50, 272), 0x55, dtype=torch.uint8, device="cuda")
    s = bh.row_scales(50, 272, "cuda")
    s.fill_(-5.0)
    g.quantize(x.cuda(), q, s, rows=rows.cuda())
    on = (rows >= 0) & (rows < 21)
    q, s = q.cpu(), s.cpu()
    assert torch.equal(q[on], want_q.view(torch.uint8)[rows[on].long()]) and torch.equal(s[on], want_s[rows[on].long()])
    assert bool((q[~on] == 0x55).all()) and bool((s[~on] == -5.0).all())


@pytest.mark.parametrize("form", ["ROWS", "BLOCKS"])
def test_quantize_many_rows(g, form):
    """More rows than the workgroups a grid has along a second axis of 65535."""
    M = 8500003 // 8 if form == "ROWS" else (1 << 22) - 5
    x = (torch.arange(M, device="cuda") % 251 + 1).bfloat16()[:, None].expand(M, 16).contiguous()
    q = torch.zeros(M, 16, dtype=torch.uint8, device="cuda")
    if form == "ROWS":
        s = bh.row_scales(M, 16, "cuda")
        g.quantize(x, q, s)
        assert bool((q == 0x7e).all())  # 448
        # (the nearest fp32 value; a division of tensors on the GPU may be a product by 1 / 448)
        assert torch.equal(s[:, 0], (x[:, 0].double() / 448).float())
    else:
        s = torch.zeros(bh.blocks(M), 1, device="cuda")
        g.quantize(x, q, s, form=tg.Quant.BLOCKS)
        top = torch.nn.functional.pad(x[:, 0].float(), (0, -M % 128)).view(-1, 128).amax(1)
        assert torch.equal(s[:, 0], (top.double() / 448).float())
        back = q.view(bh.FP8).float() * s.repeat_interleave(128, 0)[:M]
        assert bool(((back - x.float()).abs() <= x.float() / 16 * 1.0001).all())


@pytest.mark.parametrize("gate", ["SILU", "GELU", "GELU_TANH", "RELU", "SIGMOID"])
@pytest.mark.parametrize("M,K", [(1, 16), (40, 400)])
def test_quantize_gated(g, M, K, gate):
    from train_helpers import act_slope
    x = torch.randn(M, 2 * K, generator=gen(K)).bfloat16() * 2
    act, _ = act_slope(x[:, :K].double(), gate)
    want = act * x[:, K:].double()
    q = torch.empty(M, K, dtype=bh.FP8, device="cuda")
    s = bh.row_scales(M, K, "cuda")
    g.quantize(padded(x, 8, NAN), q, s, gate=tg.Gate[gate])
    top = torch.nn.functional.pad(want.abs(), (0, -K % 128)).view(M, -1, 128).amax(2).clamp(min=2.0 ** -100)
    # the activation in fp32: EVAL of the value, and 2^-22 where it is a small difference
    err = bh.EVAL * want.abs() + 2.0 ** -22 * x[:, K:].double().abs()
    worst = torch.nn.functional.pad(err, (0, -K % 128)).view(M, -1, 128).amax(2)
    assert bool(((s.cpu().double() - top / 448).abs() <= worst / 448 + 2.0 ** -23 * top / 448).all())
    wide = s.cpu().double().repeat_interleave(128, 1)[:, :K]
    half_step = torch.maximum(2.0 ** -4 * (want.abs() + err), 2.0 ** -10 * wide)
    bh.close(q.cpu().double() * wide, want, err + half_step + 2.0 ** -22 * want.abs(), False, gate)


# --------------------------------------------------------------- as it is used

def test_streams_and_graph(g):
    """A projection on another stream, and captured and replayed on new values."""
    M, N, K = 70, 264, 528
    x = rows_of((M, K), 9).bfloat16().cuda()
    w = rows_of((N, K), 11).bfloat16().cuda()
    e = torch.empty
    qw, sw = e(N, K, dtype=bh.FP8, device="cuda"), e(3, 5, device="cuda")
    g.quantize(w, qw, sw, form=tg.Quant.BLOCKS)

    def step(x, q, s, c, stream=None):
        g.quantize(x, q, s, stream=stream)
        g.fp8(q, qw, c, s, sw, stream=stream)

    def buffers():
        return e(M, K, dtype=bh.FP8, device="cuda"), bh.row_scales(M, K, "cuda"), torch.full((M, N), NAN, device="cuda")
    eager = buffers()
    step(x, *eager)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    b1 = buffers()
    torch.cuda.synchronize()
    step(x, *b1, stream=other)
    other.synchronize()
    assert torch.equal(b1[2], eager[2])
    b2, x2 = buffers(), x.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x2, *b2)
    for r in range(3):
        x2.copy_(x * (r + 1))
        step(x2, *eager)
        b2[2].fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b2[2], eager[2])


def test_runs_are_identical(g):
    a, sa, b, sb = operands(300, 520, 1040)
    args = a.cuda(), b.cuda(), to_row_scales(sa), sb.cuda()
    first = None
    for _ in range(5):
        c = torch.empty(300, 520, device="cuda", dtype=torch.bfloat16)
        g.fp8(args[0], args[1], c, *args[2:])
        first = c if first is None else first
        assert torch.equal(c, first)


def test_binding_refusals(g):
    a, sa, b, sb = operands(20, 136, 272)
    a, b, sb, c = a.cuda(), b.cuda(), sb.cuda(), torch.empty(20, 136, device="cuda")
    s = to_row_scales(sa)
    for bad, error in (((a.float(), b, c, s, sb), TypeError), ((a, b[:, :256], c, s, sb), ValueError),
                       ((a, b, c[:, :130], s, sb), ValueError), ((a, b, c.half(), s, sb), TypeError),
                       ((a, b, c, s.contiguous(), sb), ValueError), ((a, b, c, s[:, :2], sb), ValueError),
                       ((a, b, c, s, sb[:1]), ValueError), ((a, b, c, s.double(), sb), TypeError),
                       ((a.cpu(), b, c, s, sb), ValueError), ((a, b, c.t(), s, sb), ValueError),
                       ((a, b.t(), c, s, sb), ValueError)):
        with pytest.raises(error):
            g.fp8(*bad)
    be, sbe, off = b.view(1, *b.shape), sb.view(1, *sb.shape), torch.tensor([0, 20], dtype=torch.int32).cuda()
    g.fp8_experts(a, be, c, s, sbe, off)
    for call, good in ((g.fp8, (a, b, c, s, sb)), (g.fp8_experts, (a, be, c, s, sbe, off))):
        for i, t in enumerate(good):  # one of them in host memory, or of another type
            with pytest.raises(ValueError):
                call(*good[:i], t.cpu(), *good[i + 1:])
            with pytest.raises(TypeError):
                call(*good[:i], t.to(torch.float64), *good[i + 1:])
    for bad, error in (((a, be[:, :, :256], c, s, sbe, off), ValueError), ((a, be, c, s, sbe[:, :1], off), ValueError),
                       ((a, be, c, s, sbe, off[:1]), ValueError), ((a, b, c, s, sb, off), ValueError)):
        with pytest.raises(error):
            g.fp8_experts(*bad)
    with pytest.raises(tg.TileGemmError):  # K not a multiple of 16
        g.fp8(a[:, :264], b[:, :264], c, s, sb)
    x, q = torch.empty(20, 272, dtype=torch.bfloat16, device="cuda"), torch.empty(20, 272, dtype=bh.FP8, device="cuda")
    for args, kw, error in (((x.float(), q, s), {}, TypeError), ((x[:, :256], q, s), {}, ValueError),
                            ((x, q, s), dict(gate=tg.Gate.SILU), ValueError),
                            ((x, q, s), dict(form=tg.Quant.GATED_ROWS), ValueError),
                            ((x, q, sb[:1]), dict(form=tg.Quant.BLOCKS, gate=tg.Gate.SILU), ValueError),
                            ((x, q, s), dict(rows=torch.zeros(19, dtype=torch.int32, device="cuda")), ValueError),
                            ((x, q, s), dict(rows=torch.zeros(20, device="cuda")), TypeError)):
        with pytest.raises(error):
            g.quantize(*args, **kw)
