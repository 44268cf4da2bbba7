"""Host-side checks of the E4M3 products with block scales, of the
quantization, of the routing to experts and of the experts' sums: refusals
before anything is enqueued, plans and workspace sizes. No GPU: pointers are
plain integers."""

import ctypes

import pytest

import tile_partitioned_dense_amd as tg
from tile_partitioned_dense_amd import Fp8Strides, RouteOptions, Status, binding

A0, B0, C0, SA, SB, BIAS, OFF, ROWS, IDS, WS = (i << 34 for i in range(1, 11))
OK, SHAPE, STRIDE, NULL = Status.OK, Status.ERR_BAD_SHAPE, Status.ERR_BAD_STRIDE, Status.ERR_NULL_ARG
MISALIGNED, ALIAS, DTYPE = Status.ERR_MISALIGNED, Status.ERR_ALIAS, Status.ERR_DTYPE


def lib():
    return tg.load_library()


def ref(x):
    return None if x is None else ctypes.byref(x)


def fp8(E=None, **kw):
    M, N, K = kw.pop("M", 100), kw.pop("N", 200), kw.pop("K", 272)
    kb = -(-K // 128)
    s = dict(a_stride=K, b_stride=K, c_stride=N, a_scale_stride=M, b_scale_stride=kb, b_expert_stride=N * K,
             b_scale_expert_stride=-(-N // 128) * kb)
    s |= {k: kw.pop(k) for k in list(kw) if k in s}
    a = dict(A=A0, B=B0, C=C0, offsets=OFF, sa=SA, sb=SB, dtype=1, bias=None, act=0,
             strides=Fp8Strides(**s)) | kw
    if E is None:
        return Status(lib().tile_gemm_check_fp8(a["A"], a["B"], a["C"], M, N, K, ref(a["strides"]), a["sa"], a["sb"],
                                                a["dtype"], a["bias"], a["act"]))
    return Status(lib().tile_gemm_check_fp8_experts(a["A"], a["B"], a["C"], M, N, K, E, a["offsets"],
                                                    ref(a["strides"]), a["sa"], a["sb"], a["dtype"]))


@pytest.mark.parametrize("kw,status", [
    ({}, OK),
    (dict(bias=BIAS, act=4), OK),
    (dict(dtype=0), OK),
    (dict(dtype=2), DTYPE),
    (dict(act=5), Status.ERR_EPILOGUE),
    (dict(act=-1), Status.ERR_EPILOGUE),
    (dict(A=None), NULL), (dict(B=None), NULL), (dict(C=None), NULL), (dict(sa=None), NULL), (dict(sb=None), NULL),
    (dict(strides=None), NULL),
    (dict(M=0, A=None, C=None), OK), (dict(N=0, B=None, C=None), OK),
    (dict(K=0, A=None, B=None, sa=None, sb=None), OK),
    (dict(M=-1), SHAPE), (dict(M=1 << 22), SHAPE), (dict(N=1 << 22), SHAPE), (dict(K=1 << 22), SHAPE),
    (dict(K=264), SHAPE),
    (dict(M=(1 << 22) - 16, N=(1 << 22) - 16, K=16), SHAPE),  # too many tiles
    (dict(M=(1 << 22) - 16, N=(1 << 18) + 64, K=16), SHAPE),   # (of 16 x 32)
    (dict(a_stride=256), STRIDE), (dict(a_stride=1 << 22), STRIDE), (dict(a_stride=280), MISALIGNED),
    (dict(b_stride=256), STRIDE), (dict(b_stride=280), MISALIGNED),
    (dict(c_stride=196), STRIDE), (dict(c_stride=202), MISALIGNED),
    (dict(a_scale_stride=99), STRIDE), (dict(a_scale_stride=1 << 31), STRIDE),
    (dict(b_scale_stride=2), STRIDE), (dict(b_scale_stride=1 << 22), STRIDE),
    (dict(K=128, a_scale_stride=0), OK),                       # one block: its stride is any
    (dict(N=128, b_scale_stride=0), OK),
    (dict(M=1, a_stride=3), OK),
    (dict(A=A0 + 8), MISALIGNED), (dict(B=B0 + 8), MISALIGNED), (dict(C=C0 + 8), MISALIGNED),
    (dict(sa=SA + 2), MISALIGNED), (dict(sa=SA + 4), OK), (dict(sb=SB + 4), OK), (dict(bias=BIAS + 4), MISALIGNED),
    (dict(C=A0), ALIAS), (dict(C=B0 + 16), ALIAS), (dict(C=SA), ALIAS), (dict(C=SB), ALIAS),
    (dict(C=BIAS, bias=BIAS), ALIAS),
])
def test_fp8(kw, status):
    assert fp8(**kw) == status, tg.last_error_detail()


@pytest.mark.parametrize("kw,status", [
    (dict(E=8), OK),
    (dict(E=1024), OK),
    (dict(E=0), SHAPE), (dict(E=-1), SHAPE), (dict(E=1025), SHAPE),
    (dict(E=8, offsets=None), NULL), (dict(E=8, offsets=OFF + 2), MISALIGNED), (dict(E=8, offsets=C0), ALIAS),
    (dict(E=8, b_expert_stride=200 * 272 - 16), STRIDE), (dict(E=8, b_expert_stride=200 * 272 + 8), MISALIGNED),
    (dict(E=1, b_expert_stride=0, b_scale_expert_stride=0), OK),
    (dict(E=8, b_scale_expert_stride=5), STRIDE),
    (dict(E=8, b_stride=280), MISALIGNED),
    (dict(E=8, N=1 << 21, K=1024, b_expert_stride=1 << 31), SHAPE),  # 2 GiB for one expert
    (dict(E=8, C=B0 + 7 * 200 * 272), ALIAS),                       # the last expert's matrix
])
def test_fp8_experts(kw, status):
    assert fp8(**kw) == status, tg.last_error_detail()


def test_expert_matrices_past_4_gib():
    # 64 experts of 128 MiB
    assert fp8(E=64, N=16384, K=8192, M=512, C=1 << 60) == OK


def quantize(**kw):
    M, K = kw.pop("M", 100), kw.pop("K", 272)
    form = kw.get("form", 0)
    kb = -(-K // 128)
    a = dict(X=A0, Q=B0, scale=SA, ldx=2 * K if form == 1 else K, ldq=K, lds=kb if form == 2 else M, form=0, gate=0,
             rows=None, x_rows=0) | kw
    return Status(lib().tile_gemm_check_quantize(a["X"], a["Q"], a["scale"], M, K, a["ldx"], a["ldq"], a["lds"],
                                                 a["form"], a["gate"], a["rows"], a["x_rows"]))


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(form=1), OK), (dict(form=2), OK),
    (dict(form=3), DTYPE), (dict(form=-1), DTYPE), (dict(form=1, gate=5), Status.ERR_EPILOGUE),
    (dict(form=0, gate=77), OK),                              # not looked at
    (dict(rows=ROWS, x_rows=7), OK), (dict(rows=ROWS, x_rows=0, X=None), OK), (dict(rows=ROWS, x_rows=-1), SHAPE),
    (dict(form=2, rows=ROWS, x_rows=7), SHAPE),
    (dict(M=0, X=None, Q=None, scale=None), OK), (dict(K=0, X=None, Q=None, scale=None), OK),
    (dict(M=1 << 22), SHAPE), (dict(K=1 << 22), SHAPE), (dict(K=264), SHAPE), (dict(M=-1), SHAPE),
    (dict(X=None), NULL), (dict(Q=None), NULL), (dict(scale=None), NULL),
    (dict(ldx=256), STRIDE), (dict(form=1, ldx=528), STRIDE), (dict(ldq=256), STRIDE), (dict(lds=99), STRIDE),
    (dict(form=2, lds=2), OK), (dict(form=2, lds=2, M=200), STRIDE), (dict(ldx=276), MISALIGNED), (dict(ldq=280), MISALIGNED),
    (dict(X=A0 + 8), MISALIGNED), (dict(Q=B0 + 8), MISALIGNED), (dict(scale=SA + 2), MISALIGNED),
    (dict(rows=ROWS + 2, x_rows=7), MISALIGNED),
    (dict(Q=A0), ALIAS), (dict(scale=A0), ALIAS), (dict(scale=B0), ALIAS), (dict(rows=B0, x_rows=7), ALIAS),
])
def test_quantize(kw, status):
    assert quantize(**kw) == status, tg.last_error_detail()


def route(back=False, **kw):
    T, E, k = kw.pop("T", 100), kw.pop("E", 64), kw.pop("k", 4)
    o = dict(score=0, logits_type=0, groups=1, top_groups=1, group_top=2, renormalize=1, scale=1.0)
    o |= {n: kw.pop(n) for n in list(kw) if n in o}
    a = dict(logits=A0, bias=None, ids=IDS, weights=B0, ld=E, ldd=E, dlogits=C0, options=RouteOptions(**o)) | kw
    if back:
        return Status(lib().tile_gemm_check_route_backward(a["logits"], a["ids"], a["weights"], a["dlogits"], T, E, k,
                                                           a["ld"], a["ldd"], ref(a["options"])))
    return Status(lib().tile_gemm_check_route(a["logits"], a["bias"], a["ids"], a["weights"], T, E, k, a["ld"],
                                              ref(a["options"])))


COMMON = [
    ({}, OK), (dict(score=1, logits_type=1), OK), (dict(score=2), DTYPE), (dict(logits_type=2), DTYPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(options=None), NULL),
    (dict(E=0), SHAPE), (dict(E=1024), OK), (dict(E=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=32), OK),
    (dict(k=33), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(ld=63), STRIDE),
    (dict(T=1 << 25), SHAPE),
    (dict(T=0, logits=None, ids=None, weights=None, dlogits=None), OK),
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(weights=None), NULL),
    (dict(logits=A0 + 2), MISALIGNED), (dict(logits=A0 + 2, logits_type=1), OK), (dict(ids=IDS + 2), MISALIGNED),
    (dict(T=1, ld=0), OK),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(groups=8, top_groups=4), OK), (dict(groups=7), SHAPE), (dict(groups=0), SHAPE),
    (dict(E=128, groups=128, top_groups=64), SHAPE), (dict(groups=8, top_groups=9), SHAPE),
    (dict(groups=8, top_groups=0), SHAPE), (dict(group_top=3), SHAPE), (dict(group_top=0), SHAPE),
    (dict(groups=8, top_groups=1, k=8), OK), (dict(groups=8, top_groups=1, k=9), SHAPE), (dict(E=3, k=4), SHAPE),
    (dict(bias=BIAS), OK), (dict(bias=BIAS + 2), MISALIGNED),
    (dict(ids=A0), ALIAS), (dict(weights=A0 + 4), ALIAS), (dict(weights=IDS), ALIAS), (dict(bias=B0), ALIAS),
])
def test_route(kw, status):
    assert route(**kw) == status, tg.last_error_detail()


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(dlogits=None), NULL), (dict(ldd=63), STRIDE), (dict(dlogits=C0 + 2), MISALIGNED),
    (dict(dlogits=A0), ALIAS), (dict(dlogits=IDS), ALIAS), (dict(dlogits=B0), ALIAS),
    (dict(groups=7, top_groups=0, group_top=9), OK),          # of the choice: not looked at
])
def test_route_backward(kw, status):
    assert route(back=True, **kw) == status, tg.last_error_detail()


def place(**kw):
    a = dict(ids=IDS, T=5000, k=4, first=0, E=64, offsets=OFF, rows=ROWS, places=A0, ws=WS, bytes=1 << 30) | kw
    return Status(lib().tile_gemm_check_place(a["ids"], a["T"], a["k"], a["first"], a["E"], a["offsets"], a["rows"],
                                              a["places"], a["ws"], a["bytes"]))


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(rows=None), OK), (dict(places=None), OK), (dict(rows=None, places=None), OK),
    (dict(ids=None), NULL), (dict(offsets=None), NULL), (dict(T=0, ids=None, rows=None, places=None), OK),
    (dict(T=0, offsets=None), NULL),                          # its zeros are still written
    (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(k=0), SHAPE), (dict(T=-1), SHAPE), (dict(first=-1), SHAPE),
    (dict(first=1 << 31), SHAPE), (dict(T=1 << 30, k=2), SHAPE),
    (dict(ws=None), Status.ERR_WORKSPACE), (dict(ws=WS + 8), Status.ERR_WORKSPACE),
    (dict(bytes=64), Status.ERR_WORKSPACE), (dict(T=100, ws=None, bytes=0), OK),
    (dict(ids=IDS + 1), MISALIGNED), (dict(rows=IDS), ALIAS), (dict(places=IDS), ALIAS), (dict(offsets=ROWS), ALIAS),
    (dict(ws=IDS), ALIAS),
])
def test_place(kw, status):
    assert place(**kw) == status, tg.last_error_detail()


def test_place_workspace():
    assert tg.tile_gemm_place_workspace(8, 4, 64) == 0
    for T, k, E in ((5000, 4, 64), (100000, 8, 256), (1 << 28, 7, 1024)):
        n = tg.tile_gemm_place_workspace(T, k, E)
        assert 0 < n <= 128 * E * 4
        assert place(T=T, k=k, E=E, bytes=n, rows=1 << 50, places=1 << 51, ids=1 << 52) == OK
        assert place(T=T, k=k, E=E, bytes=n - 1, rows=1 << 50, places=1 << 51, ids=1 << 52) == Status.ERR_WORKSPACE
    with pytest.raises(tg.TileGemmError):
        tg.tile_gemm_place_workspace(-1, 4, 64)


def combine(**kw):
    T, N, k = kw.pop("T", 100), kw.pop("N", 200), kw.pop("k", 4)
    a = dict(Z=A0, places=IDS, weights=B0, Y=C0, z_rows=400, ldz=N, ldy=N, dtype=1) | kw
    return Status(lib().tile_gemm_check_combine(a["Z"], a["places"], a["weights"], a["Y"], T, N, k, a["z_rows"],
                                                a["ldz"], a["ldy"], a["dtype"]))


@pytest.mark.parametrize("kw,status", [
    ({}, OK), (dict(dtype=0), OK), (dict(dtype=3), DTYPE), (dict(weights=None), OK),
    (dict(z_rows=0, Z=None), OK), (dict(z_rows=-1), SHAPE),
    (dict(T=0, places=None, Y=None, weights=None), OK), (dict(N=0, Z=None, Y=None), OK),
    (dict(k=0), SHAPE), (dict(k=64), OK), (dict(k=65), SHAPE), (dict(T=1 << 22), SHAPE), (dict(N=1 << 22), SHAPE),
    (dict(T=(1 << 22) - 1, N=8200), SHAPE),  # threads of one launch
    (dict(Z=None), NULL), (dict(places=None), NULL), (dict(Y=None), NULL),
    (dict(ldz=196), STRIDE), (dict(ldy=196), STRIDE), (dict(ldz=204), MISALIGNED), (dict(ldy=204), MISALIGNED),
    (dict(Z=A0 + 2), MISALIGNED), (dict(places=IDS + 2), MISALIGNED),
    (dict(Y=A0), ALIAS), (dict(Y=IDS), ALIAS), (dict(Y=B0), ALIAS),
])
def test_combine(kw, status):
    assert combine(**kw) == status, tg.last_error_detail()


def test_null_handle():
    L, s, o = lib(), Fp8Strides(), RouteOptions()
    assert L.tile_gemm_run_fp8(None, A0, B0, C0, 1, 1, 16, ctypes.byref(s), SA, SB, 1, None, 0, None) == NULL
    assert L.tile_gemm_run_fp8_experts(None, A0, B0, C0, 1, 1, 16, 1, OFF, ctypes.byref(s), SA, SB, 1, None) == NULL
    assert L.tile_gemm_run_quantize(None, A0, B0, SA, 1, 16, 16, 16, 1, 0, 0, None, 0, None) == NULL
    assert L.tile_gemm_run_route(None, A0, None, IDS, B0, 1, 8, 1, 8, ctypes.byref(o), None) == NULL
    assert L.tile_gemm_run_route_backward(None, A0, IDS, B0, C0, 1, 8, 1, 8, 8, ctypes.byref(o), None) == NULL
    assert L.tile_gemm_run_place(None, IDS, 1, 1, 0, 1, OFF, None, None, None, 0, None) == NULL
    assert L.tile_gemm_run_combine(None, A0, IDS, None, C0, 1, 8, 1, 1, 8, 8, 1, None) == NULL


@pytest.mark.parametrize("M,N,E,dtype", [
    (1, 64, 0, 1), (16, 28672, 0, 1), (33, 200, 0, 0), (100, 100, 0, 1), (8192, 7168, 0, 1), (1999, 5464, 0, 0),
    (192, 4096, 64, 1), (16396, 7168, 16, 1), (16396, 7168, 16, 0), (1, 16, 1024, 1),
])
def test_plan(M, N, E, dtype):
    p = tg.tile_gemm_plan_fp8(M, N, 1024, E, tg.Dtype(dtype))
    assert p.tiles >= -(-M // p.bm) * -(-N // p.bn) and 1 <= p.grid <= p.tiles
    assert p.lds_bytes <= 160 * 1024 and p.threads <= 1024


def test_plan_refusals():
    for bad in (dict(M=-1), dict(K=1 << 22), dict(experts=1025), dict(cu_count=0)):
        with pytest.raises(tg.TileGemmError):
            tg.tile_gemm_plan_fp8(**(dict(M=8, N=8, K=16) | bad))
    p = binding.Plan()
    assert lib().tile_gemm_plan_fp8(8, 8, 16, 0, 5, 256, ctypes.byref(p)) == DTYPE
    assert lib().tile_gemm_plan_fp8(8, 8, 16, 0, 1, 256, None) == NULL


def host_operands():
    torch = pytest.importorskip("torch")
    u8, i32 = torch.uint8, torch.int32
    z = torch.zeros
    a, sa = z(8, 256, dtype=u8), z(2, 8).t()
    return {
        "fp8": (a, z(64, 256, dtype=u8), z(8, 64), sa, z(1, 2)),
        "fp8_experts": (a, z(3, 64, 256, dtype=u8), z(8, 64), sa, z(3, 1, 2), z(4, dtype=i32)),
        "quantize": (z(8, 256, dtype=torch.bfloat16), a, sa),
        "route": (z(8, 16), z(8, 2, dtype=i32), z(8, 2)),
        "route_backward": (z(8, 16), z(8, 2, dtype=i32), z(8, 2), z(8, 16)),
        "place": (z(8, 2, dtype=i32), z(17, dtype=i32), z(16, dtype=i32), z(8, 2, dtype=i32)),
        "combine": (z(16, 64, dtype=torch.bfloat16), z(8, 2, dtype=i32), z(8, 2), z(8, 64)),
    }


@pytest.mark.parametrize("name", ["fp8", "fp8_experts", "quantize", "route", "route_backward", "place", "combine"])
def test_host_tensors_are_refused(name):
    """A tensor in host memory never reaches the library."""
    call = getattr(tg, "tile_gemm_run_" + name)
    with pytest.raises(ValueError, match="must be on the GPU"):
        call(None, *host_operands()[name])
    for i in range(len(host_operands()[name])):  # nor does anything but a tensor
        bad = list(host_operands()[name])
        bad[i] = 12345
        with pytest.raises((TypeError, AttributeError)):
            call(None, *bad)
