"""Host-side checks of the gated block's backward pass and of the cross entropy
head: argument refusals before anything is enqueued, and workspace sizes. No
GPU: pointers are plain integers."""

import pytest

import tile_partitioned_dense_amd as tg
from tile_partitioned_dense_amd import Status, XentOptions

A0, B0, C0, DA, DB, BIAS, DBIAS, WS = (i << 32 for i in range(1, 9))
T0, LOSS, LSE, DLOSS = (i << 32 for i in range(9, 13))
BIG = 1 << 31


def glu(**kw):
    M, N, K = kw.pop("M", 100), kw.pop("N", 64), kw.pop("K", 40)
    a = dict(A=A0, B=B0, dC=C0, dA=DA, dB=DB, strides=(K, 1, 1, K, 0, 0), grad_strides=(K, 1, 1, K, N // 2, 1),
             bias=BIAS, dbias=DBIAS, gate=0, workspace=WS, workspace_bytes=BIG) | kw
    return tg.tile_gemm_check_glu_backward(M=M, N=N, K=K, **a)


def xent(back=False, **kw):
    M, N, K = kw.pop("M", 100), kw.pop("N", 1000), kw.pop("K", 40)
    o = dict(ignore_index=-100, label_smoothing=0.0, z_loss=0.0, piece=0, target_type=1)
    o |= {k: kw.pop(k) for k in list(kw) if k in o}
    a = dict(A=A0, B=B0, target=T0, strides=(K, 1, 1, K, 0, 0), options=XentOptions(**o), workspace=WS,
             workspace_bytes=BIG)
    if back:
        a |= dict(lse=LSE, dloss=DLOSS, dA=DA, dB=DB, grad_strides=(K, 1, 1, K, 0, 0))
        return tg.tile_gemm_check_xent_backward(M=M, N=N, K=K, **(a | kw))
    return tg.tile_gemm_check_xent(M=M, N=N, K=K, **(a | dict(loss=LOSS, lse=LSE) | kw))


@pytest.mark.parametrize("kw,status", [
    ({}, Status.OK),
    (dict(bias=None, dbias=None), Status.OK),
    (dict(dA=None), Status.OK),
    (dict(dA=None, dB=None), Status.OK),
    (dict(dA=None, dB=None, dbias=None), Status.ERR_NULL_ARG),
    (dict(A=None), Status.ERR_NULL_ARG),
    (dict(B=None), Status.ERR_NULL_ARG),
    (dict(dC=None), Status.ERR_NULL_ARG),
    (dict(strides=None), Status.ERR_NULL_ARG),
    (dict(M=0, A=None, B=None, dC=None, dA=None, workspace=None), Status.OK),
    (dict(N=0, A=None, B=None, dC=None, dB=None, bias=None, dbias=None, workspace=None), Status.OK),
    (dict(K=0), Status.ERR_BAD_SHAPE),
    (dict(M=-1), Status.ERR_BAD_SHAPE),
    (dict(N=72), Status.ERR_BAD_SHAPE),
    (dict(M=1 << 22), Status.ERR_BAD_SHAPE),
    (dict(K=1 << 22), Status.ERR_BAD_SHAPE),
    (dict(gate=5), Status.ERR_EPILOGUE),
    (dict(gate=-1), Status.ERR_EPILOGUE),
    (dict(strides=(40, 2, 1, 40, 0, 0)), Status.ERR_BAD_STRIDE),
    (dict(strides=(32, 1, 1, 40, 0, 0)), Status.ERR_BAD_STRIDE),
    (dict(strides=(40, 1, 64, 1, 0, 0)), Status.ERR_BAD_STRIDE),
    (dict(strides=(40, 1, 1, 32, 0, 0)), Status.ERR_BAD_STRIDE),
    (dict(strides=(40, 1, 1, 1 << 22, 0, 0)), Status.ERR_BAD_STRIDE),
    (dict(strides=(1 << 31, 1, 1, 40, 0, 0)), Status.ERR_BAD_STRIDE),
    (dict(grad_strides=(40, 1, 1, 40, 24, 1)), Status.ERR_BAD_STRIDE),
    (dict(grad_strides=(40, 1, 64, 1, 32, 1)), Status.ERR_BAD_STRIDE),
    (dict(grad_strides=(40, 2, 1, 40, 32, 1)), Status.ERR_BAD_STRIDE),
    (dict(strides=(44, 1, 1, 40, 0, 0)), Status.ERR_MISALIGNED),
    (dict(grad_strides=(44, 1, 1, 40, 32, 1)), Status.ERR_MISALIGNED),
    (dict(A=A0 + 8), Status.ERR_MISALIGNED),
    (dict(dB=DB + 2), Status.ERR_MISALIGNED),
    (dict(bias=BIAS + 4), Status.ERR_MISALIGNED),
    (dict(M=1, strides=(7, 1, 1, 40, 0, 0)), Status.OK),  # a single row has no stride
    (dict(M=1 << 21, K=2048, strides=(2048, 1, 1, 2048, 0, 0), grad_strides=(2048, 1, 1, 2048, 32, 1),
          workspace_bytes=1 << 40), Status.ERR_BAD_SHAPE),  # A of 8 GiB
    (dict(dA=A0), Status.ERR_ALIAS),
    (dict(dB=B0 + 64 * 80 - 16), Status.ERR_ALIAS),
    (dict(dB=B0 + 64 * 80), Status.OK),
    (dict(dbias=BIAS), Status.ERR_ALIAS),
    (dict(workspace=C0), Status.ERR_ALIAS),
    (dict(dC=A0, M=100), Status.OK),  # inputs may share memory
    (dict(workspace=None), Status.ERR_WORKSPACE),
    (dict(workspace=WS + 16), Status.ERR_WORKSPACE),
    (dict(workspace_bytes=1000), Status.ERR_WORKSPACE),
])
def test_glu_backward(kw, status):
    assert glu(**kw) == status, tg.last_error_detail()


@pytest.mark.parametrize("kw,status", [
    ({}, Status.OK),
    (dict(loss=None), Status.OK),
    (dict(lse=None), Status.OK),
    (dict(loss=None, lse=None), Status.ERR_NULL_ARG),
    (dict(A=None), Status.ERR_NULL_ARG),
    (dict(target=None), Status.ERR_NULL_ARG),
    (dict(M=0, A=None, target=None, loss=LOSS, workspace=None), Status.OK),
    (dict(N=0), Status.ERR_BAD_SHAPE),
    (dict(K=0), Status.ERR_BAD_SHAPE),
    (dict(N=1 << 31), Status.ERR_BAD_SHAPE),
    (dict(M=1 << 21, N=(1 << 31) - 1, K=8, strides=(8, 1, 1, 8, 0, 0)), Status.ERR_BAD_SHAPE),  # 2^41 tiles
    (dict(target_type=2), Status.ERR_DTYPE),
    (dict(label_smoothing=-0.1), Status.ERR_BAD_SHAPE),
    (dict(label_smoothing=float("nan")), Status.ERR_BAD_SHAPE),
    (dict(label_smoothing=1.0), Status.OK),
    (dict(z_loss=-1.0), Status.ERR_BAD_SHAPE),
    (dict(z_loss=float("inf")), Status.ERR_BAD_SHAPE),
    (dict(strides=(40, 1, 1000, 1, 0, 0)), Status.ERR_BAD_STRIDE),
    (dict(strides=(40, 2, 1, 40, 0, 0)), Status.ERR_BAD_STRIDE),
    (dict(strides=(40, 1, 1, 44, 0, 0)), Status.ERR_MISALIGNED),
    (dict(target=T0 + 4), Status.ERR_MISALIGNED),
    (dict(target=T0 + 4, target_type=0), Status.OK),
    (dict(loss=LSE), Status.ERR_ALIAS),
    (dict(loss=T0 + 8), Status.ERR_ALIAS),
    (dict(N=1 << 20, K=4096, strides=(4096, 1, 1, 4096, 0, 0), A=1 << 40, target=1 << 41, lse=1 << 42,
          loss=1 << 43, workspace=1 << 44), Status.OK),  # B of 8 GiB
    (dict(workspace=None), Status.ERR_WORKSPACE),
    (dict(workspace_bytes=64), Status.ERR_WORKSPACE),
])
def test_xent(kw, status):
    assert xent(**kw) == status, tg.last_error_detail()


@pytest.mark.parametrize("kw,status", [
    ({}, Status.OK),
    (dict(dA=None), Status.OK),
    (dict(dB=None), Status.OK),
    (dict(dA=None, dB=None), Status.ERR_NULL_ARG),
    (dict(lse=None), Status.ERR_NULL_ARG),
    (dict(dloss=None), Status.ERR_NULL_ARG),
    (dict(grad_strides=None), Status.ERR_NULL_ARG),
    (dict(piece=-1), Status.ERR_BAD_SHAPE),
    (dict(piece=1), Status.OK),
    (dict(piece=1 << 40), Status.OK),
    (dict(grad_strides=(40, 1, 1000, 1, 0, 0)), Status.ERR_BAD_STRIDE),
    (dict(grad_strides=(32, 1, 1, 40, 0, 0)), Status.ERR_BAD_STRIDE),
    (dict(grad_strides=(40, 1, 1, 44, 0, 0)), Status.ERR_MISALIGNED),
    (dict(dA=A0), Status.ERR_ALIAS),
    (dict(dB=B0), Status.ERR_ALIAS),
    (dict(dA=LSE), Status.ERR_ALIAS),
    (dict(lse=DLOSS), Status.OK),
    (dict(workspace=None), Status.ERR_WORKSPACE),
    (dict(workspace_bytes=64), Status.ERR_WORKSPACE),
    (dict(M=0, A=None, B=None, target=None, lse=None, dloss=None, dA=None, workspace=None), Status.OK),
])
def test_xent_backward(kw, status):
    assert xent(back=True, **kw) == status, tg.last_error_detail()


def test_details_name_the_argument():
    assert glu(dA=A0) == Status.ERR_ALIAS and "dA overlaps A" in tg.last_error_detail()
    assert xent(target=None) == Status.ERR_NULL_ARG and "target" in tg.last_error_detail()
    assert tg.tile_gemm_status_str(Status.ERR_WORKSPACE).startswith("workspace")


@pytest.mark.parametrize("M", [1, 16, 17, 100, 1000, 8192])
@pytest.mark.parametrize("N", [16, 1000 * 16, 131072])
@pytest.mark.parametrize("K", [1, 100, 4096])
def test_workspaces(M, N, K):
    """A call with exactly the size asked for is accepted, one byte less is not;
    a pieced backward pass needs no more than both copies of its pieces' G, the
    fp32 partial results and 256-byte rounding allow."""
    ld = (K + 7) // 8 * 8
    st, gs = (ld, 1, 1, ld, 0, 0), (ld, 1, 1, ld, N // 2, 1)
    far = [i << 44 for i in range(1, 10)]
    need = tg.tile_gemm_glu_backward_workspace(None, M, N, K)
    args = dict(A=far[0], B=far[1], dC=far[2], dA=far[3], dB=far[4], dbias=far[5], bias=None, M=M, N=N, K=K, strides=st,
                grad_strides=gs, workspace=far[6])
    assert tg.tile_gemm_check_glu_backward(workspace_bytes=need, **args) == Status.OK
    assert tg.tile_gemm_check_glu_backward(workspace_bytes=need - 1, **args) == Status.ERR_WORKSPACE
    o = XentOptions(-100, 0.1, 0.0, 0, 1)
    need = tg.tile_gemm_xent_workspace(None, M, N, K, 0.1)
    args = dict(A=far[0], B=far[1], target=far[2], loss=far[3], lse=far[4], M=M, N=N, K=K, strides=st, options=o,
                workspace=far[6])
    assert tg.tile_gemm_check_xent(workspace_bytes=need, **args) == Status.OK
    assert tg.tile_gemm_check_xent(workspace_bytes=need - 1, **args) == Status.ERR_WORKSPACE
    for piece in (0, 256, 1000):
        need = tg.tile_gemm_xent_backward_workspace(None, M, N, K, ld, piece)
        o = XentOptions(-100, 0.0, 0.0, piece, 1)
        args = dict(A=far[0], B=far[1], target=far[2], lse=far[3], dloss=far[4], dA=far[5], dB=far[7], M=M, N=N, K=K,
                    strides=st, grad_strides=st, options=o, workspace=far[6])
        assert tg.tile_gemm_check_xent_backward(workspace_bytes=need, **args) == Status.OK
        assert tg.tile_gemm_check_xent_backward(workspace_bytes=need - 1, **args) == Status.ERR_WORKSPACE


def test_plans():
    """A training product's plan is a partition like a plain product's: tiles
    that cover the output, no more workgroups than pieces of work."""
    for product in tg.TrainProduct:
        for M, N, K in ((1, 1, 1), (1, 131072, 4096), (45, 10928, 4096), (1501, 5488, 4104), (8192, 7168, 8192),
                        (129, 129, 129), (5000, 64, 200000)):
            p = tg.tile_gemm_plan_train(M, N, K, product)
            assert p.tiles_m == -(-M // p.bm) and p.tiles_n == -(-N // p.bn) and p.tiles == p.tiles_m * p.tiles_n
            assert 1 <= p.grid <= p.tiles * p.k_split
            assert p.k_split == 1 or product == tg.TrainProduct.GRADIENT
            cover = 0
            for i in range(min(p.tiles, 4096)):
                _, _, rows, cols = tg.tile_gemm_tile_of(p, M, N, i)
                assert rows > 0 and cols > 0
                cover += rows * cols
            assert p.tiles > 4096 or cover == M * N
    with pytest.raises(tg.TileGemmError):
        tg.tile_gemm_plan_train(0, 1, 1, 0)
    with pytest.raises(tg.TileGemmError):
        tg.tile_gemm_plan_train(1, 1, 1, 3)
    assert tg.tile_gemm_plan_train(101, 999, 77, 0).config < 5  # an odd K: no stream configuration
