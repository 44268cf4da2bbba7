"""What the torch bindings of the gated block hand to the library: strides as
they are. No GPU: host tensors, and the library's own argument checks in place
of its launch."""

import pytest
import torch

import tile_partitioned_dense_amd as tg
from tile_partitioned_dense_amd import Status, binding

K, F = 64, 16


class Checks:
    """Stands for the library: the forward call performs its checks only."""

    def __init__(self, lib):
        self.lib = lib

    def tile_gemm_run_glu(self, h, A, B, C, M, N, K, strides, dtype, bias, gate, stream):
        self.strides = strides._obj
        # (C has the width of one half: checked as the product with that half)
        return self.lib.tile_gemm_check_args(A, B, C, M, N // 2, K, strides, dtype)


@pytest.fixture
def glu(monkeypatch):
    lib = Checks(tg.load_library())
    monkeypatch.setattr(binding, "load_library", lambda: lib)
    monkeypatch.setattr(binding, "_current_device", lambda names, tensors: 0)
    monkeypatch.setattr(binding, "_launch_stream", lambda stream, device: (0, None))

    def call(A, B, C):
        return tg.tile_gemm_run_glu(None, A, B, C, check=False), lib.strides
    return call


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("rows", [1, 2, 5])
def test_columns_apart_are_refused(glu, rows):
    """Any number of rows, one included."""
    w = bf16(2 * F, K).t()
    x, h = bf16(rows, K), bf16(rows, F)
    column_x, column_h = bf16(K, 8)[:, :1].t(), bf16(F, 8)[:, :1].t()
    apart_h = bf16(rows, 2 * F)[:, ::2]
    assert glu(x, w, h)[0] == Status.OK
    for bad in (bf16(rows, 2 * K)[:, ::2], column_x.expand(rows, K)):
        st, s = glu(bad, w, h)
        assert st == Status.ERR_BAD_STRIDE and s.a_k == bad.stride(1) != 1
    for bad in (apart_h, column_h) if rows == 1 else (apart_h,):
        st, s = glu(x, w, bad)
        assert st == Status.ERR_BAD_STRIDE and s.c_n == bad.stride(1) != 1


def test_one_row_of_any_row_stride(glu):
    w = bf16(2 * F, K).t()
    for pitch in (0, 3, K, 2 ** 40):
        x, h = bf16(K).as_strided((1, K), (pitch, 1)), bf16(F).as_strided((1, F), (pitch, 1))
        assert glu(x, w, h)[0] == Status.OK


def test_one_value(glu):
    """An axis of one element has no stride of its own."""
    w = bf16(1, 2 * F)
    for rows in (1, 3):
        x = bf16(rows, 8).as_strided((rows, 1), (8, 5))
        assert glu(x, w, bf16(rows, F))[0] == Status.OK
